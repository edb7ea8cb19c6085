"""The layer operators at the ends of their ranges: shapes that fill shared
memory, kernel forms that only large sizes reach, caches that are cut back,
waits that run out, very long contexts, very large scores."""

import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_layer import BF16, F64, gen, layer, randn, weights, within  # noqa: E402, F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- qmv

def qmv_case(layer, t, n, k, q8):
    """Every weight row in fp32 against the exact product; the error bound is test_qmv's."""
    g = gen(t + 7 * n + k)
    w, ref_w, mag = weights(g, n, k)
    if q8:
        xc = torch.randint(-127, 128, (t, k), dtype=torch.int8, generator=g, device="cuda")
        xs = torch.rand(t, k // 64, generator=g, device="cuda") * 0.1
        x, rx = (xc, xs), xc.to(F64) * xs.to(F64).repeat_interleave(64, 1)
    else:
        x = randn(g, t, k).bfloat16()
        rx = x.to(F64)
    out = layer.moe_qmv(x, w, out_dtype=torch.float32)
    for i in range(0, n, 8192):
        sl = slice(i, i + 8192)
        tol = (k / 64 + 32) * 2.0 ** -23 * (rx.abs() @ mag[sl].t())
        within(out[:, sl], rx @ ref_w[sl].t(), tol)


# Sizes whose rows of x leave less than 128 bytes of a CTA's shared memory.
@pytest.mark.parametrize("t,n,k", [(4, 4000, 3968), (7, 4000, 4864), (3, 4000, 8640), (2, 4000, 10688), (16, 1000, 3776),
                                   (5, 1000, 12864)])
def test_qmv_rows_that_fill_shared_memory(layer, t, n, k):
    qmv_case(layer, t, n, k, False)
