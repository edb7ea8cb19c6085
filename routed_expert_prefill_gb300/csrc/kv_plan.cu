// Page tables and row maps of a batch (moe_kv_plan).
#include "api_checks.cuh"

namespace moe {

namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_SEQS = 1024;  // sequences of the one-kernel form, at most
constexpr int PLAN_ROWS = 8192;  // and rows

// What the first kernel leaves for the second, behind the status block.
struct PlanHeader {
  int rows;   // new rows of all sequences
  int taken;  // pages taken
  int top;    // free pages after the others were given back
  int pad;
};

struct PlanParams {
  const int32_t* fresh;    // new tokens, or < 0: the sequence ends
  const int32_t* lens_in;  // may be lens
  int32_t* lens;
  int32_t* table;
  moe_kv_pages pages;
  int n_seq, n_pages, max_blocks, block, t;
  int32_t* starts;
  int32_t* seq;
  int32_t* pos;
  int64_t* slot;
  DeviceStatus* st;
  PlanHeader* head;
  int32_t* held_before;  // [n_seq]
  int32_t* take_off;     // [n_seq]: pages taken by the sequences before
};

// One sequence's part: what it adds, takes and gives back.
struct PlanItem {
  int held, grow, take, give, len;
  bool bad, ends;
};

__device__ __forceinline__ PlanItem plan_item(const PlanParams& p, int s) {
  PlanItem r;
  const int fresh = p.fresh[s], before = p.lens_in[s];
  const int64_t held = p.pages.held[s];
  r.held = (int)held;
  r.grow = max(fresh, 0);
  const int64_t len = (int64_t)before + r.grow, need = (len + p.block - 1) / p.block;
  r.bad = held < 0 || held > p.max_blocks || r.grow > p.t || before < 0 || before > held * p.block ||
          need > p.max_blocks;
  if (fresh < 0) r.bad = held < 0 || held > p.max_blocks;
  r.ends = fresh < 0;
  r.take = fresh < 0 || r.bad ? 0 : (int)max((int64_t)0, need - held);
  r.give = fresh < 0 && !r.bad ? (int)held : 0;
  r.len = fresh < 0 ? 0 : (int)len;
  if (r.bad) r.grow = 0;
  return r;
}

struct PlanSums {
  long long grow, take, give;
};
__device__ __forceinline__ PlanSums operator+(PlanSums a, PlanSums b) { return {a.grow + b.grow, a.take + b.take, a.give + b.give}; }

__device__ __forceinline__ PlanSums warp_scan(PlanSums v, int lane) {  // this lane's included
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const PlanSums u{__shfl_up_sync(~0u, v.grow, o), __shfl_up_sync(~0u, v.take, o), __shfl_up_sync(~0u, v.give, o)};
    if (lane >= o) v = v + u;
  }
  return v;
}
__device__ __forceinline__ PlanSums of_lane(PlanSums v, int from) {
  return {__shfl_sync(~0u, v.grow, from), __shfl_sync(~0u, v.take, from), __shfl_sync(~0u, v.give, from)};
}

// Sums over the threads before this one, and over all, of the CTA.
__device__ PlanSums cta_scan(PlanSums v, PlanSums (&part)[32], PlanSums& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PlanSums in = warp_scan(v, lane);
  __syncthreads();  // part may still be read
  if (lane == 31) part[warp] = in;
  __syncthreads();
  const PlanSums to = warp_scan(part[lane], lane);
  all = of_lane(to, 31);
  const PlanSums before = of_lane(to, warp ? warp - 1 : 0);
  const PlanSums off{in.grow - v.grow, in.take - v.take, in.give - v.give};
  return warp ? off + before : off;
}

// What the rows' maps are made from: in shared memory where one kernel does all.
struct PlanView {
  const int32_t* starts;
  const int32_t* lens;
  const int32_t* held;      // before the call
  const int32_t* take_off;  // pages taken by the sequences before
  PlanHeader h;
};

// The last of n places whose value is at most x (the first one's is): the
// places of the same value before it are empty.
__device__ __forceinline__ int last_at_most(const int32_t* v, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Rows and pages first, first + step, ... of what was decided.
__device__ __forceinline__ void plan_rows(const PlanParams& p, const PlanView& w, int first, int step) {
  for (int i = first; i < p.t; i += step) {
    int seq = -1, pos = -1;
    int64_t slot = -1;
    if (i < w.h.rows) {
      seq = last_at_most(w.starts, p.n_seq, i);
      const int from = w.starts[seq], n = w.starts[seq + 1] - from;
      pos = w.lens[seq] - n + i - from;
      const int b = pos / p.block, held = w.held[seq];
      const int page = b < held ? p.table[(size_t)seq * p.max_blocks + b]
                                : p.pages.free[w.h.top - 1 - (w.take_off[seq] + b - held)];
      slot = (int64_t)page * p.block + pos % p.block;
    }
    if (p.seq) p.seq[i] = seq;
    if (p.pos) p.pos[i] = pos;
    if (p.slot) p.slot[i] = slot;
  }
  for (int i = first; i < w.h.taken; i += step) {  // no more pages than rows are taken
    const int s = last_at_most(w.take_off, p.n_seq, i);
    p.table[(size_t)s * p.max_blocks + w.held[s] + i - w.take_off[s]] = p.pages.free[w.h.top - 1 - i];
  }
}

// Decides about the whole batch, then changes lengths and accounts and gives
// back pages.  One CTA: a batch has a few thousand sequences at most, and the
// decision needs all of their sums.  What bounds it is latency: loads of what
// it checks, a scan, barriers.  ALL (up to PLAN_SEQS sequences, a thread each,
// and PLAN_ROWS rows): it goes on to the rows' maps, from shared memory.
template <bool ALL>
__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(PlanParams p) {
  __shared__ PlanSums part[32];
  __shared__ int32_t kept[4][ALL ? PLAN_SEQS + 1 : 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int count = *p.pages.count;
  PlanItem mine{};
  PlanSums mine_off{0, 0, 0}, sum;
  bool bad = false;
  if (ALL) {
    if (tid < p.n_seq) mine = plan_item(p, tid);
    bad = mine.bad;
    mine_off = cta_scan({mine.grow, mine.take, mine.give}, part, sum);
  } else {
    PlanSums all{0, 0, 0};
    for (int s = tid; s < p.n_seq; s += PLAN_THREADS) {
      const PlanItem r = plan_item(p, s);
      bad |= r.bad;
      all = all + PlanSums{r.grow, r.take, r.give};
    }
    cta_scan(all, part, sum);
  }
  bad = __syncthreads_or(bad) || count < 0 || count > p.n_pages || sum.grow > p.t || count + sum.give > p.n_pages;
  const bool few = !bad && sum.take > count + sum.give;
  // The pages that a warp's sequences give back, a sequence at a time.
  const auto given = [&](int s, const PlanItem& r, const PlanSums& off, auto f) {
    for (uint32_t m = __ballot_sync(~0u, r.give > 0); m; m &= m - 1) {
      const int from = __ffs(m) - 1, n = __shfl_sync(~0u, r.give, from);
      const int to = count + __shfl_sync(~0u, (int)off.give, from);
      const int32_t* row = p.table + (size_t)__shfl_sync(~0u, s, from) * p.max_blocks;
      for (int b = lane; b < n; b += 32) f(to + b, row[b]);
    }
  };
  // All sequences, PLAN_THREADS at a time.
  const auto sequences = [&](auto f) {
    if (ALL) {
      f(tid, mine, mine_off);
    } else {
      PlanSums base{0, 0, 0}, some;
      for (int s0 = 0; s0 < p.n_seq; s0 += PLAN_THREADS) {
        const PlanItem r = s0 + tid < p.n_seq ? plan_item(p, s0 + tid) : PlanItem{};
        const PlanSums off = base + cta_scan({r.grow, r.take, r.give}, part, some);
        base = base + some;
        f(s0 + tid, r, off);
      }
    }
  };
  if (!bad && !few) {  // pages that change hands have to exist
    bool none = false;
    const int top = (int)(count - max(0LL, sum.take - sum.give));  // free pages below it stay
    for (int i = top + tid; i < count; i += PLAN_THREADS) none |= (unsigned)p.pages.free[i] >= (unsigned)p.n_pages;
    if (sum.give)
      sequences([&](int s, const PlanItem& r, const PlanSums& off) {
        given(s, r, off, [&](int, int page) { none |= (unsigned)page >= (unsigned)p.n_pages; });
      });
    bad = __syncthreads_or(none);
  }
  PlanHeader head{0, 0, count, 0};
  if (bad || few) {  // nothing is changed, no sequence has rows
    if (tid == 0) raise_flag(p.st, bad ? FLAG_BAD_CACHE : FLAG_NO_PAGES);
    for (int s = tid; s <= p.n_seq; s += PLAN_THREADS) p.starts[s] = 0;
  } else {
    head = {(int)sum.grow, (int)sum.take, (int)(count + sum.give), 0};
    sequences([&](int s, const PlanItem& r, const PlanSums& off) {
      given(s, r, off, [&](int to, int page) { p.pages.free[to] = page; });
      if (s >= p.n_seq) return;
      p.starts[s] = (int)off.grow;
      p.lens[s] = r.len;
      p.pages.held[s] = r.ends ? 0 : r.held + r.take;
      if (ALL) {
        kept[0][s] = (int)off.grow, kept[1][s] = r.len, kept[2][s] = r.held, kept[3][s] = (int)off.take;
      } else {
        p.held_before[s] = r.held;
        p.take_off[s] = (int)off.take;
      }
    });
    if (tid == 0) {
      p.starts[p.n_seq] = (int)sum.grow;
      if (ALL) kept[0][p.n_seq] = (int)sum.grow;
      *p.pages.count = (int)(count + sum.give - sum.take);
    }
  }
  if (ALL) {
    __syncthreads();
    plan_rows(p, {kept[0], kept[1], kept[2], kept[3], head}, tid, PLAN_THREADS);
  } else if (tid == 0) {
    *p.head = head;
  }
}

__global__ void __launch_bounds__(256) plan_rows_kernel(PlanParams p) {
  pdl_wait();
  pdl_trigger();
  plan_rows(p, {p.starts, p.lens, p.held_before, p.take_off, *p.head}, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

size_t plan_ws_bytes(int n_seq) { return sizeof(DeviceStatus) + 256 + 2 * align_up((size_t)n_seq * 4, 256); }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_kv_plan_workspace_bytes(int32_t n_seq) { return n_seq >= 1 && n_seq <= 65536 ? plan_ws_bytes(n_seq) : 0; }

int moe_kv_plan(const int32_t* fresh, const int32_t* lens_before, int32_t* lens, int32_t* table, const moe_kv_pages* pages,
                int32_t n_seq, int32_t n_pages, int32_t max_blocks, int32_t block, int32_t t, int32_t* starts, int32_t* seq,
                int32_t* pos, int64_t* slot, void* ws, size_t ws_bytes, void* stream) {
  if (!pages) return set_error(MOE_EINVAL, "pages is NULL");
  if (t < 1 || t > 65536) return set_error(MOE_ESHAPE, "t=%d outside [1, 65536]", t);
  if (n_seq < 1 || n_seq > 65536) return set_error(MOE_ESHAPE, "n_seq=%d outside [1, 65536]", n_seq);
  if (n_pages < 1) return set_error(MOE_ESHAPE, "n_pages=%d must be positive", n_pages);
  if (block != 16 && block != 32 && block != 64 && block != 128)
    return set_error(MOE_ESHAPE, "block=%d must be 16, 32, 64 or 128", block);
  if (max_blocks < 1 || (int64_t)max_blocks * block > (1 << 30))
    return set_error(MOE_ESHAPE, "max_blocks=%d: at most 2^30 tokens a sequence", max_blocks);
  TRY(check_ptr(fresh, "fresh", 4));
  TRY(check_ptr(lens_before, "lens_before", 4));
  TRY(check_ptr(lens, "lens", 4));
  TRY(check_ptr(table, "table", 4));
  TRY(check_ptr(pages->free, "pages->free", 4));
  TRY(check_ptr(pages->held, "pages->held", 4));
  TRY(check_ptr(pages->count, "pages->count", 4));
  TRY(check_ptr(starts, "starts", 4));
  TRY(check_ptr(seq, "seq", 4, true));
  TRY(check_ptr(pos, "pos", 4, true));
  TRY(check_ptr(slot, "slot", 8, true));
  if (!ws) return set_error(MOE_EWORKSPACE, "workspace is NULL");
  if ((uintptr_t)ws % 256) return set_error(MOE_EWORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < plan_ws_bytes(n_seq))
    return set_error(MOE_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, plan_ws_bytes(n_seq));
  unsigned char* w = (unsigned char*)ws + sizeof(DeviceStatus);
  const PlanParams p{fresh,  lens_before, lens, table, *pages, n_seq, n_pages, max_blocks, block, t, starts, seq, pos, slot,
                     (DeviceStatus*)ws, (PlanHeader*)w, (int32_t*)(w + 256),
                     (int32_t*)(w + 256 + align_up((size_t)n_seq * 4, 256))};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (n_seq <= PLAN_SEQS && t <= PLAN_ROWS) {
    MOE_LAUNCH("kv_plan", s, { e = launch_k(plan_kernel<true>, dim3(1), dim3(PLAN_THREADS), 0, s, p); });
    return cuda_status(e, "moe_kv_plan launch");
  }
  MOE_LAUNCH("kv_plan", s, { e = launch_k(plan_kernel<false>, dim3(1), dim3(PLAN_THREADS), 0, s, p); });
  TRY(cuda_status(e, "moe_kv_plan launch"));
  MOE_LAUNCH("kv_plan_rows", s, { e = launch_k(plan_rows_kernel, dim3((t + 255) / 256), dim3(256), 0, s, p); });
  return cuda_status(e, "moe_kv_plan rows launch");
}

}  // extern "C"
