// page_plan.cu -- the pages of a paged KV cache handed out and taken back, and the
// slots of a step's tokens, from lengths on the device.
//
// Sequence b holds held[b] pages, past[b] of their rows in use, and gets fresh[b] new
// tokens (below 0: it has ended, and its pages go back).  Three running sums over the
// sequences say everything: of the tokens (where b's rows of the step start), of the
// pages that b needs on top of its own, max(0, ceil((past + fresh) / page) - held), and
// of the pages that go back.  The k-th page of the call is free_pages[n_free - 1 - k];
// what goes back lies on top of what is left, so a page is handed out again from the
// next call on.  Integers throughout: the result does not depend on any order.
//
// One launch, one cluster.  Every CTA forms the sums for itself (B is at most 4096), then
// takes its share of the sequences (new table entries) and of the tokens (a thread a
// token: its sequence by bisection, its page from the table or straight from the free
// ones).  The state that all of them read is written after a cluster barrier.  Bound by
// latency: a load, the sums, a load and a store in a chain.  64 sequences of one token take
// 3.2 us, 256 of up to 127 with room for 16,384 tokens 6.3 (28.0 with one CTA).
#include "kv_common.cuh"
#include "launch.h"

namespace m4q {

namespace {

// Exclusive running sums of x and y over the CTA's threads, and their totals.
struct Sums {
  long long x, y, all_x, all_y;
};
__device__ __forceinline__ long long warp_upto(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}
__device__ __forceinline__ Sums scan(long long x, long long y, longlong2* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const long long ux = warp_upto(x, lane), uy = warp_upto(y, lane);
  __syncthreads();
  if (lane == 31) part[warp] = make_longlong2(ux, uy);
  __syncthreads();
  const longlong2 mine = lane < warps ? part[lane] : make_longlong2(0, 0);
  const long long wx = warp_upto(mine.x, lane), wy = warp_upto(mine.y, lane);
  Sums s;
  s.all_x = __shfl_sync(0xffffffffu, wx, 31);
  s.all_y = __shfl_sync(0xffffffffu, wy, 31);
  s.x = ux - x + (warp ? __shfl_sync(0xffffffffu, wx, warp - 1) : 0);
  s.y = uy - y + (warp ? __shfl_sync(0xffffffffu, wy, warp - 1) : 0);
  return s;
}

// Pages of `rows` rows, at most W (rows + page may be past 32 bits).
__device__ __forceinline__ int pages_of(const PlanParams& p, uint32_t rows) {
  const uint32_t n = rows / p.page;
  return (int)min(n + (n * p.page < rows ? 1u : 0u), (uint32_t)p.W);
}

__global__ void __launch_bounds__(1024) plan_kernel(const PlanParams p) {
  extern __shared__ int mem[];
  int* starts = mem;               // [B + 1]
  int* first = starts + p.B + 1;   // [B] pages of this call before b's (b ended: pages back before b's)
  int* held = first + p.B;         // [B]
  int* past = held + p.B;          // [B]; -1: ended
  __shared__ longlong2 part[32];
  const int threads = blockDim.x, rank = p.ctas > 1 ? (int)cluster_ctarank() : 0;
  pdl_launch_dependents();
  pdl_wait();
  const int avail = min(max(p.n_free[0], 0), p.P);
  long long tokens = 0, takes = 0, backs = 0;
  for (int b0 = 0; b0 < p.B; b0 += threads) {
    const int b = b0 + threadIdx.x;
    int fresh = 0, h = 0, n = 0;
    if (b < p.B) {
      fresh = p.fresh[b];
      h = min(max(p.held[b], 0), p.W);
      n = max(p.past[b], 0);
    }
    const Sums t = scan(max(fresh, 0), 0, part);
    const int s0 = (int)min(tokens + t.x, (long long)p.T);
    const int s1 = (int)min(tokens + t.x + max(fresh, 0), (long long)p.T);
    tokens += t.all_x;
    long long take = 0;
    if (b < p.B && fresh >= 0) take = max(pages_of(p, (uint32_t)n + (uint32_t)(s1 - s0)) - h, 0);
    const Sums g = scan(take, fresh < 0 ? h : 0, part);
    if (b < p.B) {
      starts[b] = s0;
      first[b] = (int)min(fresh < 0 ? backs + g.y : takes + g.x, (long long)INT32_MAX);
      held[b] = h;
      past[b] = fresh < 0 ? -1 : n;
      if (rank == 0) p.starts[b] = s0;
      if (b == p.B - 1) {
        starts[p.B] = s1;
        if (rank == 0) p.starts[p.B] = s1;
      }
    }
    takes += g.all_x;
    backs += g.all_y;
  }
  __syncthreads();
  const int left = avail - (int)min(takes, (long long)avail);   // free pages that stay
  // The k-th page of the call.
  auto page_of = [&](long long k) { return k < avail ? p.free_pages[avail - 1 - k] : -1; };
  auto want_of = [&](int b) { return pages_of(p, (uint32_t)past[b] + (uint32_t)(starts[b + 1] - starts[b])); };
  // Slots: a thread a token, its sequence the last that starts at or before it.
  const int used = starts[p.B];
  for (int t = rank * threads + threadIdx.x; t < p.T; t += p.ctas * threads) {
    int slot = -1, pos = 0;
    if (t < used) {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= t) lo = mid;
        else hi = mid;
      }
      const uint32_t at = (uint32_t)past[lo] + (uint32_t)(t - starts[lo]);
      pos = (int)min(at, (uint32_t)INT32_MAX);
      const uint32_t j = at / p.page;
      if (j < (uint32_t)p.W && in_bounds(lo < p.B && t < p.T, p.status, kSitePlan)) {
        const int id = (int)j < held[lo] ? p.table[(long long)lo * p.W + j] : page_of((long long)first[lo] + (int)j - held[lo]);
        if ((unsigned)id < (unsigned)p.P) slot = id * p.page + (int)(at - j * p.page);
      }
    }
    p.slots[t] = slot;
    p.pos[t] = pos;
  }
  // Pages handed out: a thread a sequence where few are (a decode step), else a warp.
  const int lane = threadIdx.x & 31;
  const bool few = takes <= 2ll * p.B;
  for (int b = few ? rank * threads + threadIdx.x : (rank * threads + threadIdx.x) >> 5; b < p.B;
       b += few ? p.ctas * threads : p.ctas * threads / 32) {
    if (past[b] < 0) continue;
    const int want = want_of(b);
    for (int j = held[b] + (few ? 0 : lane); j < want; j += few ? 1 : 32)
      p.table[(long long)b * p.W + j] = page_of((long long)first[b] + j - held[b]);
  }
  // From here on what every CTA has read is written.
  if (p.ctas > 1) cluster_sync_all();
  else __syncthreads();
  for (int b = rank * threads + threadIdx.x; b < p.B; b += p.ctas * threads) {
    int now = 0, rows = 0;
    if (past[b] >= 0) {
      now = held[b] + max(min(want_of(b) - held[b], avail - first[b]), 0);
      rows = (int)min((long long)past[b] + starts[b + 1] - starts[b], (long long)now * p.page);
    }
    p.held[b] = now;
    p.lengths[b] = rows;
  }
  if (rank == 0 && threadIdx.x == 0) p.n_free[0] = (int)min((long long)left + backs, (long long)p.P);
  if (backs)
    for (int b = (rank * threads + threadIdx.x) >> 5; b < p.B; b += p.ctas * threads / 32) {
      if (past[b] >= 0) continue;
      for (int j = lane; j < held[b]; j += 32) {
        int32_t* entry = p.table + (long long)b * p.W + j;
        const long long to = (long long)left + first[b] + j;
        if (to < p.P) p.free_pages[to] = *entry;
        *entry = -1;
      }
    }
}

}  // namespace

cudaError_t launch_page_plan(const PlanParams& p, int threads, cudaStream_t s) {
  const size_t smem = (4 * (size_t)p.B + 1) * sizeof(int);
  std::atomic<unsigned long long>& configured = attr_flag<PlanParams>();
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)((4 * (size_t)kPlanSeqs + 1) * sizeof(int)));
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  return launch_proj(plan_kernel, (unsigned)p.ctas, (unsigned)threads, smem, s, (unsigned)p.ctas, p);
}

}  // namespace m4q
