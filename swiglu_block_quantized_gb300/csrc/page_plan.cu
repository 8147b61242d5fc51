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
#include "kv_common.cuh"
#include "launch.h"

namespace m4q {

namespace {

constexpr int kThreads = 1024;

// Exclusive running sum over the CTA's threads; `total` is the whole sum.
__device__ __forceinline__ long long scan(long long x, long long* part, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long in = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += y;
  }
  __syncthreads();
  if (lane == 31) part[warp] = in;
  __syncthreads();
  long long before = 0;
  total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  return before + in - x;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanParams p) {
  __shared__ int starts[kPlanSeqs + 1];
  __shared__ int first[kPlanSeqs];   // pages of this call before b's (b ended: pages back before b's)
  __shared__ long long part[kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int avail = min(max(p.n_free[0], 0), p.P);
  long long tokens = 0, takes = 0, backs = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int fresh = 0, held = 0, past = 0;
    if (b < p.B) {
      fresh = p.fresh[b];
      held = min(max(p.held[b], 0), p.W);
      past = max(p.past[b], 0);
    }
    long long sum;
    const long long at = tokens + scan(max(fresh, 0), part, sum);
    tokens += sum;
    const int s0 = (int)min(at, (long long)p.T), s1 = (int)min(at + max(fresh, 0), (long long)p.T);
    long long take = 0, back = 0;
    if (fresh < 0) back = held;
    else if (b < p.B) take = max(min(((long long)past + (s1 - s0) + p.page - 1) / p.page, (long long)p.W) - held, 0ll);
    const long long t0 = takes + scan(take, part, sum);
    takes += sum;
    const long long k0 = backs + scan(back, part, sum);
    backs += sum;
    if (b < p.B) {
      starts[b] = s0;
      first[b] = (int)min(fresh < 0 ? k0 : t0, (long long)INT32_MAX);
      p.starts[b] = s0;
      if (b == p.B - 1) starts[p.B] = p.starts[p.B] = s1;
    }
  }
  __syncthreads();
  const int left = avail - (int)min(takes, (long long)avail);   // free pages that stay
  // Pages handed out, a warp a sequence.
  const int lane = threadIdx.x & 31;
  for (int b = threadIdx.x >> 5; b < p.B; b += kThreads / 32) {
    if (p.fresh[b] < 0) continue;
    const int held = min(max(p.held[b], 0), p.W), n = starts[b + 1] - starts[b];
    const long long past = max(p.past[b], 0);
    const int want = (int)min((past + n + p.page - 1) / p.page, (long long)p.W);
    for (int j = held + lane; j < want; j += 32) {
      const long long k = (long long)first[b] + j - held;
      p.table[(long long)b * p.W + j] = k < avail ? p.free_pages[avail - 1 - k] : -1;
    }
  }
  __syncthreads();
  // Pages back on the free ones, and each sequence's new state.
  for (int b = threadIdx.x >> 5; b < p.B; b += kThreads / 32) {
    const int held = min(max(p.held[b], 0), p.W);
    __syncwarp();
    if (p.fresh[b] < 0) {
      for (int j = lane; j < held; j += 32) {
        int32_t* entry = p.table + (long long)b * p.W + j;
        const long long to = (long long)left + first[b] + j;
        if (to < p.P) p.free_pages[to] = *entry;
        *entry = -1;
      }
      if (lane == 0) {
        p.held[b] = 0;
        p.lengths[b] = 0;
      }
    } else if (lane == 0) {
      const long long rows = (long long)max(p.past[b], 0) + starts[b + 1] - starts[b];
      const int want = (int)min((rows + p.page - 1) / p.page, (long long)p.W);
      const int got = max(min(want - held, avail - first[b]), 0);
      p.held[b] = held + got;
      p.lengths[b] = (int)min(rows, (long long)(held + got) * p.page);
    }
  }
  if (threadIdx.x == 0) p.n_free[0] = (int)min((long long)left + backs, (long long)p.P);
  // Slots: a thread a token, its sequence the last that starts at or before it.
  const int used = starts[p.B];
  for (int t = threadIdx.x; t < p.T; t += kThreads) {
    int slot = -1, pos = 0;
    if (t < used) {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= t) lo = mid;
        else hi = mid;
      }
      const long long at = (long long)max(p.past[lo], 0) + t - starts[lo];
      pos = (int)min(at, (long long)INT32_MAX);
      const long long j = at / p.page;
      if (j < p.W && in_bounds(lo < p.B && t < p.T, p.status, kSitePlan)) {
        const int id = p.table[(long long)lo * p.W + j];
        if ((unsigned)id < (unsigned)p.P) slot = id * p.page + (int)(at % p.page);
      }
    }
    p.slots[t] = slot;
    p.pos[t] = pos;
  }
}

}  // namespace

cudaError_t launch_page_plan(const PlanParams& p, cudaStream_t s) {
  return launch_proj(plan_kernel, 1u, (unsigned)kThreads, 0, s, 1u, p);
}

}  // namespace m4q
