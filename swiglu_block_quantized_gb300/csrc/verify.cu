// verify.cu -- drafted trees of tokens verified against the target's probabilities, by
// speculative sampling with the siblings of a node tried in turn (the published rule:
// accept x with probability min(1, p(x) / q(x)), else go on with the normalised
// max(p - q, 0)), so that what comes out is distributed as the target's own samples.
//
// At a node with distributions p and q, after children have been turned down, the
// target's rest is r(x) = max(p(x) - M q(x), 0) up to its sum m, where M is the sum of
// the m's before (1 + ...): max(max(p, 0) - a, 0) - b and so on is one max for a, b >= 0.
// The next child x is taken if u m q(x) < r(x); when none is left the next token is the
// first whose running sum of r exceeds u m.
//
// Decisions stand beside borders, so every difference p - M q and every sum over a row
// is a pair of fp32 values (their exact sum and what its rounding lost: TwoSum, and a
// product's error by fma), good to 2^-45; 64-bit floats would cost more than the
// reading: 16 of them an SM and clock at most.
#include "kv_common.cuh"
#include "launch.h"

namespace m4q {

namespace {

constexpr int kThreads = 1024, kVWarps = kThreads / 32;

struct Two {   // hi + lo, |lo| within an ulp of hi
  float hi, lo;
};
__device__ __forceinline__ Two quick(float a, float b) {   // |a| >= |b| or a = 0
  const float s = __fadd_rn(a, b);
  return {s, __fadd_rn(b, -__fadd_rn(s, -a))};
}
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
  return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return quick(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ bool above(Two a, Two b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ Two shfl_up(Two a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
}
__device__ __forceinline__ Two shfl(Two a, int l) {
  return {__shfl_sync(0xffffffffu, a.hi, l), __shfl_sync(0xffffffffu, a.lo, l)};
}
__device__ __forceinline__ Two warp_scan(Two x, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two y = shfl_up(x, o);
    if (lane >= o) x = add(y, x);
  }
  return x;
}
__device__ __forceinline__ Two warp_sum(Two x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x = add(x, Two{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)});
  return x;
}

// A probability: what is not a finite positive number counts as zero.
__device__ __forceinline__ float prob(float x) { return x > 0.f && x <= 3.402823466e38f ? x : 0.f; }
__device__ __forceinline__ float load(const float* p) { return prob(*p); }
__device__ __forceinline__ float load(const __half* p) { return prob(__half2float(*p)); }

// A row's rest r(x) = max(p(x) - M q(x), 0).
template <typename T>
struct Rest {
  const T* p;
  const T* q;
  float mh, ml;   // M; 0: q is not read
  __device__ __forceinline__ Two operator()(int x) const {
    const float a = load(p + x);
    if (mh == 0.f) return {a, 0.f};
    const float b = load(q + x);
    const float ph = __fmul_rn(mh, b);
    const float pl = __fmaf_rn(ml, b, __fmaf_rn(mh, b, -ph));   // mh b + ml b - ph
    const Two d = two_sum(a, -ph);
    const Two r = quick(d.hi, __fadd_rn(d.lo, -pl));
    return r.hi > 0.f ? r : Two{0.f, 0.f};
  }
};

struct Shared {
  int par[kVerifyNodes], path[kVerifyNodes];
  float p[kVerifyNodes], q[kVerifyNodes], u[kVerifyNodes];
  Two sum[kVWarps];
  Two total;
  int node, count, next, pass;
  double off, mass;
  int strip;
  Two aim;
};

// Sums of r over the strips [lo + w step, lo + (w + 1) step) of [lo, hi), one a warp.
template <typename T>
__device__ void strips(const Rest<T>& r, int lo, int hi, int step, Shared& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long a = lo + (long long)warp * step;
  const int e = (int)min((long long)hi, a + step);
  Two acc = {0.f, 0.f};
  float low = 0.f;
  for (long long x = a + lane; x < e; x += 32) {
    const Two v = r((int)x);
    const Two t = two_sum(acc.hi, v.hi);
    acc.hi = t.hi;
    low = __fadd_rn(low, __fadd_rn(t.lo, v.lo));
  }
  acc = warp_sum(quick(acc.hi, low));
  if (lane == 0) s.sum[warp] = acc;
  __syncthreads();
}

// The first lane whose running sum of v exceeds `aim`, else the last with a value
// above 0 (else -1); `aim` becomes what is left of it at that lane.
__device__ __forceinline__ int pick(Two v, Two& aim, int lane) {
  const Two upto = warp_scan(v, lane);
  const uint32_t over = __ballot_sync(0xffffffffu, above(upto, aim) && v.hi > 0.f);
  const uint32_t some = __ballot_sync(0xffffffffu, v.hi > 0.f);
  const int l = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : -1;
  if (l > 0) {
    const Two before = shfl(upto, l - 1);
    aim = add(aim, Two{-before.hi, -before.lo});
  }
  return l;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyParams p) {
  __shared__ Shared s;
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();
  const T* target = static_cast<const T*>(p.target) + b * p.t_bs;
  const T* draft = static_cast<const T*>(p.draft) + b * p.d_bs;
  if (tid < p.N) {
    const long long at = (long long)b * p.N + tid;
    int par = p.parents[at];
    const int x = p.tokens[at];
    s.u[tid] = p.u[at];
    s.path[tid] = -1;
    if (tid > 0) {
      if (par < 0 || par >= tid || x < 0 || x >= p.V) {
        par = -2;
      } else {
        s.p[tid] = load(target + par * p.t_rs + x);
        s.q[tid] = load(draft + par * p.d_rs + x);
      }
    }
    s.par[tid] = par;
  }
  __syncthreads();
  if (s.par[0] != -1) {   // an unused sequence
    if (tid < p.N) p.path[(long long)b * p.N + tid] = -1;
    if (tid == 0) p.count[b] = 0, p.token[b] = -1;
    return;
  }
  if (tid == 0) {
    s.node = 0, s.count = 1, s.path[0] = 0, s.next = 1;
    s.off = 0., s.mass = 1.;
  }
  const int step = ((p.V + kVWarps - 1) / kVWarps + 31) / 32 * 32;
  Rest<T> r;
  for (;;) {
    // Children in turn, until one is turned down or there are none.
    if (tid == 0) {
      int i = s.next, node = s.node;
      bool down = false;
      for (; i < p.N && !down; ++i) {
        if (s.par[i] != node) continue;
        const double rest = (double)s.p[i] - s.off * (double)s.q[i];
        if ((double)s.u[i] * s.mass * (double)s.q[i] < rest) {
          node = i;
          s.path[s.count++] = i;
          s.off = 0., s.mass = 1.;
        } else {
          down = true;
          s.off += s.mass;
        }
      }
      s.next = i;
      s.node = node;
      s.pass = down;
    }
    __syncthreads();
    const bool more = s.pass;
    r.p = target + s.node * p.t_rs;
    r.q = draft + s.node * p.d_rs;
    r.mh = (float)s.off;
    r.ml = (float)(s.off - (double)r.mh);
    // a node whose rest has been summed (its last child was turned down) is done
    const bool known = !more && s.off > 0.;
    if (!known) {
      strips(r, 0, p.V, step, s);
      if (warp == 0) {
        const Two all = warp_sum(lane < kVWarps ? s.sum[lane] : Two{0.f, 0.f});
        if (lane == 0) {
          s.total = all;
          s.mass = (double)all.hi + (double)all.lo;
        }
      }
      __syncthreads();
    }
    if (!more) break;
  }
  // The target is covered by the draft (only roundings led here): its own samples.
  if (!(s.total.hi > 0.f) && r.mh != 0.f) {
    r.mh = r.ml = 0.f;
    __syncthreads();
    strips(r, 0, p.V, step, s);
    if (warp == 0) {
      const Two all = warp_sum(lane < kVWarps ? s.sum[lane] : Two{0.f, 0.f});
      if (lane == 0) s.total = all;
    }
    __syncthreads();
  }
  // The strip, the strip of the strip, and the token in it.
  int lo = 0, hi = p.V, width = step;
  Two aim = {0.f, 0.f};
  if (warp == 0) {
    const float u = s.u[0];
    const float h = __fmul_rn(u, s.total.hi);
    aim = quick(h, __fmaf_rn(u, s.total.lo, __fmaf_rn(u, s.total.hi, -h)));
  }
  for (int level = 0; level < 2; ++level) {
    if (level) {
      width = ((hi - lo + kVWarps - 1) / kVWarps + 31) / 32 * 32;
      strips(r, lo, hi, width, s);
    }
    if (warp == 0) {
      const int l = pick(lane < kVWarps ? s.sum[lane] : Two{0.f, 0.f}, aim, lane);
      if (lane == 0) s.strip = l;
    }
    __syncthreads();
    if (s.strip < 0) break;
    lo += s.strip * width;
    hi = min(hi, lo + width);
  }
  if (warp == 0) {
    int token = -1;
    if (s.strip >= 0)
      for (int x0 = lo; x0 < hi; x0 += 32) {
        const Two v = x0 + lane < hi ? r(x0 + lane) : Two{0.f, 0.f};
        const Two upto = warp_scan(v, lane);
        const uint32_t over = __ballot_sync(0xffffffffu, above(upto, aim) && v.hi > 0.f);
        const uint32_t some = __ballot_sync(0xffffffffu, v.hi > 0.f);
        if (over) {
          token = x0 + __ffs(over) - 1;
          break;
        }
        if (some) token = x0 + 31 - __clz(some);
        const Two all = shfl(upto, 31);
        aim = add(aim, Two{-all.hi, -all.lo});
      }
    if (lane == 0) {
      p.token[b] = token;
      p.count[b] = s.count;
    }
  }
  if (tid < p.N) p.path[(long long)b * p.N + tid] = s.path[tid];
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, bool f16, cudaStream_t s) {
  return launch_proj(f16 ? verify_kernel<__half> : verify_kernel<float>, (unsigned)p.B, (unsigned)kThreads, 0, s, 1u,
                     p);
}

}  // namespace m4q
