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
// product's error by fma); the 64-bit units, 2 operations an SM and clock, would need
// several times as long (the walk alone took 5 us of 24 with them).  What is lost in a sum
// is itself summed in fp32, so only the 8 or 16 values of a thread's step share such a sum,
// good to 2^-41; steps and strips are added as pairs, each addition good to 2^-47.  (One sum
// of all of a thread's values, up to 32,768, was off by 2^-26 for equal values and 2^-34 for
// a softmax's; it took 20.9, 17.0 and 16.1 us below, not 21.2, 17.4 and 16.6.)
//
// A sequence is one cluster of CTAs.  All of them walk its nodes (a warp, from shared
// memory; the drafted tokens' p and q are gathered ahead); a row's sum is formed
// by strips, a CTA's and then a warp's, and the CTAs' sums are exchanged through
// distributed shared memory in a fixed order.  The CTA in whose strip the next token lies
// sums its warp's strip again by finer strips, then goes through the one that holds it.
//
// Bound by latency: a row's sum takes about 4 us (its loads, two sums over warps, a cluster
// barrier), one for each child turned down; with many sequences by the 23 to 27 additions a
// value.  16 trees of 8 nodes over 128,000 values in 21.2 us (one CTA a sequence and 4-byte
// loads: 88.6), one chain of 5 over 32,000 in 7.7, 96 chains of 4 over 50,001 fp16 values in
// 17.4, 128 samples (N = 1) from 128,000 fp16 values in 16.6 (2.0 TB/s).
#include <type_traits>

#include "kv_common.cuh"
#include "launch.h"

namespace m4q {

namespace {

constexpr int kThreads = 512, kVWarps = kThreads / 32;
constexpr int kBatch = 2;   // 16-byte vectors of p and of q that a thread has on their way

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
__device__ __forceinline__ Two times(Two a, float b) {
  const float h = __fmul_rn(a.hi, b);
  return quick(h, __fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -h)));
}
__device__ __forceinline__ Two times(Two a, Two b) {
  const float h = __fmul_rn(a.hi, b.hi);
  return quick(h, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.hi, b.hi, -h))));
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

// A probability: what is not a finite positive number counts as zero (as bits: below those
// of infinity, which the sign's, too, lie above).
__device__ __forceinline__ float prob(float x) { return __float_as_uint(x) < 0x7F800000u ? x : 0.f; }
__device__ __forceinline__ float load(const float* p) { return prob(*p); }
__device__ __forceinline__ float load(const __half* p) { return prob(__half2float(*p)); }

// A row's rest r(x) = max(p(x) - M q(x), 0).
__device__ __forceinline__ Two rest_of(float a, float b, float mh, float ml) {
  const float ph = __fmul_rn(mh, b);
  const float pl = __fmaf_rn(ml, b, __fmaf_rn(mh, b, -ph));   // mh b + ml b - ph
  const Two d = two_sum(a, -ph);
  const Two r = quick(d.hi, __fadd_rn(d.lo, -pl));
  return r.hi > 0.f ? r : Two{0.f, 0.f};
}
template <typename T>
struct Rest {
  const T* p;
  const T* q;
  float mh, ml;   // M; 0: q is not read
  // Elements from the 16-byte boundary at or before the row to its start: vectors are cut
  // by p's, q's are read as such where it lies alike (rows of one layout do).
  __device__ __forceinline__ int skew() const { return (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T)); }
  __device__ __forceinline__ bool alike() const {
    return ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
  }
  __device__ __forceinline__ Two operator()(int x) const {
    const float a = load(p + x);
    return mh == 0.f ? Two{a, 0.f} : rest_of(a, load(q + x), mh, ml);
  }
};

struct Shared {
  int par[kVerifyNodes], path[kVerifyNodes];
  float p[kVerifyNodes], q[kVerifyNodes], u[kVerifyNodes];
  Two sum[kVWarps];
  Two mine[2];       // the CTA's sum of a pass, for the others (two passes' in turn)
  Two total, aim;    // of the row; what the next token's running sum has to exceed, in its CTA
  int rank;          // that CTA
  int node, more;          // where the walk stands; whether it goes on once the row is summed
  Two off;                 // M
  int strip;
};

// The 16 bytes of a row from value x on, those outside [a, e) 0: one load where all of
// them are inside and aligned.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int x, int a, int e, bool vec) {
  constexpr int W = 16 / sizeof(T);
  if (vec && x >= a && x + W <= e) return *reinterpret_cast<const uint4*>(row + x);
  uint32_t w[4] = {0, 0, 0, 0};
  if (x >= e) return make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (x + i >= a && x + i < e) {
      if constexpr (sizeof(T) == 4) w[i] = reinterpret_cast<const uint32_t*>(row)[x + i];
      else w[i / 2] |= (uint32_t) reinterpret_cast<const unsigned short*>(row)[x + i] << (16 * (i & 1));
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The probabilities of a vector.
__device__ __forceinline__ void values(const uint4& v, float (&x)[4]) {
  x[0] = prob(__uint_as_float(v.x)), x[1] = prob(__uint_as_float(v.y));
  x[2] = prob(__uint_as_float(v.z)), x[3] = prob(__uint_as_float(v.w));
}
__device__ __forceinline__ void values(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = prob(h.x);
    x[2 * i + 1] = prob(h.y);
  }
}

// Sums of r over the strips [lo + w step, lo + (w + 1) step) of [lo, hi), one a warp.
template <typename T>
__device__ void strips(const Rest<T>& r, int lo, int hi, int step, Shared& s) {
  constexpr int W = 16 / sizeof(T);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int a = min(lo + warp * step, hi), e = min(hi, a + step), skew = r.skew();
  const bool alike = r.alike();
  Two sum = {0.f, 0.f};
  float acc, low;   // a step's values: their sum and what its roundings lost
  auto take = [&](float hi, float lo) {
    const Two t = two_sum(acc, hi);
    acc = t.hi;
    low = __fadd_rn(low, __fadd_rn(t.lo, lo));
  };
  for (int x0 = (a + skew) / W * W - skew + lane * W; x0 < e; x0 += 32 * W * kBatch) {
    acc = low = 0.f;
    uint4 pv[kBatch], qv[kBatch];
    float p[W], q[W];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) pv[i] = load_vec(r.p, x0 + 32 * W * i, a, e, true);
    if (r.mh != 0.f) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) qv[i] = load_vec(r.q, x0 + 32 * W * i, a, e, alike);
      // as rest_of, but for the last step: hi and lo are taken as they are (and after one
      // child, M = 1, the product is q itself)
      auto each = [&](auto one) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          values(pv[i], p);
          values(qv[i], q);
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const float ph = one.value ? q[j] : __fmul_rn(r.mh, q[j]);
            const Two d = two_sum(p[j], -ph);
            const float lo = one.value ? d.lo : __fadd_rn(d.lo, -__fmaf_rn(r.ml, q[j], __fmaf_rn(r.mh, q[j], -ph)));
            const bool some = __fadd_rn(d.hi, lo) > 0.f;
            take(some ? d.hi : 0.f, some ? lo : 0.f);
          }
        }
      };
      if (r.mh == 1.f && r.ml == 0.f) each(std::true_type());
      else each(std::false_type());
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        values(pv[i], p);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const Two t = two_sum(acc, p[j]);
          acc = t.hi;
          low = __fadd_rn(low, t.lo);
        }
      }
    }
    sum = add(sum, two_sum(acc, low));   // (of rests beside 0 `low` may be the larger one)
  }
  const Two all = warp_sum(sum);
  if (lane == 0) s.sum[warp] = all;
  __syncthreads();
}

__device__ __forceinline__ Two peer(const Two* mine, uint32_t rank) {
  Two v;
  const uint32_t at = mapa_shared(smem_u32(mine), rank);
  asm volatile("ld.shared::cluster.f32 %0, [%2];\n\tld.shared::cluster.f32 %1, [%2 + 4];"
               : "=f"(v.hi), "=f"(v.lo)
               : "r"(at)
               : "memory");
  return v;
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
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyParams p) {
  __shared__ Shared s;
  const int ctas = p.ctas, rank = ctas > 1 ? (int)cluster_ctarank() : 0, b = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
      } else if (in_bounds(b < p.B && par < p.N, p.status, kSiteVerify)) {
        s.p[tid] = load(target + par * p.t_rs + x);
        s.q[tid] = load(draft + par * p.d_rs + x);
      }
    }
    s.par[tid] = par;
  }
  __syncthreads();
  if (s.par[0] != -1) {   // an unused sequence
    if (rank == 0 && tid < p.N) p.path[(long long)b * p.N + tid] = -1;
    if (rank == 0 && tid == 0) p.count[b] = 0, p.token[b] = -1;
    return;
  }
  // this CTA's strip of a row, and its warps'
  const int step = ((p.V + ctas * kVWarps - 1) / (ctas * kVWarps) + 31) / 32 * 32;
  const int first = min(rank * kVWarps * step, p.V), last = min(first + kVWarps * step, p.V);
  Rest<T> r;
  int pass = 0;
  // Warp 0's walk: the next node to look at, the current one and how many are kept, M, m,
  // and the CTAs' sums of the last row.
  int next = 1, node = 0, count = 1;
  Two off = {0.f, 0.f}, mass = {1.f, 0.f}, theirs = {0.f, 0.f};
  if (tid == 0) s.path[0] = 0;
  // Sum of r over the row, in s.total; the CTAs' sums stay in their s.mine[pass & 1].
  auto row_sum = [&]() {
    strips(r, first, last, step, s);
    if (warp == 0) {
      const Two all = warp_sum(lane < kVWarps ? s.sum[lane] : Two{0.f, 0.f});
      if (lane == 0) s.mine[pass & 1] = all;
    }
    if (ctas > 1) cluster_sync_all();
    if (warp == 0) {
      __syncwarp();
      theirs = ctas == 1 ? s.mine[pass & 1] : lane < ctas ? peer(&s.mine[pass & 1], lane) : Two{0.f, 0.f};
      mass = ctas > 1 ? warp_sum(theirs) : theirs;
      if (lane == 0) s.total = mass;
    }
    ++pass;
    __syncthreads();
  };
  for (;;) {
    // Children in turn, until one is turned down or there are none.
    if (warp == 0) {
      bool down = false;
      while (!down) {
        uint32_t kids = 0;
        int base = next & ~31;
        for (; base < p.N; base += 32) {
          const int i = base + lane;
          kids = __ballot_sync(0xffffffffu, i >= next && i < p.N && s.par[i] == node);
          if (kids) break;
        }
        if (!kids) break;
        const int i = base + __ffs(kids) - 1;
        next = i + 1;
        // u m q(x) < p(x) - M q(x)
        const Two have = times(mass, times(Two{s.u[i], 0.f}, s.q[i])), part = times(off, s.q[i]);
        const Two rest = add(Two{s.p[i], 0.f}, Two{-part.hi, -part.lo});
        if (above(rest, have)) {
          node = i;
          if (lane == 0) s.path[count] = i;
          ++count;
          off = Two{0.f, 0.f}, mass = Two{1.f, 0.f};
        } else {
          down = true;
          off = add(off, mass);
        }
      }
      if (lane == 0) {
        s.node = node;
        s.more = down;
        s.off = off;
      }
    }
    __syncthreads();
    const bool more = s.more;
    r.p = target + s.node * p.t_rs;
    r.q = draft + s.node * p.d_rs;
    r.mh = s.off.hi;
    r.ml = s.off.lo;
    // a node whose rest has been summed (its last child was turned down) is done
    const bool known = !more && r.mh > 0.f;
    if (!known) row_sum();
    if (!more) break;
  }
  // The target is covered by the draft (only roundings led here): its own samples.
  if (!(s.total.hi > 0.f) && r.mh != 0.f) {
    r.mh = r.ml = 0.f;
    __syncthreads();
    row_sum();
  }
  // The CTA in whose strip the token lies (none of them where p is 0 throughout).
  if (warp == 0) {
    Two aim = times(s.total, s.u[0]);
    int l = s.total.hi > 0.f ? 0 : -1;
    if (ctas > 1) l = pick(theirs, aim, lane);
    if (lane == 0) {
      s.rank = l;
      s.aim = aim;
    }
  }
  __syncthreads();
  if (rank == max(s.rank, 0)) {
    // The warp's strip, the strip of the strip, and the token in it.
    int lo = first, hi = last, width = step;
    Two aim = s.aim;   // (kept by warp 0)
    bool some = s.rank >= 0;
    for (int level = 0; level < 2 && some && (!level || hi - lo > 64); ++level) {
      if (level) {
        width = ((hi - lo + kVWarps - 1) / kVWarps + 31) / 32 * 32;
        strips(r, lo, hi, width, s);
      }
      if (warp == 0) {
        const int l = pick(lane < kVWarps ? s.sum[lane] : Two{0.f, 0.f}, aim, lane);
        if (lane == 0) s.strip = l;
      }
      __syncthreads();
      some = s.strip >= 0;
      lo += max(s.strip, 0) * width;
      hi = min(hi, lo + width);
    }
    if (warp == 0) {
      // Neighbouring values a lane; the lane that holds the token goes through its own.
      int token = -1;
      if (some) {
        const int each = (hi - lo + 31) / 32, x0 = lo + lane * each, x1 = min(x0 + each, hi);
        Two mine = {0.f, 0.f};
#pragma unroll 4
        for (int x = x0; x < x1; ++x) mine = add(mine, r(x));
        const int l = pick(mine, aim, lane);
        if (lane == l) {
          Two upto = {0.f, 0.f};
          for (int x = x0; x < x1; ++x) {
            const Two v = r(x);
            if (!(v.hi > 0.f)) continue;
            token = x;
            upto = add(upto, v);
            if (above(upto, aim)) break;
          }
        }
        token = __shfl_sync(0xffffffffu, token, max(l, 0));
      }
      if (lane == 0) {
        p.token[b] = token;
        p.count[b] = count;
      }
    }
    if (tid < p.N) p.path[(long long)b * p.N + tid] = s.path[tid];
  }
  if (ctas > 1) cluster_sync_all();   // the others have read this CTA's sums
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, bool f16, cudaStream_t s) {
  auto kern = f16 ? verify_kernel<__half> : verify_kernel<float>;
  if (p.ctas > 8) {   // more than every device takes
    std::atomic<unsigned long long>& configured = attr_flag<VerifyParams>();
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load() & bit)) {
      for (auto k : {verify_kernel<__half>, verify_kernel<float>})
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
      configured.fetch_or(bit);
    }
  }
  return launch_proj(kern, (unsigned)(p.B * p.ctas), (unsigned)kThreads, 0, s, (unsigned)p.ctas, p);
}

}  // namespace m4q
