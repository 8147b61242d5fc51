// attention_tree.cu -- attention of drafted trees of tokens (or of single new
// tokens, trees of one node) over a batch of KV caches, fp16 or Q8_0.
//
// Node i of sequence b sees the keys j < past[b] of its cache and, at rows
// past[b] + a, its ancestors a and itself.  One warp takes one (sequence,
// head, node) and walks its keys with an online softmax.
#include "kv_common.cuh"
#include "launch.h"

namespace m4q {

namespace {

template <int D, bool Q8>
__device__ __forceinline__ void load_row(const uint8_t* base, long long row, int lane, float (&x)[D / 32]) {
  if constexpr (Q8) {
    const uint8_t* r = base + row * (D / 32 * 34);
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
      const float d = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(r + 34 * b)));
      x[b] = __half2float(__float2half_rn((float)(int8_t)r[34 * b + 2 + lane] * d));
    }
  } else {
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
      x[b] = __half2float(reinterpret_cast<const __half*>(base)[row * D + 32 * b + lane]);
  }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(128) tree_simple_kernel(const TreeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long w = ((long long)blockIdx.x * 128 + threadIdx.x) >> 5;
  if (w >= (long long)p.B * p.N * p.H) return;
  const int h = (int)(w % p.H), i = (int)(w / p.H % p.N), b = (int)(w / p.H / p.N);
  const int* parents = p.parents + (long long)b * p.N;
  const int past = min(max(p.past[b], 0), p.C);
  // the walk to the context: a node is unused if it or an ancestor is
  bool used = true;
  for (int a = i; a >= 0;) {
    const int q = parents[a];
    used = used && q >= -1 && q < a;
    if (!used) break;
    a = q;
  }
  const __half* qrow = p.q + ((long long)h * p.B * p.N + (long long)b * p.N + i) * D;
  float q[D / 32], acc[D / 32], l = 0.f, top = -INFINITY;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    q[c] = __half2float(qrow[32 * c + lane]);
    acc[c] = 0.f;
  }
  const long long head = ((long long)b * p.Hkv + h / p.G) * p.C;
  auto step = [&](long long j) {
    float k[D / 32], v[D / 32];
    load_row<D, Q8>(p.k, head + j, lane, k);
    load_row<D, Q8>(p.v, head + j, lane, v);
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) s += q[c] * k[c];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= p.scale_log2;
    const float now = fmaxf(top, s), a = exp2f(top - now), e = exp2f(s - now);
    l = l * a + e;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[c] = acc[c] * a + e * v[c];
    top = now;
  };
  if (used) {
    for (int j = 0; j < past; ++j) step(j);
    for (int a = i; a >= 0; a = parents[a])
      if (past + a < p.C) step(past + a);
  }
  __half* o = p.o + ((long long)b * p.N + i) * p.H * D + (long long)h * D;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) o[32 * c + lane] = __float2half_rn(l > 0.f || l != l ? acc[c] / l : 0.f);
}

}  // namespace

cudaError_t launch_attention_tree(const TreeParams& p, bool q8, cudaStream_t s) {
  const long long warps = (long long)p.B * p.N * p.H;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((warps + 3) / 4), 1, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  if (p.D == 64) return cudaLaunchKernelEx(&cfg, q8 ? tree_simple_kernel<64, true> : tree_simple_kernel<64, false>, p);
  return cudaLaunchKernelEx(&cfg, q8 ? tree_simple_kernel<128, true> : tree_simple_kernel<128, false>, p);
}

}  // namespace m4q
