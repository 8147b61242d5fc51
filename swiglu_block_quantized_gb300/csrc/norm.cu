// norm.cu -- the residual update and the norms on both sides of a block in
// one pass over its rows:
//   u  = h / rms(h) * w_post                 (or h, without w_post)
//   r' = res_scale r + branch_scale gate u   (gate: none, [D] or [M][D])
//   y  = r' / rms(r') * w_pre                (rms(x)^2 = mean x^2 + eps)
// Every input is read once and every output written once: a row of up to 8,192
// values stays in the registers of its group of warps (V 16-byte vectors of 8 values a
// thread) between the two reductions.  Sums and r' are fp32; r' is rounded once where
// it is stored, and y is formed from the unrounded r'.
//
// Bound by HBM up to there: 8,192 rows of 4,096 with an fp32 residual, both norms and a
// gate in 67.6 us (6.0 TB/s of the 403 MB it has to move), with an fp16 one in 54 (5.0
// TB/s), 4,096 rows of 8,192 in 75 and 60; 64 rows of 2,048 in 1.8 us, a launch's own
// time.  Wider rows do not fit: 1,024 threads have at most 64 registers each, for 96
// values of r', h and the gate, so that they spill (stacks of 288 bytes a thread with
// an fp32 residual, of 376 with an fp16 one) and local memory bounds them: as many values in rows of 8,200 take 254 and
// 434 us, of 16,384 167 and 264, of 32,768 140 and 187.
#include "kv_common.cuh"
#include "launch.h"

namespace m4q {

namespace {

// Sum over the `warps` warps of a row (a warp group g of the CTA).
template <int W>
__device__ __forceinline__ float row_sum(float x, float (&red)[32], int warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) red[warp] = x;
    __syncthreads();
    const int first = warp / W * W;
    x = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) x += red[first + i];
  }
  return x;
}

__device__ __forceinline__ void half8(const __half* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store_half8(__half* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// W warps a row, V vectors a thread, blockDim.x / (32 W) rows a CTA.
template <int W, int V, bool R32>
__global__ void __launch_bounds__(W > 8 ? 32 * W : 256) norm_kernel(const NormParams p) {
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5;
  const long long row = (long long)blockIdx.x * (blockDim.x / (32 * W)) + threadIdx.x / (32 * W);
  const int t = threadIdx.x % (32 * W);
  const int nv = p.D / 8;
  const bool live = row < p.M;
  pdl_launch_dependents();
  pdl_wait();
  float r[V][8], h[V][8], g[V][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = t + i * 32 * W;
    const bool in = live && v < nv && in_bounds(8 * v + 8 <= p.D, p.status, kSiteNorm);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[i][e] = h[i][e] = 0.f, g[i][e] = 1.f;
    if (!in) continue;
    const long long at = row * p.D + 8 * v;
    if constexpr (R32) {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.r) + at);
      const float4 a = src[0], b = src[1];
      r[i][0] = a.x; r[i][1] = a.y; r[i][2] = a.z; r[i][3] = a.w;
      r[i][4] = b.x; r[i][5] = b.y; r[i][6] = b.z; r[i][7] = b.w;
    } else {
      half8(static_cast<const __half*>(p.r) + at, r[i]);
    }
    if (p.h) half8(p.h + at, h[i]);
    if (p.gate) half8(p.gate + (p.gate_rows ? at : 8 * v), g[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += h[i][e] * h[i][e];
  }
  if (p.h) {
    float scale = 1.f;
    if (p.w_post) scale = rsqrtf(row_sum<W>(ss, red[0], warp) / (float)p.D + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = t + i * 32 * W;
      float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
      if (p.w_post && v < nv) half8(p.w_post + 8 * v, w);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        r[i][e] = p.res_scale * r[i][e] + p.branch_scale * (h[i][e] * scale * w[e] * g[i][e]);
    }
  }
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = t + i * 32 * W;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += r[i][e] * r[i][e];
    if (!p.r_out || !live || v >= nv) continue;
    const long long at = row * p.D + 8 * v;
    if constexpr (R32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.r_out) + at);
      dst[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
      dst[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
    } else {
      store_half8(static_cast<__half*>(p.r_out) + at, r[i]);
    }
  }
  if (!p.y) return;
  const float scale = rsqrtf(row_sum<W>(ss, red[1], warp) / (float)p.D + p.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = t + i * 32 * W;
    if (!live || v >= nv) continue;
    float w[8];
    half8(p.w_pre + 8 * v, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= r[i][e] * scale;
    store_half8(p.y + row * p.D + 8 * v, w);
  }
}

template <int W, int V>
cudaError_t launch_norm(const NormParams& p, bool res32, cudaStream_t s) {
  const int rows = W >= 8 ? 1 : 8 / W;   // rows a CTA
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)((p.M + rows - 1) / rows), 1, 1);
  cfg.blockDim = dim3(32 * W * rows, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, res32 ? norm_kernel<W, V, true> : norm_kernel<W, V, false>, p);
}

}  // namespace

cudaError_t launch_norm_residual(const NormParams& p, bool res32, cudaStream_t s) {
  // one vector a thread up to 256 threads a row, then two, then 1024 threads
  const int nv = p.D / 8;
  if (nv <= 32) return launch_norm<1, 1>(p, res32, s);
  if (nv <= 64) return launch_norm<2, 1>(p, res32, s);
  if (nv <= 128) return launch_norm<4, 1>(p, res32, s);
  if (nv <= 256) return launch_norm<8, 1>(p, res32, s);
  if (nv <= 512) return launch_norm<8, 2>(p, res32, s);
  if (nv <= 1024) return launch_norm<16, 2>(p, res32, s);
  return launch_norm<32, 4>(p, res32, s);
}

}  // namespace m4q
