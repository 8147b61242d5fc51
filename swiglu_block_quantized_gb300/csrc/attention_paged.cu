// attention_paged.cu -- attention of one new token of each of B sequences over a paged
// KV cache: O = softmax(scale q K^T) V over the rows j < lengths[b], row j at place
// j % page of page table[b][j / page].
//
// A warp takes a key at a time, its lanes over the head dim; warps of a CTA (one query
// head of one sequence) take the keys in turn and merge their running maximum, sum and
// O at the end.
#include "kv_common.cuh"
#include "launch.h"

namespace m4q {

namespace {

constexpr int kWarps = 8;

template <int D, bool Q8>
__global__ void __launch_bounds__(32 * kWarps) paged_kernel(const PagedParams p) {
  constexpr int E = D / 32;
  constexpr int RB = Q8 ? D / 32 * 34 : 2 * D;
  __shared__ float so[kWarps][D];
  __shared__ float2 sml[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x, b = blockIdx.y, hk = h / p.G;
  pdl_launch_dependents();
  pdl_wait();
  const int len = (int)min((long long)max(p.lengths[b], 0), (long long)p.W * p.page);
  float q[E], o[E], m = -INFINITY, l = 0.f;
  for (int i = 0; i < E; ++i) {
    q[i] = __half2float(p.q[((long long)h * p.B + b) * D + lane * E + i]) * p.scale_log2;
    o[i] = 0.f;
  }
  for (int j = warp; j < len; j += kWarps) {
    const int id = p.table[(long long)b * p.W + j / p.page];
    if ((unsigned)id >= (unsigned)p.P) continue;
    const long long row = ((long long)id * p.Hkv + hk) * p.page + j % p.page;
    if (!in_bounds(row < (long long)p.P * p.Hkv * p.page, p.status, kSitePagedKV)) continue;
    float s = 0.f, v[E];
    for (int kv = 0; kv < 2; ++kv) {
      const uint8_t* r = (kv ? p.v : p.k) + row * RB;
      for (int i = 0; i < E; ++i) {
        const int d = lane * E + i;
        __half x;
        if (Q8) {
          const uint8_t* blk = r + 34 * (d / 32);
          x = __hmul(__int2half_rn((int)(int8_t)blk[2 + d % 32]), __ushort_as_half(*reinterpret_cast<const unsigned short*>(blk)));
        } else {
          x = reinterpret_cast<const __half*>(r)[d];
        }
        if (kv) v[i] = __half2float(x);
        else s += q[i] * __half2float(x);
      }
    }
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    const float top = fmaxf(m, s);
    const float ref = top == -INFINITY ? 0.f : top;
    const float keep = exp2f(m - ref), w = exp2f(s - ref);
    m = top;
    l = l * keep + w;
    for (int i = 0; i < E; ++i) o[i] = o[i] * keep + w * v[i];
  }
  for (int i = 0; i < E; ++i) so[warp][lane * E + i] = o[i];
  if (lane == 0) sml[warp] = make_float2(m, l);
  __syncthreads();
  if (threadIdx.x >= D) return;
  float top = -INFINITY, sum = 0.f, acc = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sml[w].x);
  for (int w = 0; w < kWarps; ++w) {
    const float f = sml[w].x == -INFINITY ? 0.f : exp2f(sml[w].x - top);
    sum += f * sml[w].y;
    acc += f * so[w][threadIdx.x];
  }
  if (!in_bounds(h < p.H && b < p.B, p.status, kSitePagedO)) return;
  p.o[((long long)b * p.H + h) * D + threadIdx.x] = __float2half_rn(sum > 0.f ? acc / sum : 0.f);
}

}  // namespace

cudaError_t launch_attention_paged(const PagedParams& p, bool q8, cudaStream_t s) {
  auto kern = p.D == 64 ? (q8 ? paged_kernel<64, true> : paged_kernel<64, false>)
                        : (q8 ? paged_kernel<128, true> : paged_kernel<128, false>);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)p.H, (unsigned)p.B, 1);
  cfg.blockDim = dim3(32 * kWarps, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace m4q
