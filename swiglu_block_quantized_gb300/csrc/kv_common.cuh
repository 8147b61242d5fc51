// kv_common.cuh -- device helpers of the KV cache operators: the Q8_0 encode
// of a block, the decode of half a block, and the sites of the bounds-checked
// build (common.cuh) in their kernels.
#pragma once

#include "codec.cuh"

namespace m4q {

enum : uint32_t {
  kSiteKvWrite = 31,     // cache write: cache row
  kSiteKvRead = 32,      // cache read: cache row or output row
  kSiteNorm = 33,        // norms: row element
  kSiteTreeQ = 34,       // tree attention: query row
  kSiteTreeKV = 35,      // tree attention: cache rows
  kSiteTreeO = 36,       // tree attention: output row
  kSiteTreeWs = 37,      // tree attention: partial result
  kSitePagedKV = 38,     // paged attention: cache rows
  kSitePagedO = 39,      // paged attention: output row
  kSitePagedWs = 40,     // paged attention: partial result
  kSitePlan = 41,        // page plan: table entry, free page or token
  kSiteVerify = 42,      // verification: probability row
};

// The serving kernels start while the kernel before them may still run (pdl_wait), so
// what an earlier kernel of the stream may have written is read by ordinary loads:
// __ldg is for memory that nobody writes from a kernel's start to its end, and is used
// for the frequency table alone.

// Larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(b));
  return a;
}

// Eight values of a Q8_0 block whose largest magnitude is `top`.  Returns the bits
// of the scale d and 8 code bytes.  d = top / 127 rounded up; q = x / d to the
// nearest integer, ties to even.  x times the rounded reciprocal of d can land
// beside an exact tie; the step q + (x - q d) / d, its remainder exact, ends within
// an fp32 rounding of x / d, so ties are hit and anything farther from one than that
// is not.  A test for ties with a second round of code only where one is met was
// slower (39.1 us against 26.6 for 8,000 tokens of 8 + 8 heads written and read
// back).
__device__ __forceinline__ uint16_t q8_encode8(const float* x, float top, uint32_t (&codes)[2]) {
  const __half dh = __float2half_ru(__fdiv_rn(top, 127.f));
  const uint16_t bits = __half_as_ushort(dh);
  const bool bad = !((bits & 0x7C00u) < 0x7C00u);   // infinity or NaN in the block, or a scale beyond fp16
  const float d = __half2float(dh);
  const float inv = d > 0.f && !bad ? __frcp_rn(d) : 0.f;
  constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it leaves the nearest integer in the low bits
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = x[i] * inv;
    y[i] = __fadd_rn(__fmaf_rn(__fmaf_rn(-q, d, x[i]), inv, q), kMagic);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = __byte_perm(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(y[4 * i + 2]), __float_as_uint(y[4 * i + 3]), 0x0040);
    codes[i] = bad ? 0u : __byte_perm(a, b, 0x5410);
  }
  return bad ? (uint16_t)0x7FFF : bits;
}

// Values 16 u .. 16 u + 15 of a Q8_0 row in global memory, RNE(q d), as fp16
// pairs.  Rows start on 4-byte boundaries (68 or 136 bytes); the codes of an
// odd block are 4-byte aligned, those of an even one 2 bytes past that and
// always followed by the odd block of the same row.
__device__ __forceinline__ void q8_decode16(const uint8_t* row, int u, const DecK& K, uint32_t (&out)[8]) {
  const int blk = u >> 1, off = 34 * blk + 2 + 16 * (u & 1);
  const uint32_t d2 = dup_scale(*reinterpret_cast<const unsigned short*>(row + 34 * blk));
  const uint32_t* w = reinterpret_cast<const uint32_t*>(row + (off & ~3));
  uint32_t a[5];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = w[i];
  a[4] = (blk & 1) ? 0u : w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = (blk & 1) ? a[i] : __funnelshift_r(a[i], a[i + 1], 16);
    out[2 * i] = q8_pair(__byte_perm(c, 0u, 0x4140u), d2, K);
    out[2 * i + 1] = q8_pair(__byte_perm(c, 0u, 0x4342u), d2, K);
  }
}

}  // namespace m4q
