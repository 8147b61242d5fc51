// kv_common.cuh -- device helpers of the KV cache operators: the Q8_0 encode
// of a block, the decode of half a block, and the sites of the bounds-checked
// build (common.cuh) in their kernels.
#pragma once

#include "codec.cuh"

namespace m4q {

enum : uint32_t {
  kSiteRopeOut = 30,     // rotary positions: output row
  kSiteKvWrite = 31,     // cache write: cache row
  kSiteKvRead = 32,      // cache read: cache row or output row
  kSiteNorm = 33,        // norms: row element
  kSiteTreeQ = 34,       // tree attention: query row
  kSiteTreeKV = 35,      // tree attention: cache rows
  kSiteTreeO = 36,       // tree attention: output row
  kSiteTreeWs = 37,      // tree attention: partial result
};

// Half a Q8_0 block: x[0..15] of this lane and of the lane next to it (lane ^ 1)
// are the block's 32 values.  Returns the bits of the scale d and 16 code
// bytes.  d = max|x| / 127 rounded up; q = x / d to the nearest integer, ties
// to even: x times the rounded reciprocal of d can land on the other side of
// an exact tie, which the exact remainder x - q d shows.  The whole warp calls.
__device__ __forceinline__ uint16_t q8_encode16(const float (&x)[16], uint32_t (&codes)[4]) {
  uint32_t top = 0;   // bits of max|x|; a NaN's are above infinity's
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const __half dh = __float2half_ru(__fdiv_rn(__uint_as_float(top), 127.f));
  const uint16_t bits = __half_as_ushort(dh);
  const bool bad = top >= 0x7F800000u || (bits & 0x7C00u) == 0x7C00u;
  const float d = __half2float(dh), half_d = 0.5f * d;
  const float inv = d > 0.f && !bad ? __frcp_rn(d) : 0.f;
  constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it leaves the nearest integer in the low bits
  uint32_t y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v = bad ? kMagic : __fmaf_rn(x[i], inv, kMagic);
    const float r = v - kMagic;
    const float e = __fmaf_rn(-r, d, x[i]);
    if (fabsf(e) == half_d && (__float_as_uint(v) & 1u) && inv > 0.f) v += e > 0.f ? 1.f : -1.f;
    y[i] = __float_as_uint(v);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __byte_perm(y[4 * i], y[4 * i + 1], 0x0040), b = __byte_perm(y[4 * i + 2], y[4 * i + 3], 0x0040);
    codes[i] = __byte_perm(a, b, 0x5410);
  }
  return bad ? (uint16_t)0x7FFF : bits;
}

// Values 16 u .. 16 u + 15 of a Q8_0 row in global memory, RNE(q d), as fp16
// pairs.  Rows start on 4-byte boundaries (68 or 136 bytes); the codes of an
// odd block are 4-byte aligned, those of an even one 2 bytes past that and
// always followed by the odd block of the same row.
__device__ __forceinline__ void q8_decode16(const uint8_t* row, int u, const DecK& K, uint32_t (&out)[8]) {
  const int blk = u >> 1, off = 34 * blk + 2 + 16 * (u & 1);
  const uint32_t d2 = dup_scale(__ldg(reinterpret_cast<const unsigned short*>(row + 34 * blk)));
  const uint32_t* w = reinterpret_cast<const uint32_t*>(row + (off & ~3));
  uint32_t a[5];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = __ldg(w + i);
  a[4] = (blk & 1) ? 0u : __ldg(w + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = (blk & 1) ? a[i] : __funnelshift_r(a[i], a[i + 1], 16);
    out[2 * i] = q8_pair(__byte_perm(c, 0u, 0x4140u), d2, K);
    out[2 * i + 1] = q8_pair(__byte_perm(c, 0u, 0x4342u), d2, K);
  }
}

}  // namespace m4q
