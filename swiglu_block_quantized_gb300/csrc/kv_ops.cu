// kv_ops.cu -- rotary positions, and the rows of the KV cache written (with
// the rotation fused in) and read back.  The cache is m4q_attention's and
// m4q_attention_tree's: rows of D values, fp16 or Q8_0 blocks along D.
//
// Rotation.  Pair i of the first `rot` values of a row at position n turns by
// n f_i: (a, b) -> s (a cos - b sin, b cos + a sin), with b rot / 2 values
// after a (half layout) or next to it (interleaved).  The table holds f_i as
// turns per position in units of 2^-64, so n f_i mod 2^64 is the fraction of
// a turn, exactly: no position, however far, costs the angle any accuracy
// (an fp32 product is off by 0.03 rad at position 10^6), and no 64-bit float
// is needed.  The fraction is cut to the nearest quarter turn in integers,
// and the remainder (at most 1/8 turn, 30 bits) goes to fp32 and sincospif: at most
// 2^-28 of a turn off, where an fp16 result is rounded by 2^-11.  (Of Q8_0 codes one
// beside a tie may go the other way, as it may with sines rounded from 64 bits: a
// prompt's rows are off by 2.6e-5 and 2.9e-5 of their size.)
//
// Quantisation of a block of 32 values x (Q8_0): d = max|x| / 127 rounded up
// to fp16, so that no code is cut off at 127 even where d is subnormal; codes
// q = x / d to the nearest integer, ties to even.  Rotated keys are quantised
// from their fp32 values (one rounding, not two).  A block that holds an
// infinity or a NaN, or whose d is beyond fp16, gets d = NaN and so decodes
// to NaN throughout.
//
// Work.  A unit is 16 values of a row: the 8 + 8 of eight pairs in the half
// layout, 16 neighbours otherwise, read and written as 16-byte vectors.  A
// thread keeps one (token, unit), forms its eight sines and cosines once and
// walks the heads of its chunk with them; the D / 16 threads of a row are
// neighbours in a warp.  A quantised row exchanges the largest magnitudes of its
// vectors there (a block's vectors may come from units rot / 2 apart), not its
// values (25.5 us against 26.6 for the write and read back below).  The next
// head's vectors are under way while a head is turned and packed (31.5 to 26.6 us,
// and 25.4 to 24.9 for the rotation).
//
// Bound by memory from a few thousand tokens on, by the launch below that.
// Measured: 32 heads of 8,192 tokens, 128 values, rotated in 24.9 us (5.4 TB/s
// of input and output), of 128 tokens in 3.1 us; 8,000 tokens of 8 + 8 heads
// written to Q8_0 rows and read back in 25.6 us (3.9 TB/s); 32,000 Q8_0 rows of
// 8 heads read back in 17.9 us (5.6 TB/s).
#include <type_traits>

#include "kv_common.cuh"
#include "launch.h"

namespace m4q {

namespace {

constexpr int kBlock = 128;   // threads a CTA

struct Turn8 {
  float c[8], s[8];
};

// cos and sin of pos * f turns, f in units of 2^-64.
__device__ __forceinline__ void turn(int pos, int64_t f, float mscale, float& c, float& s) {
  const uint64_t t = (uint64_t)(int64_t)pos * (uint64_t)f;          // fraction of a turn, exact mod 1
  const uint32_t q = (uint32_t)((t + (1ull << 61)) >> 62);          // nearest quarter turn
  const int64_t r = (int64_t)(t - ((uint64_t)q << 62));             // remainder in [-2^61, 2^61)
  float sn, cs;
  sincospif((float)(int)(r >> 32) * 0x1p-31f, &sn, &cs);
  const float a = (q & 1) ? sn : cs, b = (q & 1) ? cs : sn;         // quarter turns swap and flip
  c = (((q + 1) & 2) ? -a : a) * mscale;
  s = ((q & 2) ? -b : b) * mscale;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where the two vectors of unit u start in a row, and whether it is rotated.
struct UnitAt {
  int lo, hi;
  bool turns;
};
__device__ __forceinline__ UnitAt unit_at(int u, int rot, bool interleaved) {
  UnitAt a;
  a.turns = 16 * u < rot;
  const bool split = a.turns && !interleaved;
  a.lo = split ? 8 * u : 16 * u;
  a.hi = split ? 8 * u + rot / 2 : 16 * u + 8;
  return a;
}

// x[0..7] the unit's first vector, x[8..15] its second.
__device__ __forceinline__ void rotate16(float (&x)[16], const Turn8& t, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * t.c[i] - b * t.s[i];
      x[2 * i + 1] = b * t.c[i] + a * t.s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = x[i + 8];
      x[i] = a * t.c[i] - b * t.s[i];
      x[i + 8] = b * t.c[i] + a * t.s[i];
    }
  }
}

// Grid: x over token tiles, y over chunks of `per` of the H + 2 Hkv heads
// (Q heads, then K, then V).  D / 16 threads a token.
template <int D, bool Q8>
__global__ void __launch_bounds__(kBlock) rope_kv_kernel(const KvOpsParams p, int per) {
  constexpr int U = D / 16;                  // units (threads) a row
  constexpr int RB = Q8 ? D / 32 * 34 : 2 * D;
  constexpr int kRowsPerWarp = 32 / U;
  // a warp's rows: the largest magnitudes of 8 values each, then the packed bytes
  constexpr int kTops = D / 8 + 4;
  __shared__ __align__(16) float tops[Q8 ? kBlock / 32 : 1][Q8 ? kRowsPerWarp * kTops : 4];
  __shared__ __align__(16) uint16_t packed[Q8 ? kBlock / 32 : 1][Q8 ? kRowsPerWarp * RB / 2 : 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = threadIdx.x % U, rw = lane / U;
  const long long m = (long long)blockIdx.x * (kBlock / U) + threadIdx.x / U;
  const bool ok = m < p.M;
  const int heads = p.H + 2 * p.Hkv;
  const int h0 = (int)blockIdx.y * per, h1 = min(heads, h0 + per);
  pdl_launch_dependents();
  pdl_wait();
  const UnitAt at = unit_at(u, p.rot, p.interleaved);
  Turn8 t;
  if (ok && at.turns && h0 < p.H + p.Hkv) {
    const int pos = p.pos[m];
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(pos, __ldg(reinterpret_cast<const long long*>(p.freqs) + 8 * u + i), p.mscale, t.c[i], t.s[i]);
  }
  long long row = -1;                        // this token's cache row of head 0, or -1
  if (ok && h1 > p.H) {
    const int slot = p.slots[m];
    if (slot >= 0 && (long long)slot < (long long)p.B * p.C)
      row = (long long)(slot / p.C) * p.Hkv * p.C + slot % p.C;
  }
  // A head's two vectors are loaded one head ahead of their use.
  auto fetch = [&](int h, uint4& v0, uint4& v1) {
    const bool q = h < p.H, v = h >= p.H + p.Hkv;
    v0 = v1 = make_uint4(0, 0, 0, 0);
    if (h < h1 && ok && (q || row >= 0)) {
      const RowsView& src = q ? p.q : v ? p.v : p.k;
      const __half* s = src.p + (q ? h : v ? h - p.H - p.Hkv : h - p.H) * src.hs + m * src.rs;
      v0 = __ldcs(reinterpret_cast<const uint4*>(s + (v ? 16 * u : at.lo)));
      v1 = __ldcs(reinterpret_cast<const uint4*>(s + (v ? 16 * u + 8 : at.hi)));
    }
  };
  uint4 n0, n1;
  fetch(h0, n0, n1);
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const bool isq = h < p.H, isv = h >= p.H + p.Hkv;
    const int hh = isq ? h : isv ? h - p.H - p.Hkv : h - p.H;
    const bool work = ok && (isq || row >= 0);
    const int lo = isv ? 16 * u : at.lo, hi = isv ? 16 * u + 8 : at.hi;
    uint4 v0 = n0, v1 = n1;
    fetch(h + 1, n0, n1);
    const bool turns = at.turns && !isv;
    if (isq || !Q8) {
      if (!work) continue;
      if (turns) {
        float x[16];
        unpack8(v0, *reinterpret_cast<float(*)[8]>(x));
        unpack8(v1, *reinterpret_cast<float(*)[8]>(x + 8));
        rotate16(x, t, p.interleaved);
        v0 = pack8(x);
        v1 = pack8(x + 8);
      }
      __half* d;
      if (isq) {
        d = p.qo + hh * p.qo_hs + m * p.qo_rs;
      } else {
        const long long at_row = row + (long long)hh * p.C;
        if (!in_bounds(at_row < (long long)p.B * p.Hkv * p.C, p.status, kSiteKvWrite)) continue;
        d = reinterpret_cast<__half*>((isv ? p.vc : p.kc) + at_row * RB);
      }
      *reinterpret_cast<uint4*>(d + lo) = v0;
      *reinterpret_cast<uint4*>(d + hi) = v1;
    } else if constexpr (Q8) {
      float x[16];
      unpack8(v0, *reinterpret_cast<float(*)[8]>(x));
      unpack8(v1, *reinterpret_cast<float(*)[8]>(x + 8));
      if (turns) rotate16(x, t, p.interleaved);
      // the largest magnitudes of the two vectors' blocks
      float t0 = 0.f, t1 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t0 = max_nan(t0, fabsf(x[i]));
        t1 = max_nan(t1, fabsf(x[8 + i]));
      }
      float* top = &tops[warp][rw * kTops];
      __syncwarp();
      top[lo >> 3] = t0;
      top[hi >> 3] = t1;
      __syncwarp();
      const float4 b0 = *reinterpret_cast<const float4*>(top + 4 * (lo >> 5));
      const float4 b1 = *reinterpret_cast<const float4*>(top + 4 * (hi >> 5));
      uint32_t c0[2], c1[2];
      const uint16_t d0 = q8_encode8(x, max_nan(max_nan(b0.x, b0.y), max_nan(b0.z, b0.w)), c0);
      const uint16_t d1 = q8_encode8(x + 8, max_nan(max_nan(b1.x, b1.y), max_nan(b1.z, b1.w)), c1);
      // packed row: block b at byte 34 b
      uint16_t* pr = &packed[warp][rw * (RB / 2)];
      uint16_t* p0 = pr + 17 * (lo >> 5) + ((lo & 31) >> 1);
      uint16_t* p1 = pr + 17 * (hi >> 5) + ((hi & 31) >> 1);
      if (!(lo & 31)) p0[0] = d0;
      if (!(hi & 31)) p1[0] = d1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        p0[1 + 2 * i] = (uint16_t)c0[i];
        p0[2 + 2 * i] = (uint16_t)(c0[i] >> 16);
        p1[1 + 2 * i] = (uint16_t)c1[i];
        p1[2 + 2 * i] = (uint16_t)(c1[i] >> 16);
      }
      __syncwarp();
      // the row's threads copy it out in whole 8-byte (D = 128) or 4-byte words
      if (!work) continue;
      const long long at_row = row + (long long)hh * p.C;
      if (!in_bounds(at_row < (long long)p.B * p.Hkv * p.C, p.status, kSiteKvWrite)) continue;
      using Word = typename std::conditional<RB % 8 == 0, uint2, uint32_t>::type;
      const Word* from = reinterpret_cast<const Word*>(&packed[warp][rw * (RB / 2)]);
      Word* to = reinterpret_cast<Word*>((isv ? p.vc : p.kc) + at_row * RB);
      for (int i = u; i < RB / (int)sizeof(Word); i += U) to[i] = from[i];
    }
  }
}

// Cache rows slots[j] of every KV head to fp16 [Hkv][n][D]: a thread per 16
// values; z = 0 reads K, 1 reads V.  Rows whose slot is outside the cache
// give zeros.
template <int D, bool Q8>
__global__ void __launch_bounds__(kBlock) kv_read_kernel(const KvReadParams p) {
  constexpr int U = D / 16;
  constexpr int RB = Q8 ? D / 32 * 34 : 2 * D;
  pdl_launch_dependents();
  pdl_wait();
  const uint8_t* cache = blockIdx.z ? p.vc : p.kc;
  __half* dst = blockIdx.z ? p.vo : p.ko;
  const long long j = (long long)blockIdx.x * (kBlock / U) + threadIdx.x / U;
  if (!dst || j >= p.n) return;
  const int u = threadIdx.x % U, h = blockIdx.y;
  const int slot = p.slots[j];
  uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (slot >= 0 && (long long)slot < (long long)p.B * p.C) {
    const long long row = ((long long)(slot / p.C) * p.Hkv + h) * p.C + slot % p.C;
    if (!in_bounds(row < (long long)p.B * p.Hkv * p.C, p.status, kSiteKvRead)) return;
    if constexpr (Q8) {
      q8_decode16(cache + row * RB, u, make_deck(), out);
    } else {
      const uint4* s = reinterpret_cast<const uint4*>(cache + row * RB) + 2 * u;
      const uint4 a = s[0], b = s[1];
      out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
      out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
    }
  }
  uint4* o = reinterpret_cast<uint4*>(dst + ((long long)h * p.n + j) * D) + 2 * u;
  o[0] = make_uint4(out[0], out[1], out[2], out[3]);
  o[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

template <typename P, typename... More>
cudaError_t launch_grid(void (*kern)(P, More...), dim3 grid, cudaStream_t s, const P& p, More... more) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kBlock, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p, more...);
}

}  // namespace

cudaError_t launch_rope_kv(const KvOpsParams& p, bool q8, cudaStream_t s) {
  const int heads = p.H + 2 * p.Hkv;
  const int tokens = kBlock / (p.D / 16);   // a CTA's
  const long long tiles = ((long long)p.M + tokens - 1) / tokens;
  // Heads a thread walks with its sines and cosines: as many as still leave
  // eight CTAs an SM, at most 8 (their cost is then well under the copy's).  (Of the
  // Q8_0 kernels seven fit an SM: the 8,000 tokens above are 1,500 CTAs of 6, 6 and 4
  // heads, 1.4 waves; the 8,192 rotated ones are 1.7.)
  long long per = tiles * heads / (8ll * (p.nsm > 0 ? p.nsm : 1));
  per = per < 1 ? 1 : per > 8 ? 8 : per;
  const dim3 grid((unsigned)tiles, (unsigned)((heads + per - 1) / per), 1);
  if (p.D == 64) return launch_grid(q8 ? rope_kv_kernel<64, true> : rope_kv_kernel<64, false>, grid, s, p, (int)per);
  return launch_grid(q8 ? rope_kv_kernel<128, true> : rope_kv_kernel<128, false>, grid, s, p, (int)per);
}

cudaError_t launch_kv_read(const KvReadParams& p, bool q8, cudaStream_t s) {
  const int tokens = kBlock / (p.D / 16);
  const dim3 grid((unsigned)(((long long)p.n + tokens - 1) / tokens), (unsigned)p.Hkv, 2);
  if (p.D == 64) return launch_grid(q8 ? kv_read_kernel<64, true> : kv_read_kernel<64, false>, grid, s, p);
  return launch_grid(q8 ? kv_read_kernel<128, true> : kv_read_kernel<128, false>, grid, s, p);
}

}  // namespace m4q
