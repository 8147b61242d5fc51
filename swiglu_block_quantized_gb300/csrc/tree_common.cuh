// tree_common.cuh -- what the kernels of m4q_attention_tree share: the even
// split of all key tiles over the CTAs, the masks of the tiles that hold a
// tree, the decode of raw Q8_0 tiles and the handling of non-finite values.
#pragma once

#include "kv_common.cuh"
#include "launch.h"
#include "tc_attn.cuh"

namespace m4q {

constexpr int kTile = 128;         // keys of a tile
constexpr float kRaise = 8.f;      // reference kept while a row's maximum stays within 2^8 of it

// ------------------------------------------------------------------ schedule
//
// The tiles of all items (row tile, KV head, sequence: rt fastest) form one
// sequence of units, unit u of CTA c's run [start(c), start(c + 1)), start(c) =
// c base + min(c, rem).  Without a split the items are dealt out the same way.

// A run of tiles of one item.
struct Seg {
  int b, hk, rt;     // sequence, KV head, row tile
  int k0, k1, nk;    // tiles [k0, k1) of the item's nk
  int past;          // keys that every node sees
};

// In shared memory: keys and tiles of each sequence, and where the CTA starts.
struct TreeSched {
  int past[kTreeSeqs];
  int pre[kTreeSeqs + 1];
  int b, item, k;
  int left;          // units (or, without a split, items) of this CTA
  int split;         // whether items are cut
};

// n units over g shares: share c starts at c base + min(c, rem).  Unit counts fit
// 31 bits (the host sees to it): a 64-bit division is a thousand bytes of code and
// some hundred clocks, in a kernel whose short calls are bound by both.
struct Deal {
  unsigned base, rem;
};
__device__ __forceinline__ Deal deal(unsigned n, unsigned g) {
  Deal d;
  d.base = n / g;
  d.rem = n - d.base * g;
  return d;
}
__device__ __forceinline__ unsigned deal_start(const Deal& d, unsigned c) { return c * d.base + min(c, d.rem); }
// The share that holds unit u.
__device__ __forceinline__ int deal_owner(const Deal& d, unsigned u) {
  const unsigned cut = d.rem * (d.base + 1);
  return (int)(u < cut ? u / (d.base + 1) : d.rem + (u - cut) / d.base);
}
// CTAs that take part: as many as have kTreeLeast tiles each.
__device__ __forceinline__ unsigned tree_shares(unsigned units, unsigned grid) {
  return min(grid, max(1u, units / kTreeLeast));
}
// Whether items are cut (TreeWhole), from the longest one's tiles and all tiles.
// The kernel and the join have to agree: every rounding is written out.
__device__ __forceinline__ bool tree_cut(const TreeParams& p, int most, unsigned units) {
  const float u = __fmul_rn(p.share, (float)units);
  const float more = __fadd_rn(p.whole.join, fminf(__fmul_rn(0.5f, u), p.whole.run));
  return __fmul_rn((float)most, (float)p.waves) > __fadd_rn(u, more);
}
// Tiles of a sequence.
__device__ __forceinline__ int tiles_of(const TreeParams& p, int past) {
  return (int)((unsigned)(min(past, p.C - p.N) + p.N + kTile - 1) / kTile);
}

// Filled by one warp; the CTA synchronises before anyone reads.
__device__ __forceinline__ void tree_schedule(const TreeParams& p, TreeSched* s, int lane) {
  int sum = 0, most = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int n = 0;
    if (b < p.B) {
      const int past = min(max(__ldcg(p.past + b), 0), p.C);
      s->past[b] = past;
      n = tiles_of(p, past);
    }
    most = max(most, n);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += up;
    }
    if (b < p.B) s->pre[b + 1] = sum + n;
    sum += __shfl_sync(0xffffffffu, n, 31);
  }
  if (lane == 0) s->pre[0] = 0;
  most = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);
  __syncwarp();
  const unsigned hr = (unsigned)p.Hkv * p.rtiles;
  const bool split = p.split && tree_cut(p, most, hr * sum);
  const unsigned n = split ? hr * sum : hr * p.B;
  const unsigned shares = split ? tree_shares(n, gridDim.x) : gridDim.x;
  const Deal d = deal(n, shares);
  const unsigned c = blockIdx.x;
  const unsigned at = c < shares ? deal_start(d, c) : n, end = c < shares ? deal_start(d, c + 1) : n;
  unsigned b = 0, each = 1, rem = at;
  if (split) {
    // last sequence whose units start at or before `at`
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const bool le = b0 + lane < p.B && hr * s->pre[b0 + lane] <= at;
      b += __popc(__ballot_sync(0xffffffffu, le));
    }
    b = max(b, 1u) - 1;
    each = s->pre[b + 1] - s->pre[b];
    rem = at - hr * s->pre[b];
  }
  unsigned item = rem / each;
  const unsigned k = rem - item * each;
  if (!split) {
    b = item / hr;
    item -= b * hr;
  }
  if (lane == 0) {
    s->b = (int)b;
    s->item = (int)item;
    s->k = (int)k;
    s->left = (int)(end - at);
    s->split = split;
  }
}

// Each role walks the CTA's runs with a copy of this.
struct TreeWalk {
  int b, item, k, left;
};
__device__ __forceinline__ TreeWalk tree_begin(const TreeSched* s) { return TreeWalk{s->b, s->item, s->k, s->left}; }
__device__ __forceinline__ bool tree_next(const TreeParams& p, const TreeSched* s, TreeWalk& w, Seg& g) {
  if (w.left <= 0) return false;
  g.b = w.b;
  g.nk = s->pre[w.b + 1] - s->pre[w.b];
  g.past = s->past[w.b];
  g.hk = p.rtiles == 1 ? w.item : w.item / p.rtiles;
  g.rt = w.item - g.hk * p.rtiles;
  g.k0 = w.k;
  g.k1 = s->split ? min(g.nk, w.k + w.left) : g.nk;
  w.left -= s->split ? g.k1 - g.k0 : 1;
  w.k = 0;   // a run that stops inside an item is the CTA's last
  if (++w.item == p.Hkv * p.rtiles) {
    w.item = 0;
    ++w.b;
  }
  return true;
}

// First tile of an item with keys that some row does not see (at least the
// last one, where unused nodes are dealt with).  At most 3 tiles follow it.
__device__ __forceinline__ int first_masked(const Seg& g) { return min(g.past / kTile, g.nk - 1); }

// ------------------------------------------------------------------ masks

// Ancestor bits of each lane's node (-1: none), itself included, for trees of at
// most 32; 0 and false when it, or one of its ancestors, is not used.  The whole
// warp calls.  The lanes hold the parents: a step up a tree is a shuffle, not a load
// that waits for the last one.
__device__ __forceinline__ bool ancestors32(const int* parents, int n, int node, uint32_t& bits) {
  const int lane = threadIdx.x & 31;
  const int up = lane < n ? __ldcg(parents + lane) : -2;
  bits = 0u;
  bool used = true;
  int a = node;
  while (__any_sync(0xffffffffu, a >= 0)) {   // each parent is lower than its child: at most n steps
    const int next = __shfl_sync(0xffffffffu, up, a & 31);
    if (a >= 0) {
      bits |= 1u << a;
      if (next < -1 || next >= a) used = false;
      a = used ? next : -1;
    }
  }
  if (!used) bits = 0u;
  return used;
}

// The same for trees of up to 256, 32 nodes a word, word i stored at anc[i stride];
// the n parents pass through `up` in shared memory.
__device__ __forceinline__ void ancestors256(const int* parents, int n, int16_t* up, int node, uint32_t* anc,
                                             int stride) {
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < n; i += 32) {
    const int v = __ldcg(parents + i);
    up[i] = (int16_t)(v >= -1 && v < i ? v : -2);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) anc[i * stride] = 0u;
  __syncwarp();
  int a = node;
#pragma unroll 1
  while (a >= 0) {
    anc[(a >> 5) * stride] |= 1u << (a & 31);
    a = up[a];
  }
  if (a == -2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) anc[i * stride] = 0u;
  }
}

// Bits 0..31: which of the keys kq .. kq + 31 a row sees, from its ancestor bits.
template <int WORDS>
__device__ __forceinline__ uint32_t seen32(const uint32_t* anc, int stride, int kq, int past, int C) {
  const int rel = kq - past;
  uint32_t v;
  if (rel <= -32) v = 0xFFFFFFFFu;
  else if (rel < 0) v = ((1u << -rel) - 1u) | (anc[0] << -rel);
  else {
    const int w = rel >> 5, s = rel & 31;
    const uint32_t lo = w < WORDS ? anc[w * stride] : 0u, hi = w + 1 < WORDS ? anc[(w + 1) * stride] : 0u;
    v = __funnelshift_r(lo, hi, s);
  }
  const int n = C - kq;
  if (n < 32) v = n <= 0 ? 0u : v & ((1u << n) - 1u);
  return v;
}

// ------------------------------------------------------------------ non-finite values

// Non-finite halves of an fp16 pair cleared; true if there were any.
__device__ __forceinline__ bool clear_nonfinite(uint32_t& w) {
  const bool lo = (w & 0x7C00u) == 0x7C00u, hi = (w & 0x7C000000u) == 0x7C000000u;
  if (lo) w &= 0xFFFF0000u;
  if (hi) w &= 0x0000FFFFu;
  return lo || hi;
}

// Clear `count` 16-byte chunks of row `row` of an fp16 tile (D / 64 panels of
// [128 keys][128 B], swizzled), from chunk `first`.  True if there were non-finite
// values.  (Only for tiles with masks: kept short, out of the way of the decode.)
static __device__ __noinline__ bool clean_chunks(uint8_t* tile, int row, int first, int count) {
  bool any = false;
#pragma unroll 1
  for (int c = 0; c < count; ++c) {
    const int ch = first + c;
    uint4* at = reinterpret_cast<uint4*>(tile + (ch >> 3) * (kTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
    uint4 v = *at;
    bool bad = clear_nonfinite(v.x);
    bad |= clear_nonfinite(v.y);
    bad |= clear_nonfinite(v.z);
    bad |= clear_nonfinite(v.w);
    if (bad) *at = v;
    any |= bad;
  }
  return any;
}

// Which of the rows kq .. kq + 31 are in use.  Those behind hold anything (in a
// Q8_0 tile what the last one left): nobody sees them, and if they were noted each
// run's end would look for them (14 us against 22 for 8 nodes over 636 keys).
__device__ __forceinline__ uint32_t rows_in_use(const TreeParams& p, const Seg& g, int kq) {
  const int n = min(g.past, p.C - p.N) + p.N - kq;
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Value c of a V row in global memory.
template <int D, bool Q8>
__device__ __forceinline__ float value_at(const TreeParams& p, const Seg& g, int key, int c) {
  if (!in_bounds(key >= 0 && key < p.C && c >= 0 && c < D, p.status, kSiteTreeKV)) return 0.f;
  const uint8_t* row = p.v + (((long long)(p.b0 + g.b) * p.Hkv + g.hk) * p.C + key) * (Q8 ? D / 32 * 34 : 2 * D);
  if constexpr (Q8) {
    const uint8_t* blk = row + 34 * (c >> 5);
    const __half d = __ushort_as_half(*reinterpret_cast<const unsigned short*>(blk));
    return __half2float(__hmul(__int2half_rn((int)(int8_t)blk[2 + (c & 31)]), d));
  } else {
    return __half2float(reinterpret_cast<const __half*>(row)[c]);
  }
}

// ------------------------------------------------------------------ Q8_0 tiles

// Raw tiles are decoded a block at a time, four code bytes of a word to two
// fp16 pairs (bytes 0 and 2, 1 and 3: no byte permutes).  A block of an even
// column starts on a word: its first two codes share a word with the scale and
// its last two with the next block, so these four form word 0; the other 28
// are words 1 to 7 as they lie.  A block of an odd column starts in the middle
// of a word and its codes are words 0 to 7.  So the decoded row holds the
// block's values in this order; Q rows are put in the same order, and the
// columns of O come out in it.
__host__ __device__ constexpr int q8_code_at(int odd, int pos) {
  const int i = pos >> 2, j = pos & 3, byte = j == 1 ? 2 : j == 2 ? 1 : j;
  return odd ? 4 * i + byte : i > 0 ? 4 * i - 2 + byte : byte < 2 ? byte : 28 + byte;
}

// Non-finite values of the V rows kq + i, i in `bits`, added to columns c0 ..
// c0 + 15 (positions of a decoded row).
template <int D, bool Q8>
__device__ __forceinline__ void add_values(const TreeParams& p, const Seg& g, int kq, uint32_t bits, int c0,
                                           float (&x)[16]) {
  while (bits) {
    const int key = kq + __ffs(bits) - 1;
    bits &= bits - 1;
#pragma unroll 1
    for (int c = 0; c < 16; ++c) {
      const int at = c0 + c;
      const float v = value_at<D, Q8>(p, g, key, Q8 ? (at & ~31) + q8_code_at((at >> 5) & 1, at & 31) : at);
      if (!(v - v == 0.f)) x[c] += v;
    }
  }
}

// Columns col .. col + 15 (positions) of a row, to the fp16 output.
template <int D, bool Q8>
__device__ __forceinline__ void store_columns(const float (&x)[16], int col, __half* orow) {
  if constexpr (Q8) {
    // decoded order: positions 4 i, 4 i + 2 and 4 i + 1, 4 i + 3 hold neighbours
    const int odd = (col >> 5) & 1, pos0 = col & 31, at = col & ~31;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int i4 = pos0 + 4 * i;
        const int e = odd ? i4 + 2 * k : i4 > 0 ? i4 - 2 + 2 * k : 30 * k;
        *reinterpret_cast<__half2*>(orow + at + e) = __floats2half2_rn(x[4 * i + k], x[4 * i + k + 2]);
      }
  } else {
    uint32_t h[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const __half2 hh = __floats2half2_rn(x[2 * q], x[2 * q + 1]);
      h[q] = *reinterpret_cast<const uint32_t*>(&hh);
    }
    *reinterpret_cast<uint4*>(orow + col) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(orow + col + 8) = make_uint4(h[4], h[5], h[6], h[7]);
  }
}

// Block BLK of row `row` of a raw tile (rows of D / 32 blocks) as 16 fp16 pairs
// in that order, each value RNE(q d).  Rows of 136 bytes are read as 8-byte
// words (34 words apart: a half-warp's 16 rows cover every bank once), rows of
// 68 bytes as 4-byte words (17 apart).  The block is a template argument: with a
// runtime one the two word orders become selects, half as many instructions again.
template <int D, int BLK>
__device__ __forceinline__ void decode_block(const uint8_t* raw, int row, const DecK& K, uint32_t (&v)[16]) {
  constexpr int RB = D / 32 * 34, kWord = (34 * BLK) & ~3;   // the block's first word
  uint32_t w[9];   // the words that hold the block
  if constexpr (RB % 8 == 0) {
    const uint2* src = reinterpret_cast<const uint2*>(raw + row * RB + (kWord & ~7));
    uint32_t a[10];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const uint2 x = src[i];
      a[2 * i] = x.x;
      a[2 * i + 1] = x.y;
    }
#pragma unroll
    for (int i = 0; i < 9; ++i) w[i] = a[i + ((kWord >> 2) & 1)];
  } else {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(raw + row * RB + kWord);
#pragma unroll
    for (int i = 0; i < 9; ++i) w[i] = src[i];
  }
  const uint32_t d2 = __byte_perm(w[0], 0u, BLK & 1 ? 0x3232 : 0x1010);
  if constexpr (BLK % 2 == 0) w[0] = __byte_perm(w[0], w[8], 0x5432);
#pragma unroll
  for (int i = 0; i < 8; ++i) q8_word(w[i + (BLK & 1)], d2, K, v[2 * i], v[2 * i + 1]);
}

// Block BLK decoded and written to the swizzled fp16 tile (D / 64 panels of
// [128][128 B]).
template <int D, int BLK>
__device__ __forceinline__ void decode_to_tile(uint8_t* dst, const uint8_t* raw, int row, const DecK& K) {
  uint32_t v[16];
  decode_block<D, BLK>(raw, row, K, v);
  uint8_t* base = dst + (BLK >> 1) * (kTile * 128) + row * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(base + (((4 * (BLK & 1) + i) ^ (row & 7)) << 4)) =
        make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// 32 fp16 values of a Q row's block to the order of decode_block.
__device__ __forceinline__ void order_block(const uint4 (&q)[4], int odd, uint4 (&out)[4]) {
  const uint32_t s[16] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w,
                          q[2].x, q[2].y, q[2].z, q[2].w, q[3].x, q[3].y, q[3].z, q[3].w};
  uint32_t o[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int e0 = q8_code_at(0, 2 * k), e1 = q8_code_at(0, 2 * k + 1);
    const int f0 = q8_code_at(1, 2 * k), f1 = q8_code_at(1, 2 * k + 1);
    const uint32_t e = __byte_perm(s[e0 >> 1], s[e1 >> 1], ((e0 & 1) ? 0x32u : 0x10u) | ((e1 & 1) ? 0x7600u : 0x5400u));
    const uint32_t f = __byte_perm(s[f0 >> 1], s[f1 >> 1], ((f0 & 1) ? 0x32u : 0x10u) | ((f1 & 1) ? 0x7600u : 0x5400u));
    o[k] = odd ? f : e;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
}

// A place in a ring of N stages and the parity of its pass.
template <int N>
struct Ring {
  int at = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step() {
    if (++at == N) {
      at = 0;
      ph ^= 1u;
    }
  }
};

// OR of `pred` over the `count` threads of named barrier `id`.  (It has no time
// limit: all of them come to it, whatever failed before.)
__device__ __forceinline__ bool vote_or(uint32_t id, uint32_t count, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)pred)
      : "memory");
  return r != 0;
}

// 1-D bulk copy; addresses and size multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The whole 16-byte units around the rows [j kTile, min(that + kTile, last))
// of a head of the raw cache: first byte and size (the cache is a multiple of
// 16 bytes).
__device__ __forceinline__ void raw_span(long long head, int C, int row_bytes, int j, int last, long long& at,
                                         uint32_t& bytes) {
  const long long a = (head * C + (long long)j * kTile) * row_bytes;
  const long long e = (head * C + min((long long)(j + 1) * kTile, (long long)last)) * row_bytes;
  at = a & ~15ll;
  bytes = (uint32_t)(((e + 15) & ~15ll) - at);
}

// Pieces of the items that were cut.  Row r of item (sequence b, head hk, row
// tile rt), whose tiles went to CTAs c0 .. c1, is
//   sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c.
// A CTA has at most two pieces, of its first run (slot 2 c) and of its last
// (2 c + 1).
struct JoinSpan {
  unsigned c0, c1;
  bool cut;        // else its one CTA wrote the output
  bool at_start;   // the piece of c0 is of its first run
  __device__ __forceinline__ long long slot(unsigned c) const { return 2ll * c + (c > c0 || at_start ? 0 : 1); }
};

// The pieces of the item `sub` of sequence b (all threads of a CTA call).  Reads
// the lengths only, and is called before the wait for the kernel that writes the
// pieces: that kernel lets this one start after its own wait, when the lengths
// are final.
__device__ __forceinline__ JoinSpan join_span(const TreeParams& p, int b, unsigned sub, unsigned grid, int (&sums)[4]) {
  if (threadIdx.x < 32) {   // the sequences' tiles, as tree_schedule counts them
    int before = 0, all = 0, mine = 0, most = 0;
#pragma unroll 1
    for (int i = threadIdx.x; i < p.B; i += 32) {
      const int past = min(max(__ldcg(p.past + i), 0), p.C);
      const int n = tiles_of(p, past);
      all += n;
      most = max(most, n);
      before += i < b ? n : 0;
      mine += i == b ? n : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
      mine += __shfl_xor_sync(0xffffffffu, mine, o);
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    if (threadIdx.x == 0) sums[0] = before, sums[1] = mine, sums[2] = all, sums[3] = most;
  }
  __syncthreads();
  JoinSpan j{0, 0, false, false};
  const unsigned hr = (unsigned)p.Hkv * p.rtiles, nk = sums[1], units = hr * sums[2];
  if (!tree_cut(p, sums[3], units)) return j;   // no item was cut
  const Deal dl = deal(units, tree_shares(units, grid));
  const unsigned u0 = hr * sums[0] + sub * nk;
  j.c0 = deal_owner(dl, u0);
  j.c1 = deal_owner(dl, u0 + nk - 1);
  j.cut = j.c0 != j.c1;
  j.at_start = deal_start(dl, j.c0) == u0;
  return j;
}

// A row's sums over pieces taken one after the other: E columns, relative to the
// largest reference so far.
template <int E>
struct JoinSum {
  float m, l, o[E];
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
  }
  __device__ __forceinline__ void add(float mc, float lc, const float (&x)[E]) {
    const float top = fmaxf(m, mc);
    const float a = m == top ? 1.f : ex2(m - top), f = mc == top ? 1.f : ex2(mc - top);
    m = top;
    l = l * a + lc * f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + x[e] * f;
  }
};

template <typename... KArgs, typename... Args>
cudaError_t launch_tree_kernel(void (*kern)(KArgs...), unsigned grid, unsigned block, int smem, cudaStream_t s,
                               const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Once per kernel and device: its dynamic shared memory.
template <typename Tag, typename Kern>
cudaError_t allow_smem(Kern kern, int bytes) {
  std::atomic<unsigned long long>& configured = attr_flag<Tag>();
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  return cudaSuccess;
}

}  // namespace m4q
