// attention_paged.cu -- attention of one new token of each of B sequences over a paged
// KV cache: O = softmax(scale q K^T) V over the rows j < lengths[b], row j at place
// j % page of page table[b][j / page].
//
// An item is a sequence, a KV head and up to 8 NT of the query heads that share it.  Its
// keys are cut into chunks of 128 (fp16 at D = 128: 64); the chunks of all items form one
// sequence, dealt out evenly over persistent CTAs (lengths are read on the device).  A CTA's
// four warps take a quarter of each chunk each, with a running maximum, sum and O of their
// own, joined when the CTA's part of the item ends.  Parts of items that are cut go to the
// workspace, and a second kernel joins them in a fixed order.
//
// A warp's step, 16 keys at a time: S^T = K Q^T with the keys on the MMA's 16 rows and the
// query heads on its 8 columns, then O^T += V^T P^T with the head dim on the rows (mma.sync
// m16n8k16: a group of up to 8 heads fills it).  P^T comes from S^T by an 8 x 8
// transposition in registers.  Rows come through a ring in shared memory, each warp's its
// own, in groups of 8 (a group lies within a page):
//  - fp16 by TMA boxes with the 128-byte swizzle, read by ldmatrix;
//  - Q8_0 as they are, by bulk copies.  The MMA's k index may stand for any head dim that
//    Q's fragment agrees with, and its rows for any head dim of V, so a thread decodes what
//    it can read in one piece: a block of a K row, half a block of four V rows, their codes
//    paired by byte permutes.  34-byte blocks are read as aligned words, and where a block
//    starts between words its first and last codes are put together in one, so that no word
//    is shifted.
// P is fp16, as V is (the second product of what that rounding loses would cost Q8_0 pages,
// which are bound by issue slots, another half of their MMAs and packing; without it O is off
// by 2.8e-4 of its size, 2.1e-4 of which is O's own rounding).  So that weights far below the
// largest do not leave fp16's range, the reference of a row's softmax lies 2^7 to 2^15 below
// its largest score (one vote a step says whether it has to be raised): weights down to 2^-21
// of the largest keep all bits, those down to 2^-32 still count.  Sums are fp32, and no more
// than kFoldMmas products go into one: the tensor cores cut off what falls below an fp32
// sum's last bit, always to the same side, which took 0.3% off the mean of two million
// values.  A part that is longer is taken in runs, with a reference and sums of their own,
// joined in fp32 as the warps' sums are.  (Runs cost items of any length the test for their
// end: 65.5 to 66.7 us for 256 short sequences over Q8_0 pages, 36.2 to 36.6 at D = 64, 28.3
// to 29.1 for groups of 16 heads, below 1% elsewhere.  Adding to sums of the warp's own in
// its registers' place took 68.7, 37.5 and 30.2.)
//
// A warp has its ring for itself, and its copies run ahead into the parts of items that
// come next: warps meet only where an item's part ends, to put their O together.  (fp16
// fragments loaded straight from global memory to registers took 106.7 us for one sequence
// of 131,001 keys, D = 128, against 88.8 through the ring; without running ahead 256
// sequences of 50 to 1,000 keys took 150.7 against 121.7.)
//
// Bound by HBM while it streams.  Measured, 8 KV heads of 4 heads: one sequence of 131,001
// keys, D = 128, in 85.2 us over fp16 pages (6.30 TB/s) and 53.5 over Q8_0 (5.33, issue slots
// 55% taken); 32 sequences of 500 to 8,100 in 90.3 and 55.0, at D = 64 in 49.4 and 36.6; 256 of
// 50 to 1,000 in 92.5 and 66.7; 128 of 20,000 to 22,000, groups of 2, in 780 (7.06 TB/s) and
// 440; one of 300 fp16 keys in 6.9.  CTAs of equal shares end 11% apart, as SMs get unequal
// bandwidth.  Groups of more than 8 heads take 16 rows an item and two CTAs an SM: 16 sequences
// of 500 to 8,100 keys, 4 KV heads, groups of 16, in 34.5 us over fp16 and 29.2 over Q8_0 pages
// (D = 64: 21.4 and 21.3), and read their rows again for each 16 heads of a group: groups of 32
// in 43.4 and 44.0.
#include "codec.cuh"
#include "kv_common.cuh"
#include "launch.h"

namespace m4q {

namespace {

constexpr int kThreads = 128;
constexpr int kPiece = 2;         // pieces of cut items a CTA may have: its first and its last
constexpr float kLowest = -3.402823466e38f;
// The reference of a row's softmax, in powers of 2: set kBelow below the largest score, raised
// when a score exceeds it by more than kAbove, so that P (fp16) is at most 2^15.
constexpr float kBelow = 7.f, kAbove = 15.f;
// MMAs of 16 keys that go into one sum before it is added to the sum of those before.
constexpr int kFoldMmas = 128;
constexpr unsigned long long kWaitNs = 2000000000ull;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

template <int D, bool Q8, int NT>
struct Cfg {
  static constexpr int RB = Q8 ? D / 32 * 34 : 2 * D;   // bytes of a row
  static constexpr int KT = paged_chunk(D, Q8) / 4;     // keys of a warp's step
  static constexpr int KS = KT / 16;                    // its 16-key MMA rows
  static constexpr int GR = KT / 8;                     // its groups of 8 keys: within a page
  static constexpr int CH = 4 * KT;                     // keys of a chunk
  static constexpr int QS = D / 16;                     // k16 steps of S, and m16 tiles of O
  static constexpr int R = 8 * NT;                      // query rows of an item
  // Steps of a warp in its ring: what lets three CTAs share an SM (four of Q8_0 at D = 64; two
  // where an item has 16 rows, by their registers).  fp16, two steps and three CTAs against
  // three and two: 104 us against 122 for 256 short sequences, 92 against 95 for 32.
  static constexpr int NS = (Q8 && D == 128) || (!Q8 && NT == 1) ? 2 : 3;
  static constexpr int kHalf = KT * RB;                 // K rows of a step, then V rows
  static constexpr int kRing = 4 * NS * 2 * kHalf;
  static constexpr int kCopies = 2 * GR * (Q8 ? 1 : D / 64);   // copies of a step, a lane each
  // (a warp's O is handed to the others in the stage that it read last)
  static_assert(R * D * 4 <= 2 * kHalf && kCopies <= 32 && GR <= 8 && (GR & (GR - 1)) == 0, "layout");
  static constexpr int kSmem = (Q8 ? 0 : 1024) + kRing + (2 * kPagedSeqs + 1) * 4;
};

// Which key of a step's 16 stands on row r of the MMA.  Q8_0: an order in which the reads
// of K (rows r, 4 threads a row) and of V (keys 2t, 2t + 1, 2t + 8, 2t + 9 of a thread)
// meet no bank twice at D = 128; fp16: as they are (ldmatrix).
template <bool Q8>
__device__ __forceinline__ int key_of(int r) {
  return Q8 ? 8 * ((r >> 2) & 1) + 4 * (r >> 3) + 2 * (r & 1) + ((r >> 1) & 1) : r;
}

// What a warp keeps of its keys so far.
template <int D, int NT>
struct Acc {
  float o[NT][D / 16][4];   // O^T: rows of the head dim, columns 2t, 2t + 1
  float m[NT][2], l[NT][2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
      m[n][0] = m[n][1] = kLowest;
      l[n][0] = l[n][1] = 0.f;
    }
  }
};

// Scores of 16 KS keys -> P^T fragments.  s[k][n]: rows g, g + 8 of MMA k, columns 2t,
// 2t + 1 of n, scaled; -inf for keys that do not count.
template <int D, int NT, int KS>
__device__ __forceinline__ void softmax_step(float (&s)[KS][NT][4], Acc<D, NT>& a, uint32_t (&pf)[KS][NT][2]) {
  bool raise = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) top = fmaxf(top, s[k][n][2 * h + c]);
      raise |= top > a.m[n][c] + kAbove;
    }
  if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float top = s[0][n][c];
#pragma unroll
        for (int k = 0; k < KS; ++k) top = fmaxf(top, fmaxf(s[k][n][c], s[k][n][2 + c]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top - kBelow, a.m[n][c]);
        const float f = fast_exp2(a.m[n][c] - top);
        a.m[n][c] = top;
        a.l[n][c] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          a.o[n][i][c] *= f;
          a.o[n][i][2 + c] *= f;
        }
      }
  }
#pragma unroll
  for (int k = 0; k < KS; ++k)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float e[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        e[c] = fast_exp2(s[k][n][c] - a.m[n][c & 1]);
        a.l[n][c & 1] += e[c];
      }
      pf[k][n][0] = transpose8(pack_h2(e[0], e[1]));
      pf[k][n][1] = transpose8(pack_h2(e[2], e[3]));
    }
}

// What the sequences' items cost and where they begin, at[0 .. B], and their keys, in
// shared memory.  An item costs its chunks and one more: its O is put together by all warps
// at the end, about the time of a chunk.  Returns the longest's cost.
template <int CH>
__device__ __forceinline__ int count_chunks(const PagedParams& p, int* at, int* lens, int2 (&part)[4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = (p.B + kThreads - 1) / kThreads, first = threadIdx.x * each;
  int sum = 0, longest = 0;
  for (int i = first; i < min(first + each, p.B); ++i) {
    const int n = min(max(p.lengths[i], 0), p.W * p.page);
    lens[i] = n;
    at[i] = sum;
    const int cost = n > 0 ? (n - 1) / CH + 2 : 0;   // (n may be INT32_MAX)
    sum += cost;
    longest = max(longest, cost);
  }
  int in = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += y;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) part[warp] = make_int2(in, longest);
  __syncthreads();
  for (int w = 0; w < 4; ++w) {
    if (w < warp) in += part[w].x;
    longest = max(longest, part[w].y);
  }
  for (int i = first; i < min(first + each, p.B); ++i) at[i] += in - sum;
  if (threadIdx.x == kThreads - 1) at[p.B] = in;
  __syncthreads();
  return longest;
}

// Rows of a warp's groups of 8 keys, 32 groups at a time: lane l holds page and place of
// group l of the window (page -1: not seen); the next window's table entries are on their
// way.
template <typename C>
struct Rows {
  const int32_t* table;    // the sequence's entries
  int first, last;         // keys [first, last) of the warp's piece, steps CH apart
  int page_id, place;      // this window
  int entry, next_place;   // the next one
  static constexpr int kSteps = 32 / C::GR;
  __device__ __forceinline__ void fetch(const PagedParams& p, int step) {
    const int lane = threadIdx.x & 31;
    const long long k = (long long)first + (long long)(step + lane / C::GR) * C::CH + 8 * (lane % C::GR);
    entry = -1;
    next_place = 0;
    if (k < last) {
      const int j = (int)k / p.page;
      next_place = (int)k - j * p.page;
      entry = table[j];
    }
  }
  __device__ __forceinline__ void advance(const PagedParams& p, int step) {   // to the window of `step`
    page_id = (unsigned)entry < (unsigned)p.P ? entry : -1;
    place = next_place;
    if (!in_bounds(page_id < p.P && place >= 0 && place + 8 <= p.page, p.status, kSitePagedKV)) page_id = -1;
    fetch(p, step + kSteps);
  }
};

// A part of an item that a CTA takes: chunks [c0, c1) of `chunks`.  u: where the CTA goes
// on, in the cost of all (cut; an item's first unit is the extra one) or as an item (both
// fit 31 bits: 64-bit divisions took most of the 6 us that a call's first copies once
// waited).
struct Part {
  int b, item, c0, c1, chunks;
  int u;
  // The next part before u1 (the first one, from u on, with `at_start`); false: none.
  __device__ __forceinline__ bool next(const PagedParams& p, const int* at, int per, int u1, bool cut, bool at_start) {
    if (u >= u1) return false;
    if (!cut) {
      for (; u < u1; u += gridDim.x) {
        b = u / per;
        item = u - b * per;
        chunks = at[b + 1] - at[b] - 1;
        if (chunks > 0) break;
      }
      if (u >= u1) return false;
      c0 = 0;
      c1 = chunks;
      u += gridDim.x;
      return true;
    }
    if (at_start) {
      int lo = 0, hi = p.B;   // the last sequence that starts at or before u has chunks
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] * per <= u) lo = mid;
        else hi = mid;
      }
      b = lo;
      chunks = at[b + 1] - at[b] - 1;
      const int rel = u - at[b] * per;
      item = rel / (chunks + 1);
      const int r = rel - item * (chunks + 1);
      c0 = max(r - 1, 0);
      c1 = min(chunks, r - 1 + (u1 - u));
      u += c1 + 1 - r;
      return c1 > c0;   // (a run that ends with an item's extra unit)
    }
    // the part before ended its item
    if (++item == per) {
      item = 0;
      do ++b;
      while (at[b + 1] == at[b]);
      chunks = at[b + 1] - at[b] - 1;
    }
    c0 = 0;
    c1 = min(chunks, u1 - u - 1);
    u += c1 + 1;
    return c1 > 0;
  }
  // Keys [first, last) from the warp's first one on; its steps, CH keys apart.
  template <typename C>
  __device__ __forceinline__ int keys(const int* lens, int& first, int& last) const {
    last = (int)min((long long)lens[b], (long long)c1 * C::CH);
    first = (int)min((long long)c0 * C::CH + (threadIdx.x >> 5) * C::KT, (long long)last);
    return last > first ? (last - first - 1) / C::CH + 1 : 0;
  }
};

template <int D, bool Q8, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? (Q8 && D == 64 ? 4 : 3) : 2)
    paged_kernel(const PagedParams p, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<D, Q8, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int2 part[4];
  __shared__ __align__(8) uint64_t full[4][C::NS];
  __shared__ int abort_flag;
  __shared__ float2 sml[4][C::R];   // (max, sum) of the warps' rows
  __shared__ int so_at[4];          // where their O lies in the ring (-1: no keys)
  uint8_t* ring = Q8 ? smem : smem_align<1024>(smem);
  int* at = reinterpret_cast<int*>(ring + C::kRing);   // [B + 1]
  int* lens = at + kPagedSeqs + 1;                     // [B]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (threadIdx.x == 0) {
    for (int w = 0; w < 4; ++w)
      for (int i = 0; i < C::NS; ++i) mbar_init(&full[w][i], 1);
    abort_flag = 0;
    fence_mbar_init();
    if (!Q8) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  const WaitCtl ctl{&abort_flag, p.status, kWaitNs};
  const DecK dk = make_deck();
  pdl_launch_dependents();
  pdl_wait();
  const int longest = count_chunks<C::CH>(p, at, lens, part);

  const int per = p.Hkv * p.rtiles;                  // items of a sequence
  const int total = at[p.B] * per;
  // Dealt out evenly, or item by item where that loses less than the join costs.
  const bool cut = p.split && p.waves * (float)longest > p.share * (float)total + p.join;
  // this CTA's chunks [u, u1) of all (none for those past the chunks' number: every CTA
  // between an item's first and its last has a piece of it), or, not cut, its items u, u +
  // ctas, ...
  const int used = min(total, ctas);
  const int each = cut ? total / used : 0, over = total - each * used;   // the first `over` CTAs have one more
  Part now;
  now.u = cut ? (cta < used ? each * cta + min(cta, over) : 0) : cta;
  const int u1 = cut ? (cta < used ? each * (cta + 1) + min(cta + 1, over) : 0) : p.B * per;
  if (p.split && threadIdx.x == 0) p.ws_cut[cta] = make_int4(0, 0, 0, 0);
  // rows of sequences without keys
  for (int b = cta; b < p.B; b += ctas)
    if (at[b + 1] == at[b])
      for (int i = threadIdx.x; i < p.H * D / 8; i += kThreads)
        *reinterpret_cast<uint4*>(p.o + (long long)b * p.H * D + 8 * i) = make_uint4(0, 0, 0, 0);

  // Copies of a warp's steps run ahead of their use by the stages of its ring, into the
  // parts that come next as well.
  uint8_t* mine = ring + warp * C::NS * 2 * C::kHalf;
  int put = 0, get = 0;             // stages to fill and to read next
  uint32_t phase = 0;               // of the stage to read next
  uint32_t kept = 0;                // groups that are there, a byte a stage
  Part ahead = now;
  Rows<C> rows;
  int in_hk = 0, in_step = 0, in_steps = 0;
  bool in_more = ahead.next(p, at, per, u1, cut, true);
  now = ahead;
  auto open = [&]() {   // the next part with keys for this warp
    while (in_more) {
      in_steps = ahead.template keys<C>(lens, rows.first, rows.last);
      in_step = 0;
      if (in_steps > 0) {
        in_hk = ahead.item / p.rtiles;
        rows.table = p.table + (long long)ahead.b * p.W;
        rows.fetch(p, 0);
        return;
      }
      in_more = ahead.next(p, at, per, u1, cut, false);
    }
  };
  // A step's copies: its groups of K, then of V (fp16: of each half of the head dim).
  auto issue = [&]() {
    if (!in_more) return;
    const int in = in_step % Rows<C>::kSteps;
    if (in == 0) rows.advance(p, in_step);
    const int i = lane % C::GR;
    const int id = __shfl_sync(0xffffffffu, rows.page_id, in * C::GR + i);
    const int place = __shfl_sync(0xffffffffu, rows.place, in * C::GR + i);
    const uint32_t there = __ballot_sync(0xffffffffu, id >= 0) & ((1u << C::GR) - 1);
    kept = (kept & ~(0xFFu << (8 * put))) | (there << (8 * put));
    uint64_t* bar = &full[warp][put];
    uint8_t* dst = mine + put * 2 * C::kHalf;
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(there) * 16 * C::RB);
    __syncwarp();
    if (lane < C::kCopies && id >= 0) {
      const int part_no = lane / C::GR;
      if constexpr (Q8) {
        const long long row = ((long long)id * p.Hkv + in_hk) * p.page + place;
        bulk_load(dst + part_no * C::kHalf + i * 8 * C::RB, (part_no ? p.v : p.k) + row * C::RB, 8 * C::RB, bar);
      } else {
        const int is_v = part_no / (D / 64), half = part_no % (D / 64);
        tma_load_3d(dst + is_v * C::kHalf + half * C::KT * 128 + i * 1024, is_v ? &tm_v : &tm_k, bar, 64 * half, place,
                    id * p.Hkv + in_hk);
      }
    }
    put = put + 1 == C::NS ? 0 : put + 1;
    if (++in_step == in_steps) {
      in_more = ahead.next(p, at, per, u1, cut, false);
      open();
    }
  };
  bool more = in_more, ok = true;
  open();
  for (int i = 0; i < C::NS; ++i) issue();

  uint32_t qf[NT][C::QS][2];
  auto load_q = [&](int b, int hk, int row0) {
    // Q fragments: column g is query head row0 + 8 n + g
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = row0 + 8 * n + g;
      const bool has = r < p.G && in_bounds(hk * p.G + r < p.H && b < p.B, p.status, kSitePagedO);
      const __half* q = p.q + ((long long)(hk * p.G + (has ? r : 0)) * p.q_rows + b) * D;
      if constexpr (!Q8) {
#pragma unroll
        for (int i = 0; i < C::QS; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            qf[n][i][h] = has ? *reinterpret_cast<const uint32_t*>(q + 16 * i + 8 * h + 2 * t) : 0u;
      } else {
        // word i of the thread's codes (as they are read below): head dims of codes 0, 2 and 1, 3
#pragma unroll
        for (int i = 0; i < C::QS; ++i) {
          int d0, d2;   // of code 0 (code 1 next to it), of code 2
          if constexpr (D == 128) {
            const int sh = 2 + 2 * t;
            d0 = i < 6 ? 4 * (i + 2) - sh : i == 6 ? (t < 2 ? 4 - sh : 32 - sh) : (t & 1) ? 28 : 0;
            d2 = i == 7 && !(t & 1) ? 30 : d0 + 2;
            d0 += 32 * t;
            d2 += 32 * t;
          } else {
            const int sh = t < 2 ? 2 : 4;
            d0 = i < 3 ? 4 * (i + 1) - sh : t < 2 ? 0 : 12;
            d2 = i == 3 && t < 2 ? 14 : d0 + 2;
            d0 += 16 * t;
            d2 += 16 * t;
          }
          const uint32_t x = has ? *reinterpret_cast<const uint32_t*>(q + d0) : 0u;
          const uint32_t y = has ? *reinterpret_cast<const uint32_t*>(q + d2) : 0u;
          qf[n][i][0] = __byte_perm(x, y, 0x5410);
          qf[n][i][1] = __byte_perm(x, y, 0x7632);
        }
      }
    }
  };
  if (more) load_q(now.b, now.item / p.rtiles, now.item % p.rtiles * C::R);

  Acc<D, NT> acc;
  // A part is taken kFold steps at a time: where a run of them ends the warps' sums are put
  // together, and with what this thread has of the runs before (volatile: in local memory, for
  // long parts only).
  constexpr int kFold = kFoldMmas / C::KS;
  volatile float before[C::R * D / 4 / kThreads][6];   // o[4], m, l
  int from = 0;
  while (more) {
    const int hk = now.item / p.rtiles, row0 = now.item % p.rtiles * C::R;   // query heads hk G + row0 ...
    int first, last;
    const int steps = now.template keys<C>(lens, first, last), stop = min(steps, from + kFold);
    acc.clear();
    int slot = 0;
#pragma unroll 1
    for (int step = from; step < stop; ++step) {
      ok = __all_sync(0xffffffffu, mbar_wait(&full[warp][get], phase, ctl));
      if (!ok) break;
      const uint8_t* kt = mine + get * 2 * C::kHalf;
      const uint8_t* vt = kt + C::kHalf;
      const uint32_t there = (kept >> (8 * get)) & 0xFFu;
      const int left = last - (first + step * C::CH);   // keys from the step's first on
      const bool all = there == (1u << C::GR) - 1 && left >= C::KT;
      float s[C::KS][NT][4];
#pragma unroll
      for (int k = 0; k < C::KS; ++k) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[k][n][0] = s[k][n][1] = s[k][n][2] = s[k][n][3] = 0.f;
        if constexpr (!Q8) {
          // lanes 0-7: pieces 2 i of the first 8 rows, 8-15 of the other 8, 16-31 the pieces next to
          // them; pieces lie swizzled by their row, each half of the head dim apart
          const uint32_t row = 16 * k + (lane & 15), src = smem_u32(kt) + row * 128;
#pragma unroll
          for (int i = 0; i < C::QS; ++i) {
            uint32_t a[4];
            ldsm_x4(a, src + (i >> 2) * C::KT * 128 + 16 * ((2 * (i & 3) + (lane >> 4)) ^ (row & 7)));
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(s[k][n], a[0], a[1], a[2], a[3], qf[n][i][0], qf[n][i][1]);
          }
        } else {
          // the codes of rows g, g + 8 that the thread has of each, and their scale
          uint32_t w[2][C::QS], d2[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* row = kt + (16 * k + key_of<Q8>(g + 8 * h)) * C::RB;
            if constexpr (D == 128) {
              // block t starts 2 t bytes into the 40 bytes read
              uint32_t x[10];
              const uint2* src = reinterpret_cast<const uint2*>(row + 32 * t);
#pragma unroll
              for (int i = 0; i < 5; ++i) {
                const uint2 y = src[i];
                x[2 * i] = y.x;
                x[2 * i + 1] = y.y;
              }
              const uint32_t lo = t < 2 ? x[0] : x[1], hi = t < 2 ? x[8] : x[9];
#pragma unroll
              for (int i = 0; i < 6; ++i) w[h][i] = x[i + 2];
              w[h][6] = t < 2 ? x[1] : x[8];
              w[h][7] = __byte_perm(lo, hi, (t & 1) ? 0x7654 : 0x5432);
              d2[h] = __byte_perm(lo, 0u, (t & 1) ? 0x3232 : 0x1010);
            } else {
              const uint32_t* src = reinterpret_cast<const uint32_t*>(row + 16 * t);
              const uint32_t lo = src[0];
#pragma unroll
              for (int i = 0; i < 3; ++i) w[h][i] = src[i + 1];
              w[h][3] = __byte_perm(lo, src[4], t < 2 ? 0x5432 : 0x7654);
              d2[h] = dup_scale(*reinterpret_cast<const unsigned short*>(row + 34 * (t >> 1)));
            }
          }
#pragma unroll
          for (int i = 0; i < C::QS; ++i) {
            uint32_t a0, a1, a2, a3;
            q8_word(w[0][i], d2[0], dk, a0, a2);
            q8_word(w[1][i], d2[1], dk, a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(s[k][n], a0, a1, a2, a3, qf[n][i][0], qf[n][i][1]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < C::KS; ++k)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[k][n][c] *= p.scale_log2;
      if (!all) {
        // keys that are not seen: no score, and V's rows become 0 (the product would make
        // NaN of infinities with a weight of 0)
#pragma unroll
        for (int k = 0; k < C::KS; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = 16 * k + key_of<Q8>(g + 8 * h);
            if (!((there >> (key >> 3)) & 1) || key >= left)
#pragma unroll
              for (int n = 0; n < NT; ++n) s[k][n][2 * h] = s[k][n][2 * h + 1] = -INFINITY;
          }
        for (int key = 0; key < C::KT; ++key) {
          if (((there >> (key >> 3)) & 1) && key < left) continue;
          if constexpr (Q8) {
            if (lane < D / 32) *reinterpret_cast<uint16_t*>(const_cast<uint8_t*>(vt) + key * C::RB + 34 * lane) = 0;
          } else if (lane < D / 8) {
            uint8_t* row = const_cast<uint8_t*>(vt) + (lane >> 3) * C::KT * 128 + key * 128;
            *reinterpret_cast<uint4*>(row + 16 * (lane & 7)) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();   // before the copies that fill the stage next
        __syncwarp();
      }
      uint32_t pf[C::KS][NT][2];
      softmax_step<D, NT, C::KS>(s, acc, pf);
#pragma unroll
      for (int k = 0; k < C::KS; ++k) {
        auto product = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816(acc.o[n][i], a0, a1, a2, a3, pf[k][n][0], pf[k][n][1]);
        };
        if constexpr (!Q8) {
          // lanes 0-7: piece 2 i of the first 8 rows, 8-15 the piece next to it, 16-31 of the other
          // 8 rows; transposed, so that head dims are the MMA's rows
          const uint32_t row = 16 * k + (lane & 7) + 8 * (lane >> 4), src = smem_u32(vt) + row * 128;
#pragma unroll
          for (int i = 0; i < C::QS; ++i) {
            uint32_t a[4];
            ldsm_x4_t(a, src + (i >> 2) * C::KT * 128 + 16 * ((2 * (i & 3) + ((lane >> 3) & 1)) ^ (row & 7)));
            product(i, a[0], a[1], a[2], a[3]);
          }
        } else {
          // codes of the four V rows, D / 8 neighbours a thread, and their scales
          uint32_t w[4][D / 32], ds[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint8_t* row = vt + (16 * k + key_of<Q8>(2 * t + (j & 1) + 8 * (j >> 1))) * C::RB;
            if constexpr (D == 128) {
              // half a block, 2 + 2 (g / 2) bytes into the 24 bytes read
              uint32_t x[6];
              const uint2* src = reinterpret_cast<const uint2*>(row + 16 * g);
#pragma unroll
              for (int i = 0; i < 3; ++i) {
                const uint2 y = src[i];
                x[2 * i] = y.x;
                x[2 * i + 1] = y.y;
              }
              const bool far = g >= 4;
              w[j][0] = x[2];
              w[j][1] = x[3];
              w[j][2] = far ? x[4] : x[1];
              w[j][3] = __byte_perm(far ? x[1] : x[0], far ? x[5] : x[4], (g & 2) ? 0x7654 : 0x5432);
              ds[j] = *reinterpret_cast<const unsigned short*>(row + 34 * (g >> 1));
            } else {
              const uint32_t* src = reinterpret_cast<const uint32_t*>(row + 8 * g);
              w[j][0] = src[1];
              w[j][1] = __byte_perm(src[0], src[2], g < 4 ? 0x5432 : 0x7654);
              ds[j] = *reinterpret_cast<const unsigned short*>(row + 34 * (g >> 2));
            }
          }
          const uint32_t d01 = __byte_perm(ds[0], ds[1], 0x5410), d23 = __byte_perm(ds[2], ds[3], 0x5410);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t sel = half ? 0x7632 : 0x5410;
              uint32_t a0, a1, a2, a3;
              q8_word(__byte_perm(w[0][i], w[1][i], sel), d01, dk, a0, a1);
              q8_word(__byte_perm(w[2][i], w[3][i], sel), d23, dk, a2, a3);
              product(2 * i + half, a0, a1, a2, a3);
            }
          }
        }
      }
      __syncwarp();   // the stage has been read
      slot = get;
      get = get + 1 == C::NS ? 0 : get + 1;
      phase ^= get == 0;
      if (step + 1 < stop) issue();   // (the last stage first takes O)
    }
    // The four warps' maxima, sums and O (each row's head dims in an order of its own, by
    // bits 1 and 2 of the row, so that the threads of a quad write to different banks).
    const bool some = stop > from;
    if (lane == 0) so_at[warp] = some ? (int)(mine - ring) + slot * 2 * C::kHalf : -1;
    if (some) {
      float* so = reinterpret_cast<float*>(mine + slot * 2 * C::kHalf);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float l = acc.l[n][c];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
          const int r = 8 * n + 2 * t + c;
          if (g == 0) sml[warp][r] = make_float2(acc.m[n][c], l);
#pragma unroll
          for (int i = 0; i < C::QS; ++i) {
            int d;   // of the fragment's row g; row g + 8 is d + 1 (fp16: d + 8)
            if constexpr (!Q8) {
              d = 16 * i + g;
            } else if constexpr (D == 128) {
              const int sh = 2 + 2 * (g >> 1), w = i >> 1, half = i & 1;
              if (w < 2) d = 4 * (w + 2) - sh + 2 * half;
              else if (w == 2) d = (g < 4 ? 4 : 16) - sh + 2 * half;
              else d = (g & 2) ? 12 + 2 * half : 14 * half;
              d += 16 * g;
            } else {
              const int w = i >> 1, half = i & 1;
              if (w == 0) d = (g < 4 ? 2 : 0) + 2 * half;
              else d = g < 4 ? 6 * half : 4 + 2 * half;
              d += 8 * g;
            }
            if constexpr (Q8) {
              *reinterpret_cast<float2*>(so + r * D + (d ^ (8 * t))) = make_float2(acc.o[n][i][c], acc.o[n][i][2 + c]);
            } else {
              so[r * D + (d ^ (8 * t))] = acc.o[n][i][c];
              so[r * D + ((d + 8) ^ (8 * t))] = acc.o[n][i][2 + c];
            }
          }
        }
    }
    // the next part, its queries on their way
    const Part was = now;
    const bool again = from > 0, end = was.c1 - was.c0 <= from + kFold;   // (a chunk is a step of each warp)
    from = end ? 0 : from + kFold;
    if (end) {
      more = now.next(p, at, per, u1, cut, false);
      if (more) load_q(now.b, now.item / p.rtiles, now.item % p.rtiles * C::R);
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;
    const bool whole = was.c0 == 0 && was.c1 == was.chunks;
    const int piece = kPiece * cta + (was.c0 == 0 ? 1 : 0);
    for (int i = threadIdx.x; i < C::R * D / 4; i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4, q = row0 + r;
      if (q >= p.G) break;
      float m = kLowest, l = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (so_at[w] >= 0) m = fmaxf(m, sml[w][r].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (so_at[w] < 0) continue;
        const float2 ml = sml[w][r];
        const float f = fast_exp2(ml.x - m);
        const float4 x = *reinterpret_cast<const float4*>(ring + so_at[w] + 4 * (r * D + (d ^ (8 * ((r >> 1) & 3)))));
        l += f * ml.y;
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
      }
      if (again || !end) {
        volatile float* b = before[i / kThreads];
        if (again) {
          const float top = fmaxf(m, b[4]), f = fast_exp2(b[4] - top), h = fast_exp2(m - top);
          o = make_float4(o.x * h + b[0] * f, o.y * h + b[1] * f, o.z * h + b[2] * f, o.w * h + b[3] * f);
          l = l * h + b[5] * f;
          m = top;
        }
        b[0] = o.x, b[1] = o.y, b[2] = o.z, b[3] = o.w, b[4] = m, b[5] = l;
        if (!end) continue;
      }
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;   // NaN stays
        if (in_bounds(hk * p.G + q < p.H && was.b < p.B, p.status, kSitePagedO))
          *reinterpret_cast<uint2*>(p.o + ((long long)was.b * p.H + hk * p.G + q) * D + d) =
              make_uint2(pack_h2(o.x * inv, o.y * inv), pack_h2(o.z * inv, o.w * inv));
      } else if (in_bounds(piece < kPiece * ctas, p.status, kSitePagedWs)) {
        *reinterpret_cast<float4*>(p.ws_o + ((long long)piece * C::R + r) * D + d) = o;
        if (d == 0) p.ws_ml[piece * C::R + r] = make_float2(m, l);
      }
    }
    if (end && !whole && was.c0 == 0 && threadIdx.x == 0) {
      // the CTA of the item's last chunk; this one has its first
      const int end = at[was.b] * per + (was.item + 1) * (was.chunks + 1) - 1;
      const int last_cta = end < over * (each + 1) ? end / (each + 1) : over + (end - over * (each + 1)) / each;
      p.ws_cut[cta] = make_int4(was.b, was.item, last_cta, 1);
    }
    fence_proxy_async_smem();   // the stage's next copies come after these reads and writes
    __syncthreads();
    if (some) issue();
  }
  // given up: copies still under way land before the block leaves
  for (int i = 0; !ok && i < C::NS; ++i) {
    mbar_wait_drain(&full[warp][get], phase, 100000000ull);
    get = get + 1 == C::NS ? 0 : get + 1;
    phase ^= get == 0;
  }
}

// The pieces of an item that was cut: x the CTA that has its first chunk, y the query rows,
// `slices` warps a row, which take every slices-th piece each.
template <int D, int R>
__global__ void __launch_bounds__(256) join_kernel(const PagedParams p, int slices) {
  __shared__ float so[8][D];
  __shared__ float2 sml[8];
  constexpr int E = D / 32;
  // No early launch_dependents: a kernel of persistent CTAs that started beside these would
  // find its places on the SMs taken unevenly (86.6 us against 61 for 32 sequences over
  // Q8_0 pages).
  pdl_wait();
  const int4 cut = p.ws_cut[blockIdx.x];
  if (!cut.w) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.y * (8 / slices) + warp / slices;
  const int hk = cut.y / p.rtiles, q = cut.y % p.rtiles * R + r;
  const int first = blockIdx.x, n = r < R && q < p.G ? cut.z - first + 1 : 0;
  float m = kLowest, l = 0.f, o[E] = {};
  for (int i0 = warp % slices; i0 < n; i0 += 4 * slices) {   // four pieces on their way at once
    float2 ml[4];
    float x[4][E];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * slices;
      const long long at = (long long)(kPiece * (first + i) + (i == 0 ? 1 : 0)) * R + r;
      ml[j] = i < n ? p.ws_ml[at] : make_float2(kLowest, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) x[j][e] = i < n ? p.ws_o[at * D + lane + 32 * e] : 0.f;
    }
    const float top = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), m), f = fast_exp2(m - top);
    m = top;
    l *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float h = fast_exp2(ml[j].x - top);
      l += ml[j].y * h;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += x[j][e] * h;
    }
  }
  if (slices > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp % slices) return;
    for (int w = warp + 1; w < warp + slices; ++w) {
      const float2 ml = sml[w];
      const float top = fmaxf(m, ml.x), f = fast_exp2(m - top), h = fast_exp2(ml.x - top);
      m = top;
      l = l * f + ml.y * h;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + so[w][lane + 32 * e] * h;
    }
  }
  if (n == 0) return;
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  if (!in_bounds(hk * p.G + q < p.H && cut.x < p.B, p.status, kSitePagedO)) return;
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.o[((long long)cut.x * p.H + hk * p.G + q) * D + lane + 32 * e] = __float2half_rn(o[e] * inv);
}

template <int D, bool Q8, int NT>
cudaError_t launch(const PagedParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int grid, cudaStream_t s) {
  using C = Cfg<D, Q8, NT>;
  auto kern = paged_kernel<D, Q8, NT>;
  std::atomic<unsigned long long>& configured = attr_flag<std::integer_sequence<int, 11, D, Q8, NT>>();
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit);
  }
  e = launch_proj(kern, (unsigned)grid, (unsigned)kThreads, C::kSmem, s, 1u, p, tm_k, tm_v);
  if (e != cudaSuccess || !p.split) return e;
  // Pieces of an item: few in a batch (a warp a row takes them all), many of a long sequence.
  // Measured, us of the whole call with 1, 4 and 8 warps a row, by `pieces`, 8 KV heads of 4,
  // 8,000 keys a sequence, D = 128, fp16 (Q8_0: the same differences within 0.3),
  //   59: 16.5, 12.2, 11.7   30: 19.6, 17.6, 17.6   21: 24.4, 22.9, 22.8   16: 28.9, 27.8, 28.0
  //   11: 38.0, 37.5, 38.1    9: 46.6, 46.3, 46.9    6: 65.5, 65.8, 66.2    4: 122.0, 122.8, 123.9
  // so the sides are within 0.4 of each other near the bounds.  For items of 16 rows 4 warps
  // would be the better choice at 40 and 14 pieces, too (by 0.6 and 1.4); the rule is one.
  const int items = p.B * p.Hkv * p.rtiles, pieces = grid / items + 2;
  const int slices = pieces <= 4 ? 1 : pieces <= 12 ? 4 : 8;
  const int rows = p.G < C::R ? p.G : C::R, each = 8 / slices;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid, (unsigned)((rows + each - 1) / each), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<D, C::R>, p, slices);
}

template <int D, bool Q8>
cudaError_t launch_nt(const PagedParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int grid,
                      cudaStream_t s) {
  return p.G <= 8 ? launch<D, Q8, 1>(p, tm_k, tm_v, grid, s) : launch<D, Q8, 2>(p, tm_k, tm_v, grid, s);
}

}  // namespace

cudaError_t launch_attention_paged(const PagedParams& p, bool q8, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                   int grid, cudaStream_t s) {
  if (p.D == 64) return q8 ? launch_nt<64, true>(p, tm_k, tm_v, grid, s) : launch_nt<64, false>(p, tm_k, tm_v, grid, s);
  return q8 ? launch_nt<128, true>(p, tm_k, tm_v, grid, s) : launch_nt<128, false>(p, tm_k, tm_v, grid, s);
}

}  // namespace m4q
