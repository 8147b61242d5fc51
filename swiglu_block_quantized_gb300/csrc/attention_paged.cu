// attention_paged.cu -- attention of one new token of each of B sequences over a paged
// KV cache: O = softmax(scale q K^T) V over the rows j < lengths[b], row j at place
// j % page of page table[b][j / page].
//
// An item is a sequence, a KV head and up to 8 NT of the query heads that share it.  Its
// keys are cut into chunks of 64 (D = 128) or 128 (D = 64); the chunks of all items form
// one sequence, dealt out evenly over persistent CTAs (lengths are read on the device).
// A CTA's four warps take a quarter of each chunk each, with a running maximum, sum and O
// of their own, joined when the CTA's part of the item ends.  Parts of items that are cut
// go to the workspace, and a second kernel joins them in a fixed order.
//
// A warp's step of 16 keys (two at D = 64): S^T = K Q^T with the keys on the MMA's 16
// rows and the query heads on its 8 columns, then O^T += V^T P^T with the head dim on the
// rows (mma.sync m16n8k16: a group of up to 8 heads fills it, and the operands need no
// shared memory).  The MMA's k index may stand for any head dim that Q's fragment agrees
// with, and its rows for any head dim of V, so fragments are made from what a thread can
// read in one piece: 16 bytes of a K row (fp16), a block of codes (Q8_0), 16 bytes of two
// V rows whose values are paired by byte permutes.  P^T comes from S^T by an 8 x 8
// transposition in registers.
//  - fp16: K and V rows go from global memory to registers, the next step's K while this
//    step's V is used and the other way round.
//  - Q8_0: rows are copied as they are to a ring in shared memory (bulk copies of 8 rows,
//    each warp its own), and a thread decodes the codes it needs: 34-byte blocks are read
//    as aligned words, whose first and last codes of a block (where it starts between
//    words) are put together in one word, so that no word is shifted.
// The reference of a row's softmax is raised when a score exceeds it by 2^8 (one vote a
// step); P is fp16, sums are fp32.
#include "codec.cuh"
#include "kv_common.cuh"
#include "launch.h"

namespace m4q {

namespace {

constexpr int kThreads = 128;
constexpr int kStages = 3;        // Q8_0: steps of a warp in its ring
constexpr int kPiece = 2;         // pieces of cut items a CTA may have: its first and its last
constexpr float kLowest = -3.402823466e38f;
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

template <int D, bool Q8, int NT>
struct Cfg {
  static constexpr int RB = Q8 ? D / 32 * 34 : 2 * D;   // bytes of a row
  static constexpr int KS = 128 / D;                    // 16-key MMA rows a step
  static constexpr int KT = 16 * KS;                    // keys of a warp's step
  static constexpr int GR = KT / 8;                     // groups of 8 keys of a step: within a page
  static constexpr int CH = 4 * KT;                     // keys of a chunk
  static constexpr int QS = D / 16;                     // k16 steps of S, and m16 tiles of O
  static constexpr int R = 8 * NT;                      // query rows of an item
  static constexpr int kStage = 2 * KT * RB;            // Q8_0: K rows, then V rows
  static constexpr int kRing = Q8 ? 4 * kStages * kStage : 0;
  static constexpr int kPitch = D + 4;                  // floats of a row of O in shared memory
  static constexpr int kJoin = 4 * R * kPitch * 4 + 4 * R * 8;
  static constexpr int kSmem = kRing + kJoin + (kPagedSeqs + 1) * 8;
};

// Which key of a step's 16 stands on row r of the MMA.  Q8_0: an order in which the reads
// of K (rows r, 4 threads a row) and of V (keys 2t, 2t + 1, 2t + 8, 2t + 9 of a thread)
// meet no bank twice at D = 128; fp16: rows as they are.
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
// 2t + 1 of n; seen: bit 2 k + h says that row g + 8 h of MMA k counts.
template <int D, int NT, int KS>
__device__ __forceinline__ void softmax_step(float (&s)[KS][NT][4], Acc<D, NT>& a, float scale, bool all,
                                             uint32_t seen, uint32_t (&pf)[KS][NT][2]) {
  bool raise = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float& x = s[k][n][2 * h + c];
          x *= scale;
          if (!all && !((seen >> (2 * k + h)) & 1)) x = -INFINITY;
          top = fmaxf(top, x);
        }
      raise |= top > a.m[n][c] + 8.f;
    }
  if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float top = a.m[n][c];
#pragma unroll
        for (int k = 0; k < KS; ++k) top = fmaxf(top, fmaxf(s[k][n][c], s[k][n][2 + c]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
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

// Where the chunks of sequences b0 .. b0 + B - 1 begin, in shared memory: at[0 .. B].
template <int CH>
__device__ __forceinline__ void count_chunks(const PagedParams& p, long long* at, long long (&part)[4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = (p.B + kThreads - 1) / kThreads, first = threadIdx.x * each;
  const long long most = (long long)p.W * p.page;
  long long sum = 0;
  for (int i = first; i < min(first + each, p.B); ++i)
    sum += (min((long long)max(p.lengths[i], 0), most) + CH - 1) / CH;
  long long in = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += y;
  }
  if (lane == 31) part[warp] = in;
  __syncthreads();
  for (int w = 0; w < warp; ++w) in += part[w];
  long long before = in - sum;
  for (int i = first; i < min(first + each, p.B); ++i) {
    at[i] = before;
    before += (min((long long)max(p.lengths[i], 0), most) + CH - 1) / CH;
  }
  if (threadIdx.x == kThreads - 1) at[p.B] = in;
  __syncthreads();
}

// Rows of a warp's groups of 8 keys, 32 groups at a time: lane l holds the pool row of
// group l of the window (-1: not seen), the next window's table entries are on their way.
template <typename C>
struct Rows {
  const int32_t* table;   // the sequence's entries
  int hk, first, last;    // keys [first, last) of the warp's piece; steps CH apart
  int cur;                // rows of this window
  int entry, key;         // next window: the lane's entry and key (last: none)
  static constexpr int kSteps = 32 / C::GR;
  __device__ __forceinline__ void fetch(const PagedParams& p, int step) {
    const int lane = threadIdx.x & 31;
    const long long k = (long long)first + (long long)(step + lane / C::GR) * C::CH + 8 * (lane % C::GR);
    key = (int)min(k, (long long)last);
    entry = key < last ? table[key / p.page] : -1;
  }
  __device__ __forceinline__ void advance(const PagedParams& p, int step) {   // to the window of `step`
    cur = -1;
    if ((unsigned)entry < (unsigned)p.P) {
      cur = (entry * p.Hkv + hk) * p.page + key % p.page;
      if (!in_bounds(cur >= 0 && (long long)cur + 8 <= (long long)p.P * p.Hkv * p.page, p.status, kSitePagedKV)) cur = -1;
    }
    fetch(p, step + kSteps);
  }
  __device__ __forceinline__ int group(int step, int i) const {
    return __shfl_sync(0xffffffffu, cur, step % kSteps * C::GR + i);
  }
};

template <int D, bool Q8, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) paged_kernel(const PagedParams p) {
  using C = Cfg<D, Q8, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long part[4];
  __shared__ __align__(8) uint64_t full[4][kStages];
  __shared__ int abort_flag;
  uint8_t* ring = smem;
  float* so = reinterpret_cast<float*>(smem + C::kRing);              // [4][R][kPitch]
  float2* sml = reinterpret_cast<float2*>(so + 4 * C::R * C::kPitch); // [4][R]
  long long* at = reinterpret_cast<long long*>(smem + C::kRing + C::kJoin);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int cta = blockIdx.x, ctas = gridDim.x;
  if (Q8 && threadIdx.x == 0) {
    for (int w = 0; w < 4; ++w)
      for (int i = 0; i < kStages; ++i) mbar_init(&full[w][i], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  const WaitCtl ctl{&abort_flag, p.status, kWaitNs};
  const DecK dk = make_deck();
  pdl_launch_dependents();
  pdl_wait();
  count_chunks<C::CH>(p, at, part);

  const int per = p.Hkv * p.rtiles;                  // items of a sequence
  const long long total = at[p.B] * per;
  // this CTA's chunks [u, u1) of all (none for those past the chunks' number: every CTA
  // between an item's first and its last has a piece of it), or, not split, its items u, u +
  // ctas, ...
  const int used = (int)min(total, (long long)ctas);
  long long u = p.split ? (cta < used ? total * cta / used : 0) : cta;
  const long long u1 = p.split ? (cta < used ? total * (cta + 1) / used : 0) : (long long)p.B * per;
  if (p.split && threadIdx.x == 0) p.ws_cut[cta] = make_int4(0, 0, 0, 0);
  // rows of sequences without keys
  for (int b = cta; b < p.B; b += ctas)
    if (at[b + 1] == at[b])
      for (int i = threadIdx.x; i < p.H * D / 8; i += kThreads)
        *reinterpret_cast<uint4*>(p.o + (long long)b * p.H * D + 8 * i) = make_uint4(0, 0, 0, 0);

  uint32_t step_no = 0;   // Q8_0: steps this warp has issued to its ring so far, consumed ones below
  bool ok = true;
  while (u < u1) {
    // the item, and its chunks [c0, c1)
    int b, item;
    long long c0, c1, chunks;
    if (p.split) {
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] * per <= u) lo = mid;
        else hi = mid;
      }
      b = lo;
      chunks = at[b + 1] - at[b];
      const long long rel = u - at[b] * per;
      item = (int)(rel / chunks);
      c0 = rel % chunks;
      c1 = min(chunks, c0 + (u1 - u));
      u += c1 - c0;
    } else {
      b = (int)(u / per);
      item = (int)(u % per);
      chunks = at[b + 1] - at[b];
      c0 = 0;
      c1 = chunks;
      u += ctas;
      if (chunks == 0) continue;
    }
    const int hk = item / p.rtiles, row0 = item % p.rtiles * C::R;   // query heads hk G + row0 ...
    const int len = (int)min((long long)max(p.lengths[b], 0), (long long)p.W * p.page);
    Rows<C> rows;
    rows.table = p.table + (long long)b * p.W;
    rows.hk = hk;
    rows.last = (int)min((long long)len, c1 * C::CH);
    rows.first = (int)min(c0 * C::CH + warp * C::KT, (long long)rows.last);
    const int steps = (rows.last - rows.first + C::CH - 1) / C::CH;   // of this warp
    rows.fetch(p, 0);

    // Q fragments: column g is query head row0 + 8 n + g
    uint32_t qf[NT][C::QS][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = row0 + 8 * n + g;
      const bool has = r < p.G && in_bounds(hk * p.G + r < p.H && b < p.B, p.status, kSitePagedO);
      const __half* q = p.q + ((long long)(hk * p.G + (has ? r : 0)) * p.q_rows + b) * D;
      if constexpr (!Q8) {
#pragma unroll
        for (int j = 0; j < C::QS / 2; ++j) {
          const uint4 v = has ? *reinterpret_cast<const uint4*>(q + 8 * (t + 4 * j)) : make_uint4(0, 0, 0, 0);
          qf[n][2 * j][0] = v.x;
          qf[n][2 * j][1] = v.y;
          qf[n][2 * j + 1][0] = v.z;
          qf[n][2 * j + 1][1] = v.w;
        }
      } else {
        // word i of the thread's codes (see k_words): head dims of its codes 0, 2 and 1, 3
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

    Acc<D, NT> acc;
    acc.clear();
    rows.advance(p, 0);
    // Rows g, g + 8 of MMA k that are seen in `step`; all: every key of the step is.
    auto seen_of = [&](int step, bool& all) {
      const int k0 = rows.first + step * C::CH;
      uint32_t there = 0;
#pragma unroll
      for (int i = 0; i < C::GR; ++i) there |= (rows.group(step, i) >= 0 ? 1u : 0u) << i;
      all = there == (1u << C::GR) - 1 && k0 + C::KT <= rows.last;
      uint32_t seen = 0;
#pragma unroll
      for (int k = 0; k < C::KS; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = 16 * k + key_of<Q8>(g + 8 * h);
          seen |= (((there >> (key >> 3)) & 1) && k0 + key < rows.last ? 1u : 0u) << (2 * k + h);
        }
      return seen;
    };
    // which of the thread's V keys (2t, 2t + 1, 2t + 8, 2t + 9 of MMA k) are seen
    auto seen_v = [&](int step, int k, int j, uint32_t there) {
      const int key = 16 * k + key_of<Q8>(2 * t + (j & 1) + 8 * (j >> 1));
      return ((there >> (key >> 3)) & 1) && rows.first + step * C::CH + key < rows.last;
    };
    auto groups_of = [&](int step) {
      uint32_t there = 0;
#pragma unroll
      for (int i = 0; i < C::GR; ++i) there |= (rows.group(step, i) >= 0 ? 1u : 0u) << i;
      return there;
    };

    if constexpr (!Q8) {
      constexpr int KL = C::QS / 2;    // 16-byte pieces of a K row a thread has
      constexpr int VL = D / 64;       // and of a V row
      uint4 kr[C::KS][2][KL], vr[C::KS][4][VL];
      auto load_k = [&](int step) {
#pragma unroll
        for (int k = 0; k < C::KS; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = rows.group(step, 2 * k + h);
            const uint4* src = reinterpret_cast<const uint4*>(p.k + (long long)(r + g) * C::RB) + t;
            if (r >= 0) {
#pragma unroll
              for (int j = 0; j < KL; ++j) kr[k][h][j] = src[4 * j];
            } else {
#pragma unroll
              for (int j = 0; j < KL; ++j) kr[k][h][j] = make_uint4(0, 0, 0, 0);
            }
          }
      };
      auto load_v = [&](int step) {
        const int k0 = rows.first + step * C::CH;
#pragma unroll
        for (int k = 0; k < C::KS; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = rows.group(step, 2 * k + h);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint4* src = reinterpret_cast<const uint4*>(p.v + (long long)(r + 2 * t + e) * C::RB) + g;
              const bool has = r >= 0 && k0 + 16 * k + 8 * h + 2 * t + e < rows.last;
#pragma unroll
              for (int j = 0; j < VL; ++j) vr[k][2 * h + e][j] = has ? src[8 * j] : make_uint4(0, 0, 0, 0);
            }
          }
      };
      if (steps > 0) {
        load_k(0);
        load_v(0);
      }
#pragma unroll 1
      for (int step = 0; step < steps; ++step) {
        bool all;
        const uint32_t seen = seen_of(step, all);
        float s[C::KS][NT][4];
#pragma unroll
        for (int k = 0; k < C::KS; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) s[k][n][0] = s[k][n][1] = s[k][n][2] = s[k][n][3] = 0.f;
#pragma unroll
        for (int j = 0; j < KL; ++j)
#pragma unroll
          for (int k = 0; k < C::KS; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint4 &x = kr[k][0][j], &y = kr[k][1][j];
              mma16816(s[k][n], x.x, y.x, x.y, y.y, qf[n][2 * j][0], qf[n][2 * j][1]);
              mma16816(s[k][n], x.z, y.z, x.w, y.w, qf[n][2 * j + 1][0], qf[n][2 * j + 1][1]);
            }
        const bool more = step + 1 < steps;
        if (more) {
          if ((step + 1) % Rows<C>::kSteps == 0) rows.advance(p, step + 1);
          load_k(step + 1);
        }
        uint32_t pf[C::KS][NT][2];
        softmax_step<D, NT, C::KS>(s, acc, p.scale_log2, all, seen, pf);
#pragma unroll
        for (int k = 0; k < C::KS; ++k)
#pragma unroll
          for (int j = 0; j < VL; ++j) {
            const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&vr[k][0][j]);
            const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&vr[k][1][j]);
            const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&vr[k][2][j]);
            const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&vr[k][3][j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a0 = __byte_perm(w0[i], w1[i], 0x5410), a1 = __byte_perm(w0[i], w1[i], 0x7632);
              const uint32_t a2 = __byte_perm(w2[i], w3[i], 0x5410), a3 = __byte_perm(w2[i], w3[i], 0x7632);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816(acc.o[n][4 * j + i], a0, a1, a2, a3, pf[k][n][0], pf[k][n][1]);
            }
          }
        if (more) load_v(step + 1);
      }
    } else {
      uint8_t* mine = ring + warp * kStages * C::kStage;
      // Copies of a step's rows: K's groups, then V's, a lane each.
      auto issue = [&](int step, uint32_t no) {
        const uint32_t there = groups_of(step);
        uint64_t* bar = &full[warp][no % kStages];
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(there) * 16 * C::RB);
        const int i = lane % C::GR;
        const int r = rows.group(step, i);
        __syncwarp();
        if (lane < 2 * C::GR && r >= 0) {
          uint8_t* dst = mine + (no % kStages) * C::kStage + (lane < C::GR ? 0 : C::KT * C::RB) + 8 * i * C::RB;
          bulk_load(dst, (lane < C::GR ? p.k : p.v) + (long long)r * C::RB, 8 * C::RB, bar);
        }
      };
      // Rows of a step are looked up when it is issued; what is seen of it is kept for its
      // turn: groups that are there, a byte a stage.
      uint32_t kept = 0, issued = step_no;
      auto issue_next = [&](int step, uint32_t no) {
        if (step > 0 && step % Rows<C>::kSteps == 0) rows.advance(p, step);
        const int sh = 8 * (no % kStages);
        kept = (kept & ~(0xFFu << sh)) | (groups_of(step) << sh);
        issue(step, no);
        ++issued;
      };
      const int ahead = min(steps, kStages);
      for (int i = 0; i < ahead; ++i) issue_next(i, step_no + i);
#pragma unroll 1
      for (int step = 0; step < steps && ok; ++step) {
        const uint32_t no = step_no + step, slot = no % kStages;
        ok = mbar_wait(&full[warp][slot], (no / kStages) & 1, ctl);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* kt = mine + slot * C::kStage;
        const uint8_t* vt = kt + C::KT * C::RB;
        const uint32_t there = (kept >> (8 * slot)) & 0xFFu;
        const int k0 = rows.first + step * C::CH;
        const bool all = there == (1u << C::GR) - 1 && k0 + C::KT <= rows.last;
        uint32_t seen = 0;
        if (!all) {
#pragma unroll
          for (int k = 0; k < C::KS; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int key = 16 * k + key_of<Q8>(g + 8 * h);
              seen |= (((there >> (key >> 3)) & 1) && k0 + key < rows.last ? 1u : 0u) << (2 * k + h);
            }
        }
        float s[C::KS][NT][4];
#pragma unroll
        for (int k = 0; k < C::KS; ++k) {
#pragma unroll
          for (int n = 0; n < NT; ++n) s[k][n][0] = s[k][n][1] = s[k][n][2] = s[k][n][3] = 0.f;
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
        uint32_t pf[C::KS][NT][2];
        softmax_step<D, NT, C::KS>(s, acc, p.scale_log2, all, seen, pf);
#pragma unroll
        for (int k = 0; k < C::KS; ++k) {
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
          uint32_t mask01 = 0xFFFFFFFFu, mask23 = 0xFFFFFFFFu;   // values of keys that are not seen become 0
          if (!all) {
            mask01 = (seen_v(step, k, 0, there) ? 0xFFFFu : 0u) | (seen_v(step, k, 1, there) ? 0xFFFF0000u : 0u);
            mask23 = (seen_v(step, k, 2, there) ? 0xFFFFu : 0u) | (seen_v(step, k, 3, there) ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t sel = half ? 0x7632 : 0x5410;
              uint32_t a0, a1, a2, a3;
              q8_word(__byte_perm(w[0][i], w[1][i], sel), d01, dk, a0, a1);
              q8_word(__byte_perm(w[2][i], w[3][i], sel), d23, dk, a2, a3);
              if (!all) {
                a0 &= mask01;
                a1 &= mask01;
                a2 &= mask23;
                a3 &= mask23;
              }
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816(acc.o[n][2 * i + half], a0, a1, a2, a3, pf[k][n][0], pf[k][n][1]);
            }
          }
        }
        __syncwarp();   // the stage has been read
        if (step + kStages < steps) issue_next(step + kStages, no + kStages);
      }
      if (!ok)   // copies still under way land before the block leaves
        for (uint32_t i = 0; i < (uint32_t)kStages && i < issued; ++i) {
          const uint32_t no = issued - 1 - i;
          mbar_wait_drain(&full[warp][no % kStages], (no / kStages) & 1, 100000000ull);
        }
      step_no = issued;
    }

    // The four warps' maxima, sums and O.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = acc.l[n][c];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const int r = warp * C::R + 8 * n + 2 * t + c;
        if (g == 0) sml[r] = make_float2(acc.m[n][c], l);
#pragma unroll
        for (int i = 0; i < C::QS; ++i) {
          int d;   // of the fragment's row g; row g + 8 is d + 1
          if constexpr (!Q8) {
            d = 8 * (g + 8 * (i >> 2)) + 2 * (i & 3);
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
          *reinterpret_cast<float2*>(so + r * C::kPitch + d) = make_float2(acc.o[n][i][c], acc.o[n][i][2 + c]);
        }
      }
    ok = __syncthreads_and(ok);
    if (!ok) break;
    const bool whole = c0 == 0 && c1 == chunks;
    const int piece = kPiece * cta + (c0 == 0 ? 1 : 0);
    for (int i = threadIdx.x; i < C::R * D / 4; i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4, q = row0 + r;
      if (q >= p.G) break;
      float m = kLowest, l = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) m = fmaxf(m, sml[w * C::R + r].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 ml = sml[w * C::R + r];
        const float f = fast_exp2(ml.x - m);
        const float4 x = *reinterpret_cast<const float4*>(so + (w * C::R + r) * C::kPitch + d);
        l += f * ml.y;
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
      }
      if (whole) {
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;   // NaN stays
        if (in_bounds(hk * p.G + q < p.H && b < p.B, p.status, kSitePagedO))
          *reinterpret_cast<uint2*>(p.o + ((long long)b * p.H + hk * p.G + q) * D + d) =
              make_uint2(pack_h2(o.x * inv, o.y * inv), pack_h2(o.z * inv, o.w * inv));
      } else if (in_bounds(piece < kPiece * ctas, p.status, kSitePagedWs)) {
        *reinterpret_cast<float4*>(p.ws_o + ((long long)piece * C::R + r) * D + d) = o;
        if (d == 0) p.ws_ml[piece * C::R + r] = make_float2(m, l);
      }
    }
    if (!whole && c0 == 0 && threadIdx.x == 0) {
      // the CTA of the item's last chunk; this one has its first
      const long long end = at[b] * per + (long long)(item + 1) * chunks - 1;
      const int last = (int)(((end + 1) * used - 1) / total);
      p.ws_cut[cta] = make_int4(b, item, last, 1);
    }
    __syncthreads();
  }
}

// The pieces of an item that was cut: x the CTA that has its first chunk, y the query
// row.  Eight warps take every eighth piece each.
template <int D, int R>
__global__ void __launch_bounds__(256) join_kernel(const PagedParams p) {
  __shared__ float so[8][D];
  __shared__ float sl[8], sm[8];
  constexpr int E = D / 32;
  pdl_wait();
  const int4 cut = p.ws_cut[blockIdx.x];
  if (!cut.w) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y;
  const int hk = cut.y / p.rtiles, q = cut.y % p.rtiles * R + r;
  if (q >= p.G) return;
  const int first = blockIdx.x, n = cut.z - first + 1;
  float m = kLowest, l = 0.f, o[E] = {};
  for (int i = warp; i < n; i += 8) {
    const long long at = (long long)(kPiece * (first + i) + (i == 0 ? 1 : 0)) * R + r;
    const float2 ml = p.ws_ml[at];
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = p.ws_o[at * D + lane + 32 * e];
    const float top = fmaxf(m, ml.x), f = fast_exp2(m - top), h = fast_exp2(ml.x - top);
    m = top;
    l = l * f + ml.y * h;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + x[e] * h;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  if (threadIdx.x >= D) return;
  float top = kLowest, sum = 0.f, x = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) top = fmaxf(top, sm[w]);
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float f = fast_exp2(sm[w] - top);
    sum += f * sl[w];
    x += f * so[w][threadIdx.x];
  }
  const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
  if (in_bounds(hk * p.G + q < p.H && cut.x < p.B, p.status, kSitePagedO))
    p.o[((long long)cut.x * p.H + hk * p.G + q) * D + threadIdx.x] = __float2half_rn(x * inv);
}

template <int D, bool Q8, int NT>
cudaError_t launch(const PagedParams& p, int grid, cudaStream_t s) {
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
  e = launch_proj(kern, (unsigned)grid, (unsigned)kThreads, C::kSmem, s, 1u, p);
  if (e != cudaSuccess || !p.split) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid, (unsigned)(p.G < C::R ? p.G : C::R), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<D, C::R>, p);
}

template <int D, bool Q8>
cudaError_t launch_nt(const PagedParams& p, int grid, cudaStream_t s) {
  return p.G <= 8 ? launch<D, Q8, 1>(p, grid, s) : launch<D, Q8, 2>(p, grid, s);
}

}  // namespace

cudaError_t launch_attention_paged(const PagedParams& p, bool q8, int grid, cudaStream_t s) {
  if (p.D == 64) return q8 ? launch_nt<64, true>(p, grid, s) : launch_nt<64, false>(p, grid, s);
  return q8 ? launch_nt<128, true>(p, grid, s) : launch_nt<128, false>(p, grid, s);
}

}  // namespace m4q
