// attention_few.cu -- m4q_attention_tree for items of few rows (nodes times
// query heads of a group at most 32): single new tokens and small trees.
//
// With few rows the 128 lanes of a tcgen05 tile are best given to the keys:
//   S^T = K Q^T       M = 128 keys, N = 16 or 32 rows: lane = key
//   O^T += V^T P^T    M = D (two copies of 64 when D = 64), N = rows: lane = d
// so that the softmax of a tile is 16 or 32 values a thread whatever the mask,
// and the MMAs shrink with N.  K is the A operand as it lies ([key][D],
// K-major), V is the A operand as it lies ([key][D], M-major), Q and P are the
// small B operands in shared memory.  What is left is the stream of the cache:
// HBM should bound the fp16 kernel, and for Q8_0 the decode (about 2.4
// instructions a value, 640 issue slots of a scheduler for a tile of 128 keys at
// D = 128, against 1500 clocks of HBM time).
//
// A row's reference maximum is kept while its scores stay within 2^8 of it, so
// the usual tile needs no maximum across the keys: each thread forms its
// exponents against the reference and the four warps vote (one barrier) whether
// one is above 8.  If so (always in a run's first tile) they find the column
// maxima, raise the references and rescale O^T and the sums.  Row sums stay in
// the threads (one partial sum a key lane and row) until the run ends.
//
// Warps: 0 issues the S MMAs (four TMEM buffers ahead), 1 the P V MMAs, 2 and 3
// the copies, 4-7 are the softmax (lane = key), the others prepare (Q, the Q8_0
// decode, the clearing of non-finite V), as in attention_tree.cu, whose notes
// on masks, schedule and pieces hold here.
#include <algorithm>

#include "tree_common.cuh"

namespace m4q {

namespace {

template <int D, bool Q8, int NC>
struct FewCfg {
  static constexpr int N = 16 * NC;                    // rows (columns of S^T)
  static constexpr int kRow = Q8 ? D / 32 * 34 : 2 * D;
  static constexpr int kTileBytes = kTile * D * 2;     // an fp16 tile: D / 64 panels of [128][128 B]
  static constexpr int kQBytes = N * D * 2;            // D / 64 panels of [N][128 B]
  static constexpr int kPBytes = N * kTile * 2;        // two panels (64 keys) of [N][128 B]
  static constexpr int kKS = Q8 ? 2 : D == 128 ? 3 : 6;
  static constexpr int kVS = Q8 ? 2 : D == 128 ? 3 : 6;
  static constexpr int kRaw = kTile * kRow + 32;       // a raw tile, its 16-byte shift, and the decode's overread
  static constexpr int kRS = Q8 ? (D == 128 ? 4 : 12) : 0;
  static constexpr int kPrep = Q8 ? 16 : 4;            // preparing warps
  static constexpr int kPerMatrix = Q8 && D == 64 ? 8 : kPrep;   // of them, those that decode one K or V tile
  static constexpr int kThreads = 32 * (8 + kPrep);
  static constexpr int kBars = 2 * kKS + 4 * kVS + 2 * kRS + 8 + 4 + 6;
  static constexpr int kFixed = (int)sizeof(TreeSched) + 2 * kPrep * 16 + 4 * 32 * 4 + 4 * N * 4 + 5 * N * 4 +
                                kBars * 8 + 64;
  static constexpr int kSmem = 1024 + kQBytes + 2 * kPBytes + (kKS + kVS) * kTileBytes + kRS * kRaw + kFixed;
  static constexpr uint32_t kOCol = 4 * N;             // S^T buffers at N i, then O^T
  static constexpr uint32_t kCols = NC == 1 ? 128 : 256;
  static_assert(5 * N <= (int)kCols, "TMEM budget");
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kRaw % 16 == 0 && kQBytes % 1024 == 0 && kPBytes % 1024 == 0, "alignment");
};

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

template <int D, bool Q8, int NC>
__global__ void __launch_bounds__(FewCfg<D, Q8, NC>::kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const TreeParams p) {
  using Cfg = FewCfg<D, Q8, NC>;
  constexpr int N = Cfg::N, KS = Cfg::kKS, VS = Cfg::kVS, RS = Cfg::kRS > 0 ? Cfg::kRS : 1;
  constexpr int PW = Cfg::kPrep, PM = Cfg::kPerMatrix;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = smem_align<1024>(smem_raw);
  uint8_t* ps = qs + Cfg::kQBytes;                     // [2] P^T
  uint8_t* kst = ps + 2 * Cfg::kPBytes;
  uint8_t* vst = kst + KS * Cfg::kTileBytes;
  uint8_t* raws = vst + VS * Cfg::kTileBytes;
  uint32_t* noted = reinterpret_cast<uint32_t*>(raws + Cfg::kRS * Cfg::kRaw);   // [parity][PW][4]
  uint32_t* anc_all = noted + 2 * PW * 4;              // [warp][32] ancestor bits of a row
  float* wmax = reinterpret_cast<float*>(anc_all + 4 * 32);   // [warp][N] column maxima, or sums
  float* mref = wmax + 4 * N;                          // [N] references
  float* fac = mref + N;                               // [N] rescale factors
  float* linv = fac + N;                               // [N] output factors
  int* unused_all = reinterpret_cast<int*>(linv + N);  // [parity][N] row of an unused node
  TreeSched* sched = reinterpret_cast<TreeSched*>(unused_all + 2 * N);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sched) + (sizeof(TreeSched) + 7) / 8 * 8);
  uint64_t* k_empty = k_full + KS;     // [KS] S^T done with it
  uint64_t* v_full = k_empty + KS;     // [VS] V of a tile in its stage
  uint64_t* v_raw = v_full + VS;       // [VS] (fp16) V of a masked tile, not yet cleared
  uint64_t* v_clean = v_raw + VS;      // [VS] (fp16) V of a masked tile, cleared
  uint64_t* v_empty = v_clean + VS;    // [VS] P V done with it
  uint64_t* r_full = v_empty + VS;     // [RS] raw tile landed
  uint64_t* r_empty = r_full + Cfg::kRS;
  uint64_t* s_full = r_empty + Cfg::kRS;   // [4] S^T of a tile in TMEM
  uint64_t* s_free = s_full + 4;       // [4] read
  uint64_t* p_full = s_free + 4;       // [2] P^T written
  uint64_t* p_free = p_full + 2;       // [2] P V done
  uint64_t* q_full = p_free + 2;       // Q of a run written
  uint64_t* q_empty = q_full + 1;      // S^T of a run done
  uint64_t* o_done = q_empty + 1;      // P V of a run done
  uint64_t* o_free = o_done + 1;       // O^T of a run read out
  uint64_t* nf_rdy = o_free + 1;       // preparation of a run done (noted rows final)
  uint64_t* drain = nf_rdy + 1;        // both issuers: every MMA complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[i], Q8 ? PM : 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&v_full[i], Q8 ? PM : 1);
      mbar_init(&v_raw[i], 1);
      mbar_init(&v_clean[i], PW);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < Cfg::kRS; ++i) {
      mbar_init(&r_full[i], 1);
      mbar_init(&r_empty[i], PM);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&p_full[i], 4);
      mbar_init(&p_free[i], 1);
    }
    mbar_init(q_full, PW);
    mbar_init(q_empty, 1);
    mbar_init(o_done, 1);
    mbar_init(o_free, 4);
    mbar_init(nf_rdy, PW);
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, Cfg::kCols);
    tmem_relinquish();
  }
  pdl_launch_dependents();
  pdl_wait();   // every global access below comes after the previous kernel
  if (warp == 3) tree_schedule(p, sched, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{abort_flag, p.status, 2000000000ull};
  // a wait that may last a whole run; it ends at once when another wait gives up
  const WaitCtl run_ctl{abort_flag, p.status, 30000000000ull};
  TreeWalk walk = tree_begin(sched);
  Seg sg;

  if (warp == 0) {
    // ------------------------------------------------------------ S^T = K Q^T
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(128, N);
      const uint64_t qd = sdesc_sw128_kmajor(smem_u32(qs));
      const uint64_t kd = sdesc_sw128_kmajor(smem_u32(kst));
      bool ok = true;
      int g = 0;
      for (int w = 0; ok && tree_next(p, sched, walk, sg); ++w) {
        ok = mbar_wait(q_full, w & 1, ctl);
        for (int j = sg.k0; j < sg.k1 && ok; ++j, ++g) {
          const int ks = g % KS, sb = g & 3;
          ok = mbar_wait(&k_full[ks], (g / KS) & 1, ctl);
          if (g >= 4) ok = ok && mbar_wait(&s_free[sb], ((g >> 2) - 1) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kds = kd + (uint64_t)(ks * (Cfg::kTileBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_f16(tmem + N * sb, kds + (kk >> 2) * (kTile * 128 >> 4) + 2 * (kk & 3),
                       qd + (kk >> 2) * (N * 128 >> 4) + 2 * (kk & 3), idesc, kk > 0 ? 1u : 0u);
          tc_commit(&s_full[sb]);
          tc_commit(&k_empty[ks]);
        }
        if (ok) tc_commit(q_empty);
      }
      tc_commit(drain);
      mbar_wait_drain(drain, 0, 200000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ O^T += V^T P^T
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(128, N) | (1u << 15);   // A (V) M-major
      // 64 values a panel; D = 64: the second 64 lanes read the same panel
      const uint64_t vd = sdesc_sw128_nmajor(smem_u32(vst), D == 128 ? kTile * 128 : 0);
      const uint64_t pd = sdesc_sw128_kmajor(smem_u32(ps));
      uint32_t full_ph = 0, clean_ph = 0;   // phase bits of v_full and v_clean of each stage
      bool ok = true;
      int g = 0;
      for (int w = 0; ok && tree_next(p, sched, walk, sg); ++w) {
        const int jm = first_masked(sg);
        for (int j = sg.k0; j < sg.k1 && ok; ++j, ++g) {
          const int vs = g % VS, pb = g & 1;
          if (!Q8 && j >= jm) {
            ok = mbar_wait(&v_clean[vs], (clean_ph >> vs) & 1, ctl);
            clean_ph ^= 1u << vs;
          } else {
            ok = mbar_wait(&v_full[vs], (full_ph >> vs) & 1, ctl);
            full_ph ^= 1u << vs;
          }
          ok = ok && mbar_wait(&p_full[pb], (g >> 1) & 1, ctl);
          if (j == sg.k0 && w > 0) ok = ok && mbar_wait(o_free, (w - 1) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vds = vd + (uint64_t)(vs * (Cfg::kTileBytes >> 4));
          const uint64_t pds = pd + (uint64_t)(pb * (Cfg::kPBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ss_f16(tmem + Cfg::kOCol, vds + (uint32_t)(kk * (2048 >> 4)),
                       pds + (kk >> 2) * (N * 128 >> 4) + 2 * (kk & 3), idesc, (kk > 0 || j > sg.k0) ? 1u : 0u);
          tc_commit(&v_empty[vs]);
          tc_commit(&p_free[pb]);
        }
        if (ok) tc_commit(o_done);
      }
      tc_commit(drain);
      mbar_wait_drain(drain, 0, 200000000ull);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------ copies
    if (lane == 0 && (!Q8 || warp == 2)) {
      bool ok = true;
      int n = 0;          // copies issued
      const int ns = Q8 ? RS : warp == 2 ? KS : VS;
      uint64_t* full = Q8 ? r_full : warp == 2 ? k_full : v_full;
      uint64_t* empty = Q8 ? r_empty : warp == 2 ? k_empty : v_empty;
      uint8_t* ring = Q8 ? raws : warp == 2 ? kst : vst;
      const CUtensorMap* map = warp == 2 ? &tm_k : &tm_v;
      uint32_t full_ph = 0, raw_ph = 0;     // phases that have been armed, by stage
      if (!Q8) tma_prefetch_desc(map);
      while (ok && tree_next(p, sched, walk, sg)) {
        const int jm = first_masked(sg);
        const long long head = (long long)sg.b * p.Hkv + sg.hk;
        const int last = (int)min((long long)sg.past + p.N, (long long)p.C);   // rows in use
        for (int j = sg.k0; j < sg.k1 && ok; ++j)
#pragma unroll 1
          for (int kv = 0; kv < (Q8 ? 2 : 1); ++kv, ++n) {
            const int sl = n % ns;
            if (n >= ns && !mbar_wait_idle(&empty[sl], ((n / ns) - 1) & 1, ctl, 32)) { ok = false; break; }
            if constexpr (Q8) {
              long long at;
              uint32_t bytes;
              raw_span(head, p.C, Cfg::kRow, j, last, at, bytes);
              full_ph ^= 1u << sl;
              mbar_arrive_expect_tx(&full[sl], bytes);
              if (in_bounds(at >= 0 && bytes > 0 && bytes <= (uint32_t)Cfg::kRaw &&
                                at + bytes <= (long long)(p.B_all - p.b0) * p.Hkv * p.C * Cfg::kRow,
                            p.status, kSiteTreeKV))
                bulk_load(ring + sl * Cfg::kRaw, (kv ? p.v : p.k) + at, bytes, &full[sl]);
            } else {
              // V of a masked tile goes by way of the clearing warps
              const bool raw = warp == 3 && j >= jm;
              uint64_t* bar = raw ? &v_raw[sl] : &full[sl];
              (raw ? raw_ph : full_ph) ^= 1u << sl;
              mbar_arrive_expect_tx(bar, Cfg::kTileBytes);
#pragma unroll
              for (int pn = 0; pn < D / 64; ++pn)
                if (in_bounds(j >= 0 && (long long)j * kTile < p.C && head >= 0 && head < (long long)p.B * p.Hkv, p.status,
                              kSiteTreeKV))
                  tma_load_3d(ring + sl * Cfg::kTileBytes + pn * (kTile * 128), map, bar, 64 * pn, j * kTile,
                              (int)(head + (long long)p.b0 * p.Hkv));
            }
          }
      }
      if (!ok)   // copies in flight land before the CTA can leave: the last armed phase of each barrier
        for (int i = 0; i < ns; ++i) {
          mbar_wait_drain(&full[i], ((full_ph >> i) & 1) ^ 1, 100000000ull);
          if (!Q8 && warp == 3) mbar_wait_drain(&v_raw[i], ((raw_ph >> i) & 1) ^ 1, 100000000ull);
        }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int sw = warp - 4;                       // = warp & 3: TMEM lanes 32 sw ..
    const int key = 32 * sw + lane;                // this thread's key of a tile, and its d of O^T
    const uint32_t lanes = (uint32_t)(32 * sw) << 16;
    uint32_t* anc = anc_all + 32 * sw;             // each warp has a copy: [row]
    // P^T: row n, key: panel key / 64, 16-byte chunk ((key % 64) / 8) ^ (n % 8)
    uint8_t* pbase = ps + (key >> 6) * (N * 128) + (key & 7) * 2;
    const int pchunk = (key & 63) >> 3;
    const float sc = p.scale_log2;
    const int R = p.N * p.G;                       // rows, at most N
    bool bad = false;                              // a wait gave up
    bool stop = false;
    bool fresh = true;                             // the CTA's first run
    int g = 0;
    for (int w = 0; !stop && tree_next(p, sched, walk, sg); ++w) {
      const int jm = first_masked(sg);
      int* unused_s = unused_all + (w & 1) * N;
      if (sg.k1 > jm) {
        // the tree's bits, lane = row (nodes are at most 32: one word)
        uint32_t bits = 0;
        bool used = true;
        if (lane < R) used = ancestors<1>(p.parents + (long long)sg.b * p.N, lane / p.G, &bits, 1);
        anc[lane] = bits;
        if (sw == 0 && lane < N) unused_s[lane] = used ? 0 : 1;
        __syncwarp();
      }
      float l[N];
#pragma unroll
      for (int n = 0; n < N; ++n) l[n] = 0.f;
      for (int j = sg.k0; j < sg.k1; ++j, ++g) {
        const int sb = g & 3, pb = g & 1;
        const bool first = j == sg.k0;
        bad = bad || !mbar_wait(&s_full[sb], (g >> 2) & 1, ctl);
        bad = __any_sync(0xffffffffu, bad);
        const uint32_t scol = tmem + lanes + N * sb;
        const bool masked = j >= jm;
        uint32_t vis = 0xFFFFFFFFu;                // rows that see this key
        if (masked) {
          const int kabs = j * kTile + key, rel = kabs - sg.past;
          vis = 0u;
          if (kabs < p.C) {
            if (rel < 0) vis = 0xFFFFFFFFu;
            else if (rel < 32)
              for (int n = 0; n < R; ++n) vis |= ((anc[n] >> rel) & 1u) << n;
          }
        }
        bool above = first;
        float x[N];
        if (!bad) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            uint32_t v[16];
            tmem_ld16_wait(scol + 16 * c, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[16 * c + e] = __uint_as_float(v[e]) * sc;
          }
          if (masked) {
#pragma unroll
            for (int n = 0; n < N; ++n) x[n] = (vis >> n) & 1u ? x[n] : -INFINITY;
          }
          if (!first) {
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < N; n += 4) {
              const float4 m4 = *reinterpret_cast<const float4*>(mref + n);
              top = fmaxf(top, fmaxf(fmaxf(x[n] - m4.x, x[n + 1] - m4.y), fmaxf(x[n + 2] - m4.z, x[n + 3] - m4.w)));
            }
            above = top > kRaise;   // a row without a reference yet has -inf: a key that it sees is above
          }
          tc_fence_before();
        }
        // the warps go on, or leave, together (a named barrier has no time limit)
        if (vote_or(1, 128, above || bad)) {
          // ------------------------------------------------ raise references
          // column maxima over the tile's keys
#pragma unroll
          for (int n = 0; n < N; ++n) {
            float t = bad ? -INFINITY : x[n];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
            if (lane == (n & 31)) wmax[sw * N + n] = t;
          }
          // O^T holds the run's earlier tiles: their P V have to be done
          if (!first && !bad) bad = !mbar_wait(&p_free[(g - 1) & 1], ((g - 1) >> 1) & 1, ctl);
          if (vote_or(1, 128, bad)) {
            stop = true;
            break;
          }
          if (sw == 0 && lane < N) {
            const float t = fmaxf(fmaxf(wmax[lane], wmax[N + lane]), fmaxf(wmax[2 * N + lane], wmax[3 * N + lane]));
            const float m = first ? -INFINITY : mref[lane];
            const float nm = t > m + kRaise || m == -INFINITY ? fmaxf(m, t) : m;
            fac[lane] = m == -INFINITY ? 0.f : ex2(m - nm);
            mref[lane] = nm;
          }
          vote_or(1, 128, false);
          if (!first) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < NC; ++c) {
              uint32_t v[16];
              tmem_ld16_wait(tmem + lanes + Cfg::kOCol + 16 * c, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float f = fac[16 * c + e];
                v[e] = f == 1.f ? v[e] : __float_as_uint(__uint_as_float(v[e]) * f);
              }
              tmem_st16(tmem + lanes + Cfg::kOCol + 16 * c, v);
            }
            tmem_wait_st();
            tc_fence_before();
#pragma unroll
            for (int n = 0; n < N; ++n) l[n] *= fac[n];
          }
        }
        // P^T over the buffer of tile g - 2
        if (g >= 2) bad = !__all_sync(0xffffffffu, mbar_wait(&p_free[pb], ((g >> 1) - 1) & 1, ctl));
        if (!bad) {
          uint8_t* dst = pbase + pb * Cfg::kPBytes;
#pragma unroll
          for (int n = 0; n < N; n += 4) {
            const float4 m4 = *reinterpret_cast<const float4*>(mref + n);
            const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // a masked key's x is -inf, also where the reference is
              const float pv = x[n + e] == -INFINITY ? 0.f : ex2(x[n + e] - m[e]);
              l[n + e] += pv;
              *reinterpret_cast<__half*>(dst + (n + e) * 128 + ((pchunk ^ ((n + e) & 7)) << 4)) = __float2half_rn(pv);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive_warp(&s_free[sb]);
          mbar_arrive_warp(&p_full[pb]);
        }
      }
      if (stop) break;
      // ---------------------------------------------------------- end of a run
      // sums over the 128 key lanes
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float t = l[n];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == (n & 31)) wmax[sw * N + n] = t;
      }
      const int par = w & 1;
      bad = bad || !(mbar_wait(o_done, par, ctl) && mbar_wait(nf_rdy, par, ctl));
      if (vote_or(1, 128, bad)) {
        stop = true;
        break;
      }
      tc_fence_after();
      const bool whole = sg.k0 == 0 && sg.k1 == sg.nk;
      const bool tree = sg.k1 > jm;
      const long long slot = (2ll * blockIdx.x + (fresh ? 0 : 1)) * p.ws_rows;
      if (sw == 0 && lane < N) {
        const float L = wmax[lane] + wmax[N + lane] + wmax[2 * N + lane] + wmax[3 * N + lane];
        const bool un = tree && unused_s[lane];
        // a whole item is divided by its sum (a row without a key is zero)
        linv[lane] = !whole ? 1.f : L > 0.f ? 1.f / L : L;
        if (!whole && lane < R && in_bounds(p.split && lane < p.ws_rows, p.status, kSiteTreeWs))
          p.ws_ml[slot + lane] = make_float2(mref[lane], un ? -1.f : L);
      }
      uint32_t some = 0;
      if (tree)
        for (int i = lane; i < PW * 4; i += 32) some |= noted[par * PW * 4 + i];
      const bool anynf = __any_sync(0xffffffffu, some != 0u);
      vote_or(1, 128, false);   // linv is written
      const int d = Q8 ? (key & ~31) + q8_code_at((key >> 5) & 1, key & 31) : key;
#pragma unroll 1
      for (int c = 0; c < NC; ++c) {
        uint32_t v[16];
        tmem_ld16_wait(tmem + lanes + Cfg::kOCol + 16 * c, v);
        if (key < D) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int n = 16 * c + e;
            if (n >= R) break;
            float o = __uint_as_float(v[e]) * linv[n];
            const bool un = tree && unused_s[n];
            if (anynf && !un) {
              // non-finite values of cleared V rows that this row sees
              for (int mt = 0; mt < 4; ++mt)
                for (int q = 0; q < 4; ++q) {
                  if (jm + mt < sg.k0 || jm + mt >= sg.k1) continue;
                  const int kq = (jm + mt) * kTile + 32 * q;
                  uint32_t bits = 0;
                  for (int i = q; i < PW; i += 4) bits |= noted[par * PW * 4 + 4 * i + mt];
                  bits &= seen32<1>(anc + n, 0, kq, sg.past, p.C);
                  while (bits) {
                    const int k = kq + __ffs(bits) - 1;
                    bits &= bits - 1;
                    const float z = value_at<D, Q8>(p, sg, k, d);
                    if (!(z - z == 0.f)) o += z;
                  }
                }
            }
            const int node = n / p.G, h = sg.hk * p.G + n % p.G;
            if (whole) {
              if (in_bounds(node < p.N && h < p.H, p.status, kSiteTreeO))
                p.o[((long long)sg.b * p.N + node) * p.H * D + (long long)h * D + d] = __float2half_rn(un ? 0.f : o);
            } else if (in_bounds(p.split && n < p.ws_rows, p.status, kSiteTreeWs)) {
              p.ws_o[(slot + n) * D + d] = o;
            }
          }
        }
        __syncwarp();
      }
      fresh = false;
      tc_fence_before();
      mbar_arrive_warp(o_free);
    }
  } else {
    // ------------------------------------------------------------ Q, decode, clearing
    const int t = threadIdx.x - 8 * 32;         // 0 .. 32 PW - 1
    const int pw = warp - 8;
    const int R = p.N * p.G;
    const DecK K = make_deck();
    bool ok = true;
    int g = 0;
    uint32_t raw_ph = 0;                        // phase bits of v_raw of each stage
    for (int w = 0; ok && tree_next(p, sched, walk, sg); ++w) {
      const int jm = first_masked(sg);
      ok = __all_sync(0xffffffffu, w == 0 || mbar_wait_idle(q_empty, (w - 1) & 1, run_ctl, 64));
      if (!ok) break;
      uint32_t* nt = noted + (w & 1) * PW * 4 + pw * 4;
      if (lane < 4) nt[lane] = 0u;
      __syncwarp();
      // Q rows (Q8_0: in the decoded blocks' order), a block of 32 values a thread
      for (int u = t; u < N * (D / 32); u += 32 * PW) {
        const int n = u / (D / 32), blk = u % (D / 32);
        uint4 q[4] = {}, o[4];
        if (n < R) {
          const int node = n / p.G, h = sg.hk * p.G + n % p.G;
          if (in_bounds(node < p.N && h < p.H, p.status, kSiteTreeQ)) {
            const uint4* src =
                reinterpret_cast<const uint4*>(p.q + ((long long)h * p.q_rows + (long long)sg.b * p.N + node) * D) + 4 * blk;
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = __ldg(src + i);
          }
        }
        if constexpr (Q8) order_block(q, blk & 1, o);
        else
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = q[i];
        uint8_t* base = qs + (blk >> 1) * (N * 128) + n * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(base + (((4 * (blk & 1) + i) ^ (n & 7)) << 4)) = o[i];
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(q_full);
      const long long head = (long long)sg.b * p.Hkv + sg.hk;
      for (int j = sg.k0; j < sg.k1 && ok; ++j, ++g) {
        const int ks = g % KS, vs = g % VS;
        if constexpr (Q8) {
          const int sh = (int)(((head * p.C + (long long)j * kTile) * Cfg::kRow) & 15);
          // D = 128: all warps decode K, then V; D = 64: one half each
          const int row = t & 127, blk = D == 128 ? t >> 7 : (t >> 7) & 1;
#pragma unroll 1
          for (int kv = D == 128 ? 0 : t >> 8; kv < 2; kv += D == 128 ? 1 : 2) {
            const int rn = 2 * g + kv, rs = rn % RS;
            const int ns = kv ? VS : KS;
            bool go = mbar_wait(&r_full[rs], (rn / RS) & 1, ctl);
            if (g >= ns) go = go && mbar_wait(kv ? &v_empty[vs] : &k_empty[ks], ((g / ns) - 1) & 1, ctl);
            ok = __all_sync(0xffffffffu, go);
            if (!ok) break;
            uint8_t* dst = kv ? vst + vs * Cfg::kTileBytes : kst + ks * Cfg::kTileBytes;
            uint32_t v[16];
            decode_block<D>(raws + rs * Cfg::kRaw + sh, row, blk, K, v);
            if (kv && j >= jm) {
              bool any = false;
#pragma unroll
              for (int q = 0; q < 16; ++q) any |= clear_nonfinite(v[q]);
              const uint32_t bits = __ballot_sync(0xffffffffu, any);
              if (lane == 0) nt[j - jm] = bits;
            }
            uint8_t* base = dst + (blk >> 1) * (kTile * 128) + row * 128;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(base + (((4 * (blk & 1) + i) ^ (row & 7)) << 4)) =
                  make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            fence_proxy_async_smem();
            mbar_arrive_warp(kv ? &v_full[vs] : &k_full[ks]);
            mbar_arrive_warp(&r_empty[rs]);
            if (D == 64) break;
          }
        } else if (j >= jm) {
          ok = __all_sync(0xffffffffu, mbar_wait_idle(&v_raw[vs], (raw_ph >> vs) & 1, run_ctl, 64));
          if (!ok) break;
          raw_ph ^= 1u << vs;
          const uint32_t bits = clean_tile<D, 32 * PW>(vst + vs * Cfg::kTileBytes, t);
          if (lane == 0) nt[j - jm] = bits;
          fence_proxy_async_smem();
          mbar_arrive_warp(&v_clean[vs]);
        }
      }
      // The notes of run w + 1 go where those of run w - 1 were: their readers
      // are done once O of run w - 1 is free.  Waited for here, before the
      // arrival that lets run w end, so that o_free is at most one phase ahead.
      if (ok && w >= 1) ok = __all_sync(0xffffffffu, mbar_wait_idle(o_free, (w - 1) & 1, run_ctl, 64));
      if (ok) mbar_arrive_warp(nf_rdy);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kCols);
  }
}

template <int D, bool Q8, int NC>
cudaError_t launch_few(const TreeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int grid,
                       cudaStream_t s) {
  using Cfg = FewCfg<D, Q8, NC>;
  auto kern = few_kernel<D, Q8, NC>;
  cudaError_t e = allow_smem<std::integer_sequence<int, 6, D, Q8, NC>>(kern, Cfg::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_tree_kernel(kern, (unsigned)grid, Cfg::kThreads, Cfg::kSmem, s, tm_k, tm_v, p);
  return e != cudaSuccess || !p.split ? e : launch_tree_join<D>(p, grid, s);
}

template <int D, bool Q8>
cudaError_t launch_few_dq(const TreeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int grid,
                          cudaStream_t s) {
  return p.N * p.G <= 16 ? launch_few<D, Q8, 1>(p, tm_k, tm_v, grid, s) : launch_few<D, Q8, 2>(p, tm_k, tm_v, grid, s);
}

}  // namespace

cudaError_t launch_attention_few(const TreeParams& p, bool q8, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                 int grid, cudaStream_t s) {
  if (p.D == 64)
    return q8 ? launch_few_dq<64, true>(p, tm_k, tm_v, grid, s) : launch_few_dq<64, false>(p, tm_k, tm_v, grid, s);
  return q8 ? launch_few_dq<128, true>(p, tm_k, tm_v, grid, s) : launch_few_dq<128, false>(p, tm_k, tm_v, grid, s);
}

}  // namespace m4q
