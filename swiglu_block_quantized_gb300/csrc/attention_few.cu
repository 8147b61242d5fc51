// attention_few.cu -- m4q_attention_tree for items of few rows (nodes times
// query heads of a group at most 32): single new tokens and small trees.
//
// With few rows the 128 lanes of a tcgen05 tile are best given to the keys:
//   S^T = K Q^T       M = 128 keys, N = 16 or 32 rows: lane = key
//   O^T += V^T P^T    M = D (two copies of 64 when D = 64), N = rows: lane = d
// so that the softmax of a tile is a few values a thread whatever the mask, and
// the MMAs shrink with N.  V is the A operand as it lies ([key][D], M-major), P
// the small K-major B operand in shared memory.  (O += P V with P as a 128-row A
// operand took 122 us against 107 where this was measured, 32 sequences of one
// token: most of those rows are nobody's, and reading them costs the shared
// memory that the decode needs.)
// What is left is the stream of the cache: HBM should bound the fp16 kernel. For
// Q8_0 the shared memory comes close: a tile of 128 keys at D = 128 is 1500 clocks
// of HBM time, and with both decoded tiles in shared memory its copy, decode and
// MMAs move 198 KB there, 1550 clocks. So K is decoded into TMEM instead (lane =
// key, the A operand from there), which leaves 134 KB; V has to be read across
// its keys and stays in shared memory.
//
// A row's reference maximum is kept while its scores stay within 2^8 of it, so
// the usual tile needs no maximum across the keys: each thread forms its
// exponents against the reference and the four warps vote (one barrier) whether
// one is above 8.  If so (always in a run's first tile) they find the rows'
// maxima, raise the references and rescale O^T and the sums.  Row sums stay in
// the threads (one partial sum a key lane and row) until the run ends.
//
// Tiles go to two teams in turn, each with its own P^T, O^T, references and sums,
// joined when a run ends: a tile's chain from scores to P takes about 2500 clocks
// whatever its size (barriers, TMEM loads, the fence before the MMA reads P), and
// two of them overlap.
//
// Measured: 32 sequences of one token, 4 heads a group, D = 128, over 500 to 8,100
// Q8_0 keys in 95 us (300 MB: 3.1 TB/s) and as many fp16 keys in 95 (564 MB: 5.9
// TB/s), over 32,000 to 32,700 in 411 (5.5 TB/s) and 602 (4.24 GB: 7.0 TB/s, HBM's
// rate for reads); at D = 64, 70, 63, 333 and 329 us (2.1, 4.4, 3.4, 6.4 TB/s).  8
// nodes over 300 fp16 keys take 9.7.  Q8_0 is bound by the decode warps: their
// instructions, the fetch of these (72 KB of code; the second stall after TMEM and
// shared memory loads) and the latency of a group (half of the issue slots are
// empty, 64 bytes a thread are spilled at 72 registers); short calls by the start and
// end of a run.
//
// P is rounded to fp16, the type of the MMA with V (V is fp16, or decoded to it): 2^-11
// of each weight, 2.9e-4 of the result against 2.1e-4 when only that is rounded.  The
// sums are of the unrounded P.
//
// Warps: 0 issues the S MMAs (four TMEM buffers ahead), 1 the P V MMAs, 2 and 3
// the copies, 4-11 are the softmax teams (lane = key), the others prepare (Q, the
// clearing of non-finite V; Q8_0: groups of four decode K or V tiles), as in
// attention_tree.cu, whose notes on masks, schedule and pieces hold here.
#include <algorithm>

#include "tree_common.cuh"
#include "tree_rings.h"

namespace m4q {

namespace {

template <int D, bool Q8, int NC>
struct FewCfg {
  static constexpr int N = 16 * NC;                    // rows (columns of S^T)
  static constexpr int kRow = Q8 ? D / 32 * 34 : 2 * D;
  static constexpr int kTileBytes = kTile * D * 2;     // an fp16 tile: D / 64 panels of [128][128 B]
  static constexpr int kQBytes = N * D * 2;            // D / 64 panels of [N][128 B]
  static constexpr int kPBytes = N * kTile * 2;        // two panels (64 keys) of [N][128 B]
  static constexpr FewRings kRings = few_rings(D, Q8, NC);
  static constexpr int kKS = kRings.ks;                // K stages (Q8_0: in TMEM)
  static constexpr int kVS = kRings.vs;
  static constexpr int kRaw = kTile * kRow + 32;       // a raw tile, its 16-byte shift, and the decode's overread
  static constexpr int kRS = kRings.rs;
  static constexpr int kGroups = kRings.groups;
  static constexpr int kPrep = Q8 ? 8 * kGroups : 4;   // preparing warps
  static constexpr int kThreads = 32 * (12 + kPrep);
  static constexpr int kBars = 2 * kKS + 4 * kVS + 3 * kRS + 8 + 4 + 7;
  static constexpr int kFixed = (int)sizeof(TreeSched) + 2 * 8 * 16   // schedule, noted rows
                                + 8 * 32 * 4                          // ancestor bits by warp
                                + 2 * 4 * N * 4 + 4 * N * 4           // wmax, mref and fac by team
                                + 4 * N * 8                           // (m, l) [parity][team]
                                + 2 * 8 + kBars * 8 + 64;
  static constexpr int kSmem = 1024 + kQBytes + 2 * kPBytes + ((Q8 ? 0 : kKS) + kVS) * kTileBytes + kRS * kRaw + kFixed;
  static constexpr uint32_t kOCol = 4 * N;             // S^T buffers at N i, then O^T of the teams
  static constexpr uint32_t kKCol = 6 * N;             // Q8_0: K stages of D / 2 columns
  static constexpr uint32_t kUsed = kKCol + (Q8 ? kKS * D / 2 : 0);
  static constexpr uint32_t kCols = kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= 512, "TMEM budget");
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(few_groups_ok(kRings), "a raw slot is used again after its stage");
  static_assert(kRaw % 16 == 0 && kQBytes % 1024 == 0 && kPBytes % 1024 == 0, "alignment");
};

// Sums (or maxima) of N values over the warp: halves of the rows change lanes,
// N / 2 + N / 4 + ... shuffles instead of 5 N.  Returned: row `lane` (N = 32) or
// lane / 2 (N = 16).
template <int N, bool MAX>
__device__ __forceinline__ float reduce_rows(float (&l)[N], int lane) {
#pragma unroll
  for (int h = N / 2, bit = 16; h >= 1; h /= 2, bit /= 2) {
#pragma unroll
    for (int n = 0; n < h; ++n) {
      const float keep = lane & bit ? l[n + h] : l[n], give = lane & bit ? l[n] : l[n + h];
      const float got = __shfl_xor_sync(0xffffffffu, give, bit);
      l[n] = MAX ? fmaxf(keep, got) : keep + got;
    }
  }
  if constexpr (N == 16) {
    const float got = __shfl_xor_sync(0xffffffffu, l[0], 1);
    return MAX ? fmaxf(l[0], got) : l[0] + got;
  }
  return l[0];
}

// 4 consecutive 32-bit TMEM columns of this thread's lane: loaded and waited
// for, or stored.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&v)[4]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}

// Sum of the non-finite values at d of the cleared V rows that a row sees (0 if
// there is none).
template <int D, bool Q8>
__device__ __noinline__ float few_nonfinite(const TreeParams& p, Seg g, const uint32_t* noted, uint32_t anc, int d) {
  const int jm = first_masked(g);
  float z = 0.f;
#pragma unroll 1
  for (int mt = 0; mt < 4; ++mt) {
    if (jm + mt < g.k0 || jm + mt >= g.k1) continue;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      const int kq = (jm + mt) * kTile + 32 * q;
      uint32_t bits = (noted[4 * q + mt] | noted[4 * (q + 4) + mt]) & seen32<1>(&anc, 0, kq, g.past, p.C);
      while (bits) {
        const float v = value_at<D, Q8>(p, g, kq + __ffs(bits) - 1, d);
        bits &= bits - 1;
        if (!(v - v == 0.f)) z += v;
      }
    }
  }
  return z;
}

template <int D, bool Q8, int NC>
__global__ void __launch_bounds__(FewCfg<D, Q8, NC>::kThreads, 1)
    few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const TreeParams p) {
  using Cfg = FewCfg<D, Q8, NC>;
  constexpr int N = Cfg::N, KS = Cfg::kKS, VS = Cfg::kVS, RS = Cfg::kRS > 0 ? Cfg::kRS : 1;
  constexpr int PW = Cfg::kPrep, PG = Cfg::kGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = smem_align<1024>(smem_raw);
  uint8_t* ps = qs + Cfg::kQBytes;                     // [2] P^T
  uint8_t* kst = ps + 2 * Cfg::kPBytes;
  uint8_t* vst = kst + (Q8 ? 0 : KS) * Cfg::kTileBytes;
  uint8_t* raws = vst + VS * Cfg::kTileBytes;
  uint32_t* noted = reinterpret_cast<uint32_t*>(raws + Cfg::kRS * Cfg::kRaw);   // [parity][8 warps][4]
  uint32_t* anc_all = noted + 2 * 8 * 4;               // [warp][32] ancestor bits of a row
  float* wmax_all = reinterpret_cast<float*>(anc_all + 8 * 32);   // [team][warp][N] column maxima, or sums
  float* mref_all = wmax_all + 2 * 4 * N;              // [team][N] references
  float* fac_all = mref_all + 2 * N;                   // [team][N] rescale factors
  float2* ml = reinterpret_cast<float2*>(fac_all + 2 * N);        // [parity][team][N]
  uint32_t* unused_s = reinterpret_cast<uint32_t*>(ml + 4 * N);                // [parity] rows of unused nodes
  TreeSched* sched = reinterpret_cast<TreeSched*>(unused_s + 4);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sched) + (sizeof(TreeSched) + 7) / 8 * 8);
  uint64_t* k_empty = k_full + KS;     // [KS] S^T done with it
  uint64_t* v_full = k_empty + KS;     // [VS] V of a tile in its stage
  uint64_t* v_raw = v_full + VS;       // [VS] (fp16) V of a masked tile, not yet cleared
  uint64_t* v_clean = v_raw + VS;      // [VS] (fp16) V of a masked tile, cleared
  uint64_t* v_empty = v_clean + VS;    // [VS] P V done with it
  uint64_t* r_full = v_empty + VS;     // [2][RS] raw tile (K, V) landed in a slot
  uint64_t* r_empty = r_full + 2 * Cfg::kRS;
  uint64_t* s_full = r_empty + Cfg::kRS;   // [4] S^T of a tile in TMEM
  uint64_t* s_free = s_full + 4;       // [4] read
  uint64_t* p_full = s_free + 4;       // [2] P^T written
  uint64_t* p_free = p_full + 2;       // [2] P V done
  uint64_t* q_full = p_free + 2;       // Q of a run written
  uint64_t* q_empty = q_full + 1;      // S^T of a run done
  uint64_t* o_done = q_empty + 1;      // P V of a run done
  uint64_t* o_free = o_done + 1;       // O^T of a run read out
  uint64_t* nf_rdy = o_free + 1;       // preparation of a run done (noted rows final)
  uint64_t* ml_rdy = nf_rdy + 1;       // both teams' (m, l) of a run
  uint64_t* drain = ml_rdy + 1;        // both issuers: every MMA complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[i], Q8 ? 4 : 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&v_full[i], Q8 ? 4 : 1);
      mbar_init(&v_raw[i], 1);
      mbar_init(&v_clean[i], PW);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < Cfg::kRS; ++i) {
      mbar_init(&r_full[few_raw_bar(Cfg::kRS, 0, i)], 1);
      mbar_init(&r_full[few_raw_bar(Cfg::kRS, 1, i)], 1);
      mbar_init(&r_empty[i], 4);
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
    mbar_init(o_free, 8);
    mbar_init(ml_rdy, 2);
    mbar_init(nf_rdy, PW);
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, Cfg::kCols);
    tmem_relinquish();
  }
  pdl_wait();   // every global access below comes after the previous kernel
  pdl_launch_dependents();   // after it: see join_span
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
      Ring<KS> kr;
      for (int w = 0; ok && tree_next(p, sched, walk, sg); ++w) {
        ok = mbar_wait(q_full, w & 1, ctl);
        for (int j = sg.k0; j < sg.k1 && ok; ++j, ++g, kr.step()) {
          const int ks = kr.at, sb = g & 3;
          ok = mbar_wait(&k_full[ks], kr.ph, ctl);
          if (g >= 4) ok = ok && mbar_wait(&s_free[sb], ((g >> 2) - 1) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          if constexpr (Q8) {
            const uint32_t kcol = tmem + Cfg::kKCol + ks * (D / 2);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma_ts_f16(tmem + N * sb, kcol + 8 * kk, qd + (kk >> 2) * (N * 128 >> 4) + 2 * (kk & 3), idesc,
                            kk > 0 ? 1u : 0u);
          } else {
            const uint64_t kds = kd + (uint64_t)(ks * (Cfg::kTileBytes >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss_f16(tmem + N * sb, kds + (kk >> 2) * (kTile * 128 >> 4) + 2 * (kk & 3),
                         qd + (kk >> 2) * (N * 128 >> 4) + 2 * (kk & 3), idesc, kk > 0 ? 1u : 0u);
          }
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
      Ring<VS> vr;
      for (int w = 0; ok && tree_next(p, sched, walk, sg); ++w) {
        const int jm = first_masked(sg);
        for (int j = sg.k0; j < sg.k1 && ok; ++j, ++g, vr.step()) {
          const int vs = vr.at, pb = g & 1;
          if (!Q8 && j >= jm) {
            ok = mbar_wait(&v_clean[vs], (clean_ph >> vs) & 1, ctl);
            clean_ph ^= 1u << vs;
          } else {
            ok = mbar_wait(&v_full[vs], (full_ph >> vs) & 1, ctl);
            full_ph ^= 1u << vs;
          }
          ok = ok && mbar_wait(&p_full[pb], (g >> 1) & 1, ctl);
          if (j == sg.k0 && w > 0) ok = ok && mbar_wait(o_free, (w - 1) & 1, ctl);   // of both teams
          if (!ok) break;
          tc_fence_after();
          const uint64_t vds = vd + (uint64_t)(vs * (Cfg::kTileBytes >> 4));
          const uint64_t pds = pd + (uint64_t)(pb * (Cfg::kPBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ss_f16(tmem + Cfg::kOCol + N * pb, vds + (uint32_t)(kk * (2048 >> 4)),
                       pds + (kk >> 2) * (N * 128 >> 4) + 2 * (kk & 3), idesc, (kk > 0 || j > sg.k0 + 1) ? 1u : 0u);
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
        const long long head = (long long)(p.b0 + sg.b) * p.Hkv + sg.hk;
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
              const int rb = few_raw_bar(Cfg::kRS, kv, sl);
              full_ph ^= 1u << rb;
              mbar_arrive_expect_tx(&full[rb], bytes);
              if (in_bounds(at >= 0 && bytes > 0 && bytes <= (uint32_t)Cfg::kRaw &&
                                at + bytes <= (long long)p.B_all * p.Hkv * p.C * Cfg::kRow,
                            p.status, kSiteTreeKV))
                bulk_load(ring + sl * Cfg::kRaw, (kv ? p.v : p.k) + at, bytes, &full[rb]);
            } else {
              // V of a masked tile goes by way of the clearing warps
              const bool raw = warp == 3 && j >= jm;
              uint64_t* bar = raw ? &v_raw[sl] : &full[sl];
              (raw ? raw_ph : full_ph) ^= 1u << sl;
              mbar_arrive_expect_tx(bar, Cfg::kTileBytes);
#pragma unroll
              for (int pn = 0; pn < D / 64; ++pn)
                if (in_bounds(j >= 0 && (long long)j * kTile < p.C && head >= 0 && head < (long long)p.B_all * p.Hkv, p.status,
                              kSiteTreeKV))
                  tma_load_3d(ring + sl * Cfg::kTileBytes + pn * (kTile * 128), map, bar, 64 * pn, j * kTile,
                              (int)head);
            }
          }
      }
      if (!ok)   // copies in flight land before the CTA can leave: the last armed phase of each barrier
        for (int i = 0; i < (Q8 ? 2 * ns : ns); ++i) {
          mbar_wait_drain(&full[i], ((full_ph >> i) & 1) ^ 1, 100000000ull);
          if (!Q8 && warp == 3) mbar_wait_drain(&v_raw[i], ((raw_ph >> i) & 1) ^ 1, 100000000ull);
        }
    }
    __syncwarp();
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax
    const int team = (warp - 4) >> 2, sw = warp & 3;   // sw: TMEM lanes 32 sw ..
    const int key = 32 * sw + lane;                // this thread's key of a tile, and its d of O^T
    const uint32_t lanes = (uint32_t)(32 * sw) << 16;
    const uint32_t bar = 1 + team;                 // named barrier of the team
    const uint32_t ocol = tmem + lanes + Cfg::kOCol + N * team;
    uint32_t* anc = anc_all + 32 * (warp - 4);     // each warp has a copy: [row]
    float* wmax = wmax_all + team * 4 * N;
    float* mref = mref_all + team * N;
    float* fac = fac_all + team * N;
    // P: row n, key: panel key / 64, 16-byte chunk ((key % 64) / 8) ^ (n % 8)
    uint8_t* pdst = ps + team * Cfg::kPBytes + (key >> 6) * (N * 128) + (key & 7) * 2;
    const int pchunk = (key & 63) >> 3;
    const float sc = p.scale_log2;
    const int R = p.N * p.G;                       // rows, at most N
    // whole groups of 4 are computed; the P of later rows, whatever the buffer
    // holds, reaches only their own columns of O^T
    const int RU = (R + 3) & ~3;
    bool bad = false;                              // a wait gave up
    bool stop = false;
    bool fresh = true;                             // the CTA's first run
    int g = 0;
    for (int w = 0; !stop && tree_next(p, sched, walk, sg); ++w) {
      const int jm = first_masked(sg), par = w & 1;
      if (sg.k1 > jm) {
        // the tree's bits, lane = row (nodes are at most 32: one word)
        uint32_t bits;
        const bool used = ancestors32(p.parents + (long long)sg.b * p.N, p.N, lane < R ? lane / p.G : -1, bits);
        anc[lane] = bits;
        const uint32_t un = __ballot_sync(0xffffffffu, !used);
        if (warp == 4 && lane == 0) unused_s[par] = un;
        __syncwarp();
      }
      float l[N];
#pragma unroll
      for (int n = 0; n < N; ++n) l[n] = 0.f;
      for (int j = sg.k0; j < sg.k1; ++j, ++g) {
        if ((g & 1) != team) continue;
        const int sb = g & 3;
        const bool first = j < sg.k0 + 2;          // the team's first tile of the run
        // S^T, and the team's previous P V (its P is overwritten below, its O
        // rescaled when references rise)
        bool got = mbar_wait(&s_full[sb], (g >> 2) & 1, ctl);
        if (g >= 2) got = got && mbar_wait(&p_free[team], ((g >> 1) - 1) & 1, ctl);
        bad = !__all_sync(0xffffffffu, got);
        const uint32_t scol = tmem + lanes + N * sb;
        uint32_t vis = 0xFFFFFFFFu;                // rows that see this key
        if (j >= jm) {
          const int kabs = j * kTile + key, rel = kabs - sg.past;
          if (rel >= 0 || kabs >= p.C) {
            vis = 0u;
            if (kabs < p.C && rel < 32)
#pragma unroll 1
              for (int n = 0; n < R; ++n) vis |= ((anc[n] >> rel) & 1u) << n;
          }
        }
        const bool masked = __any_sync(0xffffffffu, vis != 0xFFFFFFFFu);
        // x: the thread's scaled scores (masked: -inf)
        float x[N];
        bool above = first;
        if (!bad) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            uint32_t v[16];
            tmem_ld16_wait(scol + 16 * c, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[16 * c + e] = __uint_as_float(v[e]) * sc;
          }
          tc_fence_before();
          mbar_arrive_warp(&s_free[sb]);
          if (masked) {
#pragma unroll
            for (int n = 0; n < N; ++n) x[n] = (vis >> n) & 1u ? x[n] : -INFINITY;
          }
          if (!first) {
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < N; n += 4) {
              if (n >= RU) break;
              const float4 m4 = *reinterpret_cast<const float4*>(mref + n);
              top = fmaxf(top, fmaxf(fmaxf(x[n] - m4.x, x[n + 1] - m4.y), fmaxf(x[n + 2] - m4.z, x[n + 3] - m4.w)));
            }
            above = top > kRaise;   // a row without a reference yet has -inf: a key that it sees is above
          }
        }
        // the warps go on, or leave, together (a named barrier has no time limit)
        if (vote_or(bar, 128, above || bad)) {
          if (vote_or(bar, 128, bad)) {
            stop = true;
            break;
          }
          // row maxima over the tile's keys
          float t[N];
#pragma unroll
          for (int n = 0; n < N; ++n) t[n] = x[n];
          wmax[sw * N + (NC == 1 ? lane >> 1 : lane)] = reduce_rows<N, true>(t, lane);
          vote_or(bar, 128, false);
          if (sw == 0 && lane < RU) {
            const float t = fmaxf(fmaxf(wmax[lane], wmax[N + lane]), fmaxf(wmax[2 * N + lane], wmax[3 * N + lane]));
            const float m = first ? -INFINITY : mref[lane];
            const float nm = t > m + kRaise || m == -INFINITY ? fmaxf(m, t) : m;
            fac[lane] = m == -INFINITY ? 0.f : ex2(m - nm);
            mref[lane] = nm;
          }
          vote_or(bar, 128, false);
          if (!first) {
#pragma unroll 1
            for (int n = 0; n < RU; n += 4) {
              uint32_t v[4];
              tmem_ld4(ocol + n, v);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * fac[n + e]);
              tmem_st4(ocol + n, v);
            }
            tmem_wait_st();
            tc_fence_before();
#pragma unroll
            for (int n = 0; n < N; ++n) {
              if (n >= RU) break;
              l[n] *= fac[n];
            }
          }
        }
        // P = 2^(x - m); a masked key's x is -inf, also where the reference is
#pragma unroll
        for (int n = 0; n < N; n += 4) {
          if (n >= RU) break;
          const float4 m4 = *reinterpret_cast<const float4*>(mref + n);
          const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float pv = x[n + i] == -INFINITY ? 0.f : ex2(x[n + i] - m[i]);
            l[n + i] += pv;
            *reinterpret_cast<__half*>(pdst + (n + i) * 128 + ((pchunk ^ ((n + i) & 7)) << 4)) = __float2half_rn(pv);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(&p_full[team]);
      }
      if (stop) break;
      // ---------------------------------------------------------- end of a run
      // sums over the 128 key lanes
      wmax[sw * N + (NC == 1 ? lane >> 1 : lane)] = reduce_rows<N, false>(l, lane);
      vote_or(bar, 128, false);
      const int len = sg.k1 - sg.k0, g0 = g - len;
      // a team without a tile of the run has no O^T and no references
      const bool has0 = len > 1 || !(g0 & 1), has1 = len > 1 || (g0 & 1), mine = team ? has1 : has0;
      if (sw == 0) {
        if (lane < RU)
          ml[(par * 2 + team) * N + lane] =
              mine ? make_float2(mref[lane], wmax[lane] + wmax[N + lane] + wmax[2 * N + lane] + wmax[3 * N + lane])
                   : make_float2(-INFINITY, 0.f);
        mbar_arrive_warp(ml_rdy);
      }
      const bool got = mbar_wait(ml_rdy, par, ctl) && mbar_wait(o_done, par, ctl) && mbar_wait(nf_rdy, par, ctl);
      bad = !__all_sync(0xffffffffu, got);
      if (vote_or(bar, 128, bad)) {
        stop = true;
        break;
      }
      tc_fence_after();
      const bool whole = sg.k0 == 0 && sg.k1 == sg.nk, tree = sg.k1 > jm;
      const uint32_t unused = tree ? unused_s[par] : 0u;
      // lane n: the factors of row n's two O^T columns, and where the row goes
      float f0 = 0.f, f1 = 0.f;
      int at = 0;
      if (lane < R) {
        const float2 a = ml[par * 2 * N + lane], b = ml[(par * 2 + 1) * N + lane];
        const float M = fmaxf(a.x, b.x);
        const float w0 = a.x == M ? 1.f : ex2(a.x - M), w1 = b.x == M ? 1.f : ex2(b.x - M);
        const float L = a.y * w0 + b.y * w1;
        // a whole item is divided by its sum (a row without a key is zero)
        const float inv = !whole ? 1.f : L > 0.f ? 1.f / L : L;
        f0 = w0 * inv;
        f1 = w1 * inv;
        const int node = lane / p.G, h = sg.hk * p.G + lane - node * p.G;
        const int piece = (2 * (int)blockIdx.x + (fresh ? 0 : 1)) * p.ws_rows + lane;
        at = whole ? (sg.b * p.N + node) * p.H + h : piece;   // B N H fits 31 bits
        if (warp == 4 && !whole && in_bounds(p.split && lane < p.ws_rows, p.status, kSiteTreeWs))
          p.ws_ml[piece] = make_float2(M, (unused >> lane) & 1u ? -1.f : L);
      }
      const bool anynf = __any_sync(0xffffffffu, tree && noted[par * 32 + lane] != 0u);
      // lane = d; the teams take groups of four rows in turn
      const int d = Q8 ? (key & ~31) + q8_code_at((key >> 5) & 1, key & 31) : key;
#pragma unroll 1
      for (int n0 = 4 * team; n0 < R; n0 += 8) {
        uint32_t v0[4], v1[4];
        tmem_ld4(tmem + lanes + Cfg::kOCol + n0, v0);
        tmem_ld4(tmem + lanes + Cfg::kOCol + N + n0, v1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = n0 + e;
          const float a = __shfl_sync(0xffffffffu, f0, n & 31), b = __shfl_sync(0xffffffffu, f1, n & 31);
          const int row = __shfl_sync(0xffffffffu, at, n & 31);
          float o = (has0 ? __uint_as_float(v0[e]) * a : 0.f) + (has1 ? __uint_as_float(v1[e]) * b : 0.f);
          if (n >= R || key >= D) continue;
          if (anynf) o += few_nonfinite<D, Q8>(p, sg, noted + par * 32, anc[n], d);
          if ((unused >> n) & 1u) o = 0.f;
          const long long i = (long long)row * D + d;
          if (whole) {
            if (in_bounds(row < p.B * p.N * p.H, p.status, kSiteTreeO)) p.o[i] = __float2half_rn(o);
          } else if (in_bounds(p.split && row < 2 * (int)gridDim.x * p.ws_rows, p.status, kSiteTreeWs)) {
            p.ws_o[i] = o;
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
    const int t = threadIdx.x - 12 * 32;        // 0 .. 32 PW - 1
    const int pw = warp - 12;
    // Q8_0: group pw / 4 decodes K (the first PG groups) or V tiles, those with
    // g % PG = turn: a group's waits and hand-overs, some 800 clocks a tile, pass
    // while the other works
    const int kv = Q8 ? pw / (4 * PG) : 1, turn = Q8 ? (pw >> 2) % PG : 0;
    const int R = p.N * p.G;
    const DecK K = make_deck();
    bool ok = true;
    int g = 0;
    uint32_t raw_ph = 0;                        // phase bits of v_raw of each stage, or of r_full of each slot
    Ring<KS> kr;
    Ring<VS> vr;
    Ring<RS> rr;
    if (Q8 && kv) rr.step();
    for (int w = 0; ok && tree_next(p, sched, walk, sg); ++w) {
      const int jm = first_masked(sg);
      ok = __all_sync(0xffffffffu, w == 0 || mbar_wait_idle(q_empty, (w - 1) & 1, run_ctl, 64));
      if (!ok) break;
      // notes of this warp's 32 rows, by masked tile (the V groups')
      uint32_t* nt = noted + (w & 1) * 32 + (4 * turn + (pw & 3)) * 4;
      if (kv == 1 && lane < 4) {
        nt[lane] = 0u;
        if (PG == 1) nt[16 + lane] = 0u;
      }
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
            for (int i = 0; i < 4; ++i) q[i] = __ldcg(src + i);   // (by way of L1: 97.0 us against 95.5 for the 32 tokens)
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
      const long long head = (long long)(p.b0 + sg.b) * p.Hkv + sg.hk;
      for (int j = sg.k0; j < sg.k1 && ok; ++j, ++g, kr.step(), vr.step()) {
        const int ks = kr.at, vs = vr.at;
        if constexpr (Q8) {
          const int rs = rr.at;
          const uint32_t rph = (raw_ph >> rs) & 1u;   // of the slot's barrier for this kind of tile
          raw_ph ^= 1u << rs;
          rr.step();   // K and V tiles alternate in the raw ring
          rr.step();
          if (PG > 1 && (g & 1) != turn) continue;
          const int sh = (int)(((head * p.C + (long long)j * kTile) * Cfg::kRow) & 15);
          // The stage first: with two groups of a kind the slot's last tile is the other
          // group's, and was decoded before the stage's last tile was read (few_groups_ok),
          // so that the parity can only mean this tile.  One group waits for every tile
          // that lands on its kind's barrier of the slot.
          bool go = true;
          if (kv == 0 ? g >= KS : g >= VS) go = mbar_wait(kv ? &v_empty[vs] : &k_empty[ks], (kv ? vr.ph : kr.ph) ^ 1u, ctl);
          go = go && mbar_wait(&r_full[few_raw_bar(Cfg::kRS, kv, rs)], rph, ctl);
          ok = __all_sync(0xffffffffu, go);
          if (!ok) break;
          const uint8_t* src = raws + rs * Cfg::kRaw + sh;
          const int row = t & 127;
          if (kv == 0) {
            // K: to the lanes and columns of its TMEM stage (warp % 4 = 32-row group)
            tc_fence_after();
            const uint32_t kcol = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + Cfg::kKCol + ks * (D / 2);
            uint32_t v[16];
            decode_block<D, 0>(src, row, K, v);
            tmem_st16(kcol, v);
            decode_block<D, 1>(src, row, K, v);
            tmem_st16(kcol + 16, v);
            if constexpr (D == 128) {
              decode_block<D, 2>(src, row, K, v);
              tmem_st16(kcol + 32, v);
              decode_block<D, 3>(src, row, K, v);
              tmem_st16(kcol + 48, v);
            }
            mbar_arrive_warp(&r_empty[rs]);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive_warp(&k_full[ks]);
          } else {
            uint8_t* dst = vst + vs * Cfg::kTileBytes;
            decode_to_tile<D, 0>(dst, src, row, K);
            decode_to_tile<D, 1>(dst, src, row, K);
            if constexpr (D == 128) {
              decode_to_tile<D, 2>(dst, src, row, K);
              decode_to_tile<D, 3>(dst, src, row, K);
            }
            if (j >= jm) {
              const uint32_t bits = __ballot_sync(0xffffffffu, clean_chunks(dst, row, 0, D / 8));
              if (lane == 0) nt[j - jm] = bits & rows_in_use(p, sg, j * kTile + 32 * (pw & 3));
            }
            fence_proxy_async_smem();
            mbar_arrive_warp(&v_full[vs]);
            mbar_arrive_warp(&r_empty[rs]);
          }
        } else if (j >= jm) {
          ok = __all_sync(0xffffffffu, mbar_wait_idle(&v_raw[vs], (raw_ph >> vs) & 1, run_ctl, 64));
          if (!ok) break;
          raw_ph ^= 1u << vs;
          const uint32_t bits = __ballot_sync(0xffffffffu, clean_chunks(vst + vs * Cfg::kTileBytes, t, 0, D / 8));
          if (lane == 0) nt[j - jm] = bits & rows_in_use(p, sg, j * kTile + 32 * (pw & 3));
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

// Joins the pieces of the items that were cut: W warps a row, warp k taking pieces
// k, k + W, ..., a lane D / 32 values.
template <int D, int W>
__global__ void __launch_bounds__(256) few_join_kernel(const TreeParams p, int grid) {
  constexpr int kRows = 8 / W;       // rows a CTA
  constexpr int E = D / 32;          // values a lane
  __shared__ float red_o[8][D];
  __shared__ float2 red_ml[8];
  __shared__ int sums[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = warp % W;
  const unsigned blocks = (p.ws_rows + kRows - 1) / kRows;
  const unsigned item = blockIdx.x / blocks;
  const int row = (int)(blockIdx.x - item * blocks) * kRows + warp / W;
  const int b = (int)(item / p.Hkv), hk = (int)item - b * p.Hkv;
  const JoinSpan js = join_span(p, b, hk, grid, sums);
  pdl_wait();
  if (!js.cut) return;
  JoinSum<E> acc;
  acc.clear();
  bool unused = false;
  const bool live = row < p.ws_rows && row < p.N * p.G;
  if (live && in_bounds(js.c1 < (unsigned)grid && js.c0 <= js.c1, p.status, kSiteTreeWs)) {
#pragma unroll 4
    for (unsigned c = js.c0 + k; c <= js.c1; c += W) {
      const long long s = js.slot(c) * p.ws_rows + row;
      const float2 v = __ldcg(p.ws_ml + s);
      const float* src = p.ws_o + s * D + E * lane;
      float x[E];
      if constexpr (E == 4) {
        const float4 q = __ldcg(reinterpret_cast<const float4*>(src));
        x[0] = q.x; x[1] = q.y; x[2] = q.z; x[3] = q.w;
      } else {
        const float2 q = __ldcg(reinterpret_cast<const float2*>(src));
        x[0] = q.x; x[1] = q.y;
      }
      unused |= v.y == -1.f;
      acc.add(v.x, v.y, x);
    }
  }
  if constexpr (W > 1) {
    if (k > 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) red_o[warp][E * lane + e] = acc.o[e];
      if (lane == 0) red_ml[warp] = make_float2(acc.m, unused ? -1.f : acc.l);
    }
    __syncthreads();
    if (k != 0) return;
#pragma unroll
    for (int i = 1; i < W; ++i) {
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = red_o[warp + i][E * lane + e];
      const float2 v = red_ml[warp + i];
      unused |= v.y == -1.f;
      acc.add(v.x, v.y, x);
    }
  }
  if (!live || !in_bounds(row / p.G < p.N, p.status, kSiteTreeO)) return;
  const float inv = acc.l > 0.f ? 1.f / acc.l : acc.l;
  __half* orow = p.o + ((long long)b * p.N + row / p.G) * p.H * D + (long long)(hk * p.G + row % p.G) * D + E * lane;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__half2*>(orow + e) =
        unused ? __floats2half2_rn(0.f, 0.f) : __floats2half2_rn(acc.o[e] * inv, acc.o[e + 1] * inv);
}

template <int D, bool Q8, int NC>
cudaError_t launch_few(const TreeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int grid,
                       cudaStream_t s) {
  using Cfg = FewCfg<D, Q8, NC>;
  auto kern = few_kernel<D, Q8, NC>;
  cudaError_t e = allow_smem<std::integer_sequence<int, 6, D, Q8, NC>>(kern, Cfg::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_tree_kernel(kern, (unsigned)grid, Cfg::kThreads, Cfg::kSmem, s, tm_k, tm_v, p);
  if (e != cudaSuccess || !p.split) return e;
  // Warps a row by the pieces that an item is likely to have.
  const long long items = (long long)p.B * p.Hkv;
  if (grid >= 24 * items)
    return launch_tree_kernel(few_join_kernel<D, 8>, (unsigned)(items * p.ws_rows), 256, 0, s, p, grid);
  if (grid >= 6 * items)
    return launch_tree_kernel(few_join_kernel<D, 4>, (unsigned)(items * ((p.ws_rows + 1) / 2)), 256, 0, s, p, grid);
  return launch_tree_kernel(few_join_kernel<D, 1>, (unsigned)(items * ((p.ws_rows + 7) / 8)), 256, 0, s, p, grid);
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
