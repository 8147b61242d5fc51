// attention_tree.cu -- attention of drafted trees of tokens (or of single new
// tokens, trees of one node) over a batch of KV caches, fp16 or Q8_0, on the
// tcgen05 tensor cores.
//
//   O_i = sum_j softmax_j(scale Q_i . K_j) V_j
// over the keys j < past[b] and, at rows past[b] + a, node i's ancestors a and
// itself.  The lengths and the trees are read on the device, so that a captured
// call follows them.
//
// Work.  The rows of one (sequence, KV head) are its N nodes times the G query
// heads of the group, r = i G + g; an item is 128 of them, and its work is a
// walk over tiles of 128 keys.  The tiles of all items of the call form one
// sequence, cut into equal runs, one for each persistent CTA (one an SM): a
// ragged batch loads every SM alike whatever its lengths.  A run that covers a
// whole item writes its output; pieces of an item go to the workspace as
// (O, max, sum) and a second kernel joins them.  Without a workspace the CTAs
// take whole items.
//
// A decode step reads each key once for few rows, so HBM should bound it: per
// SM 23 bytes a clock, i.e. a tile of 128 fp16 keys (K and V, D = 128, 64 KB)
// in about 2800 clocks and one of Q8_0 in 1500.  A 128-row tcgen05 tile pair
// (S = Q K^T and O += P V) takes about 1000, whatever part of its rows is used.
// Items of at most 32 rows go to attention_few.cu.  (Pairs of row tiles that share
// each copied and decoded key tile, for more than 128 rows, took 86 us against 74
// for 256 rows over 32K Q8_0 keys: both teams then wait for the same tile.)
//
// Measured: 8 sequences of 24 nodes, 4 heads a group, D = 64, over 1,000 to 8,100
// fp16 keys in 32.9 us (75.6 MB: 2.3 TB/s), one of 64 nodes, D = 128, over 32,500
// Q8_0 keys in 56.2 us (34 GFLOP: 607 TFLOP/s).  Long calls, the 8 sequences over
// 32,000 to 32,700 keys: fp16 in 171 us at D = 128 (1.06 GB: 6.2 TB/s) and 115 at D =
// 64 (4.6 TB/s), Q8_0 in 168 and 129 (3.3 and 2.2 TB/s).  All but the first of these
// are bound by a team's chain of a tile (scores 650 to 950 clocks, maxima 500,
// exponentials 1300, hand-over 350, P V 700); short calls by the start (schedule, Q: 3
// us), the end of a run (2 us) and the join (3 us).  (Q8_0 at D = 128 spills 44 bytes a
// thread at 72 registers.)
//
// TMEM holds two O and, at D = 64, three score buffers: a team's next scores are
// formed in the third while it works on the last ones, off its chain (1.10 to 0.91
// us a tile).  At D = 128 there are two, one a team, whose P lies over its S.
//
// Warps (fp16 768 threads, Q8_0 896):
//   0, 1    one lane each issues the MMAs of tile team 0 or 1 (tiles of even
//           and odd number): S into the team's TMEM buffer, then, when the
//           softmax has put P over it, O_team += P V;
//   2, 3    copies: fp16 caches by TMA into the swizzled K (warp 2) and V
//           (warp 3) stages; Q8_0 rows as they lie (warp 2, 1-D bulk copies)
//           into a raw ring;
//   4-19    softmax, one team of eight warps a tile parity, two threads a row,
//           keys 0-63 and 64-127: the row's maximum (exchanged through shared
//           memory), P = 2^(s - m) against a reference m that is raised only
//           when the maximum passes it by 2^8 (O is then rescaled in TMEM),
//           fp32 row sums, P rounded to fp16, the type of the MMA with V (2^-11 of
//           each weight: 2.9e-4 of the result against 2.1e-4 when only that is
//           rounded) (one thread a row: 37.7 us against 35.9 for the first case above
//           as it then was);
//   20-     per run: Q into swizzled shared memory; Q8_0: four warps decode each
//           raw K tile and four each V tile to fp16 (RNE(q d), the weights'
//           exact decode) in the swizzled stages; in tiles that hold keys which
//           some row does not see, non-finite V values are replaced by zero and
//           noted.
// The two teams have their own O and reference, so the only ties between them
// are the shared K/V stages; they are joined when a run of an item ends.  (A team
// held half a tile behind the other, so that their exponentials do not meet: 35.3
// against 35.7 and 55.4 against 55.3 us.)
//
// Masks.  Tiles below past[b] have none.  In the others each row has 128
// visibility bits, from its ancestors' bits; scores of unseen keys are replaced
// before the maximum and their P is zero.  P = 0 does not silence a NaN or an
// infinity in V (0 x inf), hence the replacement above; where a row does see
// such a value it is added to the row's result at the end.
//
// Every wait is bounded in time; on expiry the CTA records the failure in the
// status word and returns.
#include <algorithm>

#include "tree_common.cuh"
#include "tree_rings.h"

namespace m4q {

namespace {

constexpr int kSoft = 16;   // softmax warps

template <int D, bool Q8>
struct TreeCfg {
  static constexpr int kRow = Q8 ? D / 32 * 34 : 2 * D;
  static constexpr int kTileBytes = kTile * D * 2;     // an fp16 tile: D / 64 panels of [128][128 B]
  static constexpr RowsRings kRings = rows_rings(D, Q8);
  static constexpr int kKS = kRings.ks;
  static constexpr int kVS = kRings.vs;
  static constexpr int kRS = kRings.rs;                // raw ring (K, V, K, ...)
  static constexpr int kRaw = kTile * kRow + 32;       // a tile, its 16-byte shift, and the decode's overread
  static constexpr int kPrep = Q8 ? 8 : 4;             // preparing warps
  static constexpr int kThreads = 32 * (4 + kSoft + kPrep);
  static constexpr int kSB = kRings.sb;                // score buffers
  static constexpr int kBars = 3 * kKS + 4 * kVS + 3 * kRS + 17;
  static constexpr int kFixed = 8 * kTile * 4          // ancestor bits [8][128]
                                + (4 * rows_max_slots(kSB) + 2) * kTile * 4   // maxima [slot][team][half][128], sums [team][128]
                                + 2 * 2 * kTile * 8    // (m, l) [parity][team][128]
                                + 256 * 2              // parents
                                + 2 * 8 * 4 * 4        // noted V rows [parity][warp][masked tile]
                                + (int)sizeof(TreeSched) + 8
                                + kBars * 8 + 16;
  static constexpr int kSmem =
      1024 + (1 + kKS + kVS) * kTileBytes + kRS * kRaw + kFixed;
  static constexpr uint32_t kOCol = 128 * kSB;         // O of team t at kOCol + t D, S/P buffers at 128 i
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kRaw % 16 == 0, "bulk copy alignment");
};

// Non-finite values of the V rows that were cleared and that this row sees,
// added to its columns c0 .. c0 + 15 (Q8_0: positions of a decoded row).
template <int D, bool Q8>
__device__ __noinline__ void add_nonfinite(const TreeParams& p, Seg g, const uint32_t* noted,
                                           const uint32_t* anc, int c0, float (&x)[16]) {
  const int jm = first_masked(g);
#pragma unroll 1
  for (int mt = 0; mt < 4; ++mt) {
    const int j = jm + mt;
    if (j < g.k0 || j >= g.k1) continue;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      const int kq = j * kTile + 32 * q;
      add_values<D, Q8>(p, g, kq, (noted[4 * q + mt] | noted[4 * (q + 4) + mt]) & seen32<8>(anc, kTile, kq, g.past, p.C),
                        c0, x);
    }
  }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(TreeCfg<D, Q8>::kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const TreeParams p) {
  using Cfg = TreeCfg<D, Q8>;
  constexpr int SB = Cfg::kSB, PW = Cfg::kPrep, KS = Cfg::kKS, VS = Cfg::kVS, RS = Cfg::kRS > 0 ? Cfg::kRS : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qs = smem_align<1024>(smem_raw);
  uint8_t* kst = qs + Cfg::kTileBytes;
  uint8_t* vst = kst + KS * Cfg::kTileBytes;
  uint8_t* raws = vst + VS * Cfg::kTileBytes;
  uint32_t* anc_all = reinterpret_cast<uint32_t*>(raws + Cfg::kRS * Cfg::kRaw);   // [8][128]
  float* xmax = reinterpret_cast<float*>(anc_all + 8 * kTile);                    // [slot][team][half][128]
  float* xsum = xmax + 4 * rows_max_slots(SB) * kTile;                            // [team][128]
  float2* ml = reinterpret_cast<float2*>(xsum + 2 * kTile);                       // [parity][team][128]
  uint32_t* noted = reinterpret_cast<uint32_t*>(ml + 4 * kTile);                  // [parity][8 warps][4]
  // parents of the run's tree: its writers, one warp for 32 rows, write the same,
  // and none is a run ahead of another (ml_rdy)
  int16_t* up = reinterpret_cast<int16_t*>(noted + 64);                           // [256]
  TreeSched* sched = reinterpret_cast<TreeSched*>(up + 256);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sched) +
                                                  (sizeof(TreeSched) + 7) / 8 * 8);   // [team][KS] K of a tile in its stage
  uint64_t* k_empty = k_full + 2 * KS; // [KS] S done with it
  uint64_t* v_full = k_empty + KS;     // [VS] V of a tile in its stage
  uint64_t* v_raw = v_full + VS;       // [VS] (fp16) V of a masked tile, not yet cleared (v_full: the others')
  uint64_t* v_clean = v_raw + VS;      // [VS] (fp16) V of a masked tile, cleared
  uint64_t* v_empty = v_clean + VS;    // [VS] P V done with it
  uint64_t* r_full = v_empty + VS;     // [2][RS] raw tile (K, V) landed in a slot
  uint64_t* r_empty = r_full + 2 * Cfg::kRS;
  uint64_t* s_full = r_empty + Cfg::kRS;   // [team][2] S of the team's tile n (n % 2) in TMEM
  uint64_t* p_full = s_full + 4;       // [team][2] its P written
  uint64_t* pv_done = p_full + 4;      // [SB] P V of a buffer's tile done
  uint64_t* q_full = pv_done + 3;      // Q of a run written
  uint64_t* q_empty = q_full + 1;      // both teams' S of a run done
  uint64_t* ml_rdy = q_empty + 1;      // softmax: (m, l) of a run written
  uint64_t* nf_rdy = ml_rdy + 1;       // preparation of a run's tiles done (noted rows final)
  uint64_t* o_free = nf_rdy + 1;       // softmax: O of a run read out
  uint64_t* drain = o_free + 1;        // both issuers: every MMA complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[rows_k_bar(KS, 0, i)], Q8 ? 4 : 1);
      mbar_init(&k_full[rows_k_bar(KS, 1, i)], Q8 ? 4 : 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&v_full[i], Q8 ? 4 : 1);
      mbar_init(&v_raw[i], 1);
      mbar_init(&v_clean[i], PW);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < Cfg::kRS; ++i) {
      mbar_init(&r_full[i], 1);
      mbar_init(&r_full[Cfg::kRS + i], 1);
      mbar_init(&r_empty[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&pv_done[i], 1);
    mbar_init(q_full, PW);
    mbar_init(q_empty, 2);
    mbar_init(ml_rdy, 8);
    mbar_init(nf_rdy, PW);
    mbar_init(o_free, kSoft);
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
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
  // a wait that may last a whole run (a million keys take about 10 ms); it ends
  // at once when another wait gives up
  const WaitCtl run_ctl{abort_flag, p.status, 30000000000ull};
  TreeWalk walk = tree_begin(sched);
  Seg sg;

  if (warp < 2) {
    // ------------------------------------------------------------ MMA issuers
    if (lane == 0) {
      const int team = warp;
      constexpr uint32_t idesc_s = idesc_f16_f32(128, kTile);
      constexpr uint32_t idesc_o = idesc_f16_f32(128, D) | (1u << 16);   // B (V) N-major
      const uint64_t qd = sdesc_sw128_kmajor(smem_u32(qs));
      const uint64_t kd = sdesc_sw128_kmajor(smem_u32(kst));
      const uint64_t vd = sdesc_sw128_nmajor(smem_u32(vst), kTile * 128);
      const uint32_t ocol = tmem + Cfg::kOCol + D * team;
      uint32_t k_ph = 0, full_ph = 0, clean_ph = 0;   // phase bits of the team's k_full, of v_full and v_clean
      bool ok = true;
      int g = 0;                  // tiles of the CTA
      Ring<KS> kr;
      Ring<VS> vr;
      for (int w = 0; ok && tree_next(p, sched, walk, sg); ++w) {
        const int jm = first_masked(sg);
        // The team's next tile of the run: its stages and barriers.  Looked up while
        // the softmax has the last one: after P V it would cost 500 to 700 clocks of
        // a chain of 5000.
        struct Tile {
          int x, ks, vs;              // number in the CTA, stages
          uint32_t k_ph, v_ph;
          uint64_t* v_ready;
        };
        Tile at{};
        int j = sg.k0;
        auto look = [&]() {
          for (; j < sg.k1;) {
            const bool wants_clean = !Q8 && j >= jm, mine = (g & 1) == team;
            at.x = g;
            at.ks = kr.at;
            at.k_ph = (k_ph >> kr.at) & 1u;
            if (mine) k_ph ^= 1u << kr.at;
            at.vs = vr.at;
            at.v_ready = wants_clean ? &v_clean[vr.at] : &v_full[vr.at];
            at.v_ph = ((wants_clean ? clean_ph : full_ph) >> vr.at) & 1u;
            (wants_clean ? clean_ph : full_ph) ^= 1u << vr.at;
            ++j, ++g;
            kr.step();
            vr.step();
            if (mine) return true;
          }
          return false;
        };
        // P V of tile x done (its buffer's x / SB-th use)
        auto pv_wait = [&](int x) { return x < 0 || mbar_wait(&pv_done[x % SB], (x / SB) & 1, ctl); };
        // S of the tile looked up, into its buffer, which is free
        auto scores = [&]() {
          if (!mbar_wait(&k_full[rows_k_bar(KS, team, at.ks)], at.k_ph, ctl)) return false;
          tc_fence_after();
          const uint64_t kds = kd + (uint64_t)(at.ks * (Cfg::kTileBytes >> 4));
          const uint32_t scol = tmem + 128 * (at.x % SB);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * (kTile * 128 >> 4) + 2 * (kk & 3);
            mma_ss_f16(scol, qd + off, kds + off, idesc_s, kk > 0 ? 1u : 0u);
          }
          tc_commit(&s_full[2 * team + ((at.x >> 1) & 1)]);
          tc_commit(&k_empty[at.ks]);
          return true;
        };
        bool first = true, more = look();
        ok = mbar_wait(q_full, w & 1, ctl);
        if (ok && !more) tc_commit(q_empty);
        if (ok && more && SB == 3) ok = pv_wait(at.x - 3) && scores();
        while (ok && more) {
          if (SB == 2) {
            ok = pv_wait(at.x - 2) && scores();
            if (!ok) break;
          }
          const Tile now = at;
          more = look();
          if constexpr (SB == 3) {
            // The next scores, a tile ahead, into the buffer of the other team's last
            // tile.  Waited for without a next tile too: P V of all tiles go in order,
            // so that no barrier is ever two phases past a wait for it.
            ok = pv_wait(now.x - 1) && (!more || scores());
            if (!ok) break;
          }
          if (!more) tc_commit(q_empty);   // this team's S of the run are done with Q
          ok = mbar_wait(now.v_ready, now.v_ph, ctl);
          if (first && w > 0) ok = ok && mbar_wait(o_free, (w - 1) & 1, ctl);
          ok = ok && mbar_wait(&p_full[2 * team + ((now.x >> 1) & 1)], (now.x >> 2) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vds = vd + (uint64_t)(now.vs * (Cfg::kTileBytes >> 4));
          const uint32_t scol = tmem + 128 * (now.x % SB);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            tc_mma_ts_f16(ocol, scol + 64 * (kk >> 2) + 8 * (kk & 3), vds + (uint32_t)(kk * (2048 >> 4)), idesc_o,
                          (kk > 0 || !first) ? 1u : 0u);
          tc_commit(&pv_done[now.x % SB]);
          tc_commit(&v_empty[now.vs]);
          first = false;
        }
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
              uint64_t* bar = &full[kv * RS + sl];
              full_ph ^= 1u << (kv * RS + sl);
              mbar_arrive_expect_tx(bar, bytes);
              if (in_bounds(at >= 0 && bytes > 0 && bytes <= (uint32_t)Cfg::kRaw &&
                                at + bytes <= (long long)p.B_all * p.Hkv * p.C * Cfg::kRow,
                            p.status, kSiteTreeKV))
                bulk_load(ring + sl * Cfg::kRaw, (kv ? p.v : p.k) + at, bytes, bar);
            } else {
              // V of a masked tile goes by way of the clearing warps
              const bool raw = warp == 3 && j >= jm;
              const int fb = warp == 2 ? rows_k_bar(KS, n & 1, sl) : sl;
              uint64_t* bar = raw ? &v_raw[sl] : &full[fb];
              (raw ? raw_ph : full_ph) ^= 1u << (raw ? sl : fb);
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
        for (int i = 0; i < (Q8 || warp == 2 ? 2 * ns : ns); ++i) {
          mbar_wait_drain(&full[i], ((full_ph >> i) & 1) ^ 1, 100000000ull);
          if (!Q8 && warp == 3) mbar_wait_drain(&v_raw[i], ((raw_ph >> i) & 1) ^ 1, 100000000ull);
        }
    }
    __syncwarp();
  } else if (warp < 4 + kSoft) {
    // ------------------------------------------------------------ softmax
    const int team = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, quad = warp & 3;
    const int r = 32 * quad + lane;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t scol0 = tmem + lanes + 64 * half;                           // buffer 0: its 64 keys' scores, then P
    const uint32_t ocol = tmem + lanes + Cfg::kOCol + D * team + D / 2 * half;   // the columns it rescales
    uint32_t* anc = anc_all + r;   // this row's bits: word i at anc[128 i]
    // named barriers: the four warps of these rows, and the two of a team
    const uint32_t quad_bar = 1 + quad, pair_bar = 5 + 4 * team + quad;
    float* mine = xmax + (2 * team + half) * kTile + r;
    const float* others = xmax + (2 * team + 1 - half) * kTile + r;
    // positive: a negative scale turns Q's signs, and a scale of zero is one that
    // no score survives (an unseen key's -inf has to stay -inf)
    const float sc = fmaxf(fabsf(p.scale_log2), 1e-37f);
    const int R = p.N * p.G;
    bool ok = true;
    int g = 0;                                  // tiles of the CTA
    bool fresh = true;                          // the CTA's first run
    for (int w = 0; ok && tree_next(p, sched, walk, sg); ++w) {
      const int row = sg.rt * kTile + r;
      const bool valid = row < R;
      const bool busy = sg.rt * kTile + 32 * quad < R;   // the warp has a row
      const int node = valid ? row / p.G : 0;
      const int jm = first_masked(sg);
      bool used = true;
      if (busy && sg.k1 > jm) {
        named_bar_sync(quad_bar, 128);   // the last run's readers are done
        if (warp < 8) ancestors256(p.parents + (long long)sg.b * p.N, p.N, up, node, anc, kTile);
        named_bar_sync(quad_bar, 128);
        used = (anc[(node >> 5) * kTile] >> (node & 31)) & 1u;   // a used node sees itself
      }
      float m = -INFINITY, l = 0.f;
      bool first = true;
      for (int j = sg.k0; j < sg.k1; ++j, ++g) {
        if ((g & 1) != team) continue;
        const int sp = 2 * team + ((g >> 1) & 1);
        const uint32_t ph = (g >> 2) & 1, scol = scol0 + 128 * (g % SB);
        // warps without a row stay out of the others' way while they wait
        ok = __all_sync(0xffffffffu, busy ? mbar_wait(&s_full[sp], ph, ctl)
                                          : mbar_wait_idle(&s_full[sp], ph, ctl, 256));
        if (!busy) {
          if (!ok) break;
          mbar_arrive_warp(&p_full[sp]);
          continue;
        }
        tc_fence_after();
        float t = -INFINITY;   // the half row's largest raw score
        if (ok) {
          if (j >= jm) {
            // scores of unseen keys, whatever they are, become -inf
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t vis =
                  seen32<8>(anc, kTile, j * kTile + 64 * half + 32 * (c >> 1), sg.past, p.C) >> (16 * (c & 1));
              if (__all_sync(0xffffffffu, (vis & 0xFFFFu) == 0xFFFFu)) continue;
              uint32_t v[16];
              tmem_ld16_wait(scol + 16 * c, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = (vis >> e) & 1u ? v[e] : 0xFF800000u;
              tmem_st16(scol + 16 * c, v);
            }
            tmem_wait_st();
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t v[32];
            tmem_ld32_wait(scol + 32 * q, v);
            float x[4] = {t, t, t, t};
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e & 3] = fmaxf(x[e & 3], __uint_as_float(v[e]));
            t = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
          }
          mine[4 * kTile * rows_max_slot(SB, g)] = t;
        }
        // the two halves go on, or leave, together (a named barrier has no time limit)
        if (vote_or(pair_bar, 64, !ok)) {
          ok = false;
          break;
        }
        t = fmaxf(t, others[4 * kTile * rows_max_slot(SB, g)]);
        // the tile's maximum; -inf when the row sees no key of it
        const float mu = t == INFINITY ? -INFINITY : t * sc;   // (an infinite score gives NaN in the end)
        const float mj = mu > m + kRaise || m == -INFINITY ? fmaxf(mu, m) : m;
        const bool raise = mj > m && !first && m != -INFINITY;
        if (__any_sync(0xffffffffu, raise)) {
          // the team's last P V is done (with two buffers S has waited for it; with
          // three, PV of the buffer's next tile comes after this tile's)
          if (SB == 3) {
            mbar_wait(&pv_done[(g - 2) % SB], ((g - 2) / SB) & 1, ctl);
            __syncwarp();
            tc_fence_after();
          }
          const float a = raise ? ex2(m - mj) : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[16];
            tmem_ld16_wait(ocol + 16 * c, v);
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = __float_as_uint(__uint_as_float(v[q]) * a);
            tmem_st16(ocol + 16 * c, v);
          }
        }
        if (mj != m) l *= m == -INFINITY ? 0.f : ex2(m - mj);
        m = mj;
        const float muse = mj == -INFINITY ? 0.f : mj;
        const unsigned long long sc2 = pack2(sc, sc), nm2 = pack2(-muse, -muse);
        unsigned long long s2 = 0ull;
        // chunks of 16 keys, the next load in flight; P of keys 16 c .. + 15 to
        // columns 8 c .. + 7, whose scores have been read
        uint32_t v[2][16];
        tmem_ld16_async(scol, v[0]);
        tmem_wait_ld_tied(v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c < 3) tmem_ld16_async(scol + 16 * (c + 1), v[(c + 1) & 1]);
          const uint32_t (&x)[16] = v[c & 1];
          uint32_t wv[8];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float a0, a1;
            unpack2(fma2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), sc2, nm2), a0, a1);
            const float p0 = ex2(a0), p1 = ex2(a1);
            s2 = add2(s2, pack2(p0, p1));
            const __half2 hh = __floats2half2_rn(p0, p1);
            wv[e >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          tmem_st8(scol + 8 * c, wv);
          if (c < 3) tmem_wait_ld_tied(v[(c + 1) & 1]);
        }
        float sum0, sum1;
        unpack2(s2, sum0, sum1);
        l += sum0 + sum1;
        first = false;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(&p_full[sp]);
      }
      // ---------------------------------------------------------- end of a run
      const int par = w & 1;
      if (half) xsum[team * kTile + r] = l;
      named_bar_sync(pair_bar, 64);
      if (!half) {
        ml[(par * 2 + team) * kTile + r] = make_float2(m, l + xsum[team * kTile + r]);
        if (ok) mbar_arrive_warp(ml_rdy);
      }
      const int g0 = g - (sg.k1 - sg.k0);
      bool got = ok && mbar_wait(ml_rdy, par, ctl) && mbar_wait(nf_rdy, par, ctl);
      // (of three buffers the last tile's: P V go in order)
      got = got && mbar_wait(&pv_done[(g - 1) % SB], ((g - 1) / SB) & 1, ctl);
      if (SB == 2 && g > 1) got = got && mbar_wait(&pv_done[(g - 2) % SB], ((g - 2) / SB) & 1, ctl);
      ok = !vote_or(quad_bar, 128, !got);
      if (!ok) break;
      tc_fence_after();
      if (busy) {
        // tiles of this run by team (a team without one has no O)
        const bool has0 = sg.k1 - sg.k0 > 1 || !(g0 & 1), has1 = sg.k1 - sg.k0 > 1 || (g0 & 1);
        const float2 a = ml[(par * 2 + 0) * kTile + r], b = ml[(par * 2 + 1) * kTile + r];
        const float M = fmaxf(a.x, b.x);
        const float w0 = a.x == M ? 1.f : ex2(a.x - M), w1 = b.x == M ? 1.f : ex2(b.x - M);
        const float L = a.y * w0 + b.y * w1;
        const bool whole = sg.k0 == 0 && sg.k1 == sg.nk;
        // a whole item is divided by its sum (a row without a key is zero)
        const float inv = !whole ? 1.f : L > 0.f ? 1.f / L : L;
        const float f0 = w0 * inv, f1 = w1 * inv;
        const uint32_t* nt = noted + par * 32;
        const bool anynf = sg.k1 > jm && __any_sync(0xffffffffu, nt[lane] != 0u);
        const bool head_ok = in_bounds(node < p.N, p.status, kSiteTreeO);
        __half* orow = p.o + ((long long)sg.b * p.N + node) * p.H * D +
                       (long long)(sg.hk * p.G + (valid ? row % p.G : 0)) * D;
        const long long slot = 2ll * blockIdx.x + (fresh ? 0 : 1);
        const bool store = valid && head_ok;
        const bool ws_ok = in_bounds(whole || !valid || (p.split && r < p.ws_rows), p.status, kSiteTreeWs);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          const int col = (2 * team + half) * (D / 4) + 16 * c;
          uint32_t v0[16], v1[16];
          tmem_ld16_wait(tmem + lanes + Cfg::kOCol + col, v0);
          tmem_ld16_wait(tmem + lanes + Cfg::kOCol + D + col, v1);
          float x[16];
#pragma unroll
          for (int q = 0; q < 16; ++q)
            x[q] = (has0 ? __uint_as_float(v0[q]) * f0 : 0.f) + (has1 ? __uint_as_float(v1[q]) * f1 : 0.f);
          if (anynf) {
            if (valid && used) {   // (a copy: an array whose address is taken lives in memory)
              float y[16];
#pragma unroll
              for (int q = 0; q < 16; ++q) y[q] = x[q];
              add_nonfinite<D, Q8>(p, sg, nt, anc, col, y);
#pragma unroll
              for (int q = 0; q < 16; ++q) x[q] = y[q];
            }
            __syncwarp();
          }
          if (store && ws_ok) {
            if (!used) {
#pragma unroll
              for (int q = 0; q < 16; ++q) x[q] = 0.f;
            }
            if (whole) {
              store_columns<D, Q8>(x, col, orow);
            } else {   // [column / 4][row][4]: neighbouring lanes, neighbouring rows
              float4* piece = reinterpret_cast<float4*>(p.ws_o) + (slot * (D / 4) + col / 4) * p.ws_rows + r;
#pragma unroll
              for (int q = 0; q < 4; ++q)
                piece[q * p.ws_rows] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            }
          }
        }
        // the piece that holds the tree tells of an unused node by a sum of -1
        if (!whole && store && ws_ok && team == 0 && half == 0) p.ws_ml[slot * p.ws_rows + r] = make_float2(M, used ? L : -1.f);
      }
      fresh = false;
      tc_fence_before();
      mbar_arrive_warp(o_free);
    }
  } else {
    // ------------------------------------------------------------ Q, decode, clearing
    const int t = threadIdx.x - 32 * (4 + kSoft);   // 0 .. 32 PW - 1
    const int pw = warp - 4 - kSoft;
    const int R = p.N * p.G;
    const DecK K = make_deck();
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    bool ok = true;
    int g = 0;
    // Q8_0: the first four warps decode K tiles, the others V tiles: the waits of one pass while
    // the other works
    const int kv = pw >> 2;
    uint32_t raw_ph = 0;                        // phase bits of v_raw, or of r_full, of each stage
    for (int w = 0; ok && tree_next(p, sched, walk, sg); ++w) {
      const int jm = first_masked(sg);
      ok = __all_sync(0xffffffffu, w == 0 || mbar_wait_idle(q_empty, (w - 1) & 1, run_ctl, 64));
      if (!ok) break;
      uint32_t* nt = noted + (w & 1) * 32 + pw * 4;
      if (lane < 4) {
        nt[lane] = 0u;
        if (PW == 4) nt[16 + lane] = 0u;
      }
      __syncwarp();
      // Q rows (Q8_0: in the decoded blocks' order), a block of 32 values a step
#pragma unroll
      for (int i = 0; i < kTile * (D / 32) / (32 * PW); ++i) {
        const int u = t + 32 * PW * i, rr = u / (D / 32), blk = u % (D / 32);
        const int row = sg.rt * kTile + rr;
        uint4 q[4] = {}, o[4];
        if (row < R) {
          const int node = row / p.G, h = sg.hk * p.G + row % p.G;
          if (in_bounds(node < p.N && h < p.H, p.status, kSiteTreeQ)) {
            const uint4* src =
                reinterpret_cast<const uint4*>(p.q + ((long long)h * p.q_rows + (long long)sg.b * p.N + node) * D) + 4 * blk;
#pragma unroll
            for (int c = 0; c < 4; ++c) q[c] = src[c];   // (not by way of L1: 33.5 us against 32.9 for the first case above)
          }
        }
        if constexpr (Q8) order_block(q, blk & 1, o);
        else
#pragma unroll
          for (int c = 0; c < 4; ++c) o[c] = q[c];
#pragma unroll
        for (int c = 0; c < 4; ++c) {   // signs of a negative scale
          o[c].x ^= flip;
          o[c].y ^= flip;
          o[c].z ^= flip;
          o[c].w ^= flip;
        }
        uint8_t* base = qs + (blk >> 1) * (kTile * 128) + rr * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(base + (((4 * (blk & 1) + c) ^ (rr & 7)) << 4)) = o[c];
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(q_full);
      const long long head = (long long)(p.b0 + sg.b) * p.Hkv + sg.hk;
      for (int j = sg.k0; j < sg.k1 && ok; ++j, ++g) {
        [[maybe_unused]] const int ks = g % KS, vs = g % VS;
        if constexpr (Q8) {
          const int n = 2 * g + kv, rs = n % RS;
          const int sh = (int)(((head * p.C + (long long)j * kTile) * Cfg::kRow) & 15);
          bool go = mbar_wait(&r_full[kv * RS + rs], (raw_ph >> rs) & 1, ctl);
          raw_ph ^= 1u << rs;
          const int st = kv ? vs : ks, ns = kv ? VS : KS;
          if (g >= ns) go = go && mbar_wait(kv ? &v_empty[st] : &k_empty[st], ((g / ns) - 1) & 1, ctl);
          ok = __all_sync(0xffffffffu, go);
          if (!ok) break;
          uint8_t* dst = (kv ? vst : kst) + st * Cfg::kTileBytes;
          const int row = t & 127;
          const uint8_t* src = raws + rs * Cfg::kRaw + sh;
          decode_to_tile<D, 0>(dst, src, row, K);
          decode_to_tile<D, 1>(dst, src, row, K);
          if constexpr (D == 128) {
            decode_to_tile<D, 2>(dst, src, row, K);
            decode_to_tile<D, 3>(dst, src, row, K);
          }
          if (kv && j >= jm) {
            const uint32_t bits = __ballot_sync(0xffffffffu, clean_chunks(dst, row, 0, D / 8));
            if (lane == 0) nt[j - jm] = bits & rows_in_use(p, sg, j * kTile + 32 * (pw & 3));
          }
          fence_proxy_async_smem();
          mbar_arrive_warp(kv ? &v_full[st] : &k_full[rows_k_bar(KS, g & 1, st)]);
          mbar_arrive_warp(&r_empty[rs]);
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
      if (ok && w >= 1) ok = __all_sync(0xffffffffu, mbar_wait_idle(o_free, (w - 1) & 1, ctl, 64));
      if (ok) mbar_arrive_warp(nf_rdy);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the items that were cut.  A CTA takes 32 rows (lanes) and
// 32 columns (warps: 4 each) of an item, a block of a decoded row, which goes to
// its own order on the way out; W groups of 8 warps share its pieces.
template <int D, bool Q8, int W>
__global__ void __launch_bounds__(256 * W) tree_join_kernel(const TreeParams p, int grid) {
  constexpr int kPitch = 40;   // halves
  __shared__ float4 red_o[W > 1 ? W - 1 : 1][256];
  __shared__ float2 red_ml[W > 1 ? W - 1 : 1][256];
  __shared__ __align__(16) __half out[32 * kPitch];
  __shared__ int sums[4];
  pdl_launch_dependents();
  const int t = threadIdx.x & 255, k = threadIdx.x >> 8, lane = t & 31, warp = t >> 5;
  const unsigned blocks = (p.ws_rows + 31) / 32 * (D / 32), hr = (unsigned)p.Hkv * p.rtiles;
  const unsigned item = blockIdx.x / blocks, part = blockIdx.x - item * blocks;
  const int blk = part % (D / 32), r0 = (int)(part / (D / 32)) * 32, r = r0 + lane;
  const int b = (int)(item / hr), sub = (int)(item - b * hr), hk = sub / p.rtiles, row0 = (sub - hk * p.rtiles) * kTile;
  const JoinSpan js = join_span(p, b, sub, grid, sums);
  pdl_wait();
  if (!js.cut) return;
  JoinSum<4> acc;
  acc.clear();
  bool unused = false;
  if (r < p.ws_rows && row0 + r < p.N * p.G && in_bounds(js.c1 < (unsigned)grid && js.c0 <= js.c1, p.status, kSiteTreeWs)) {
#pragma unroll 4
    for (unsigned c = js.c0 + k; c <= js.c1; c += W) {
      const long long s = js.slot(c);
      const float2 v = __ldcg(p.ws_ml + s * p.ws_rows + r);
      const float4 q = __ldcg(reinterpret_cast<const float4*>(p.ws_o) + (s * (D / 4) + 8 * blk + warp) * p.ws_rows + r);
      const float x[4] = {q.x, q.y, q.z, q.w};
      unused |= v.y == -1.f;
      acc.add(v.x, v.y, x);
    }
  }
  if constexpr (W > 1) {
    if (k > 0) {
      red_o[k - 1][t] = make_float4(acc.o[0], acc.o[1], acc.o[2], acc.o[3]);
      red_ml[k - 1][t] = make_float2(acc.m, unused ? -1.f : acc.l);
    }
    __syncthreads();
    if (k > 0) return;
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      const float4 q = red_o[i][t];
      const float2 v = red_ml[i][t];
      const float x[4] = {q.x, q.y, q.z, q.w};
      unused |= v.y == -1.f;
      acc.add(v.x, v.y, x);
    }
  }
  const float inv = unused ? 0.f : acc.l > 0.f ? 1.f / acc.l : acc.l;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int pos = 4 * warp + e;
    out[lane * kPitch + (Q8 ? q8_code_at(blk & 1, pos) : pos)] = __float2half_rn(unused ? 0.f : acc.o[e] * inv);
  }
  if constexpr (W > 1) named_bar_sync(1, 256);
  else __syncthreads();
  // 8 lanes a row, 8 bytes each
  const int rr = t >> 3, row = row0 + r0 + rr;
  if (r0 + rr >= p.ws_rows || row >= p.N * p.G) return;
  const int node = row / p.G;
  if (!in_bounds(node < p.N, p.status, kSiteTreeO)) return;
  __half* orow = p.o + ((long long)b * p.N + node) * p.H * D + (long long)(hk * p.G + row - node * p.G) * D;
  *reinterpret_cast<uint2*>(orow + 32 * blk + 4 * (t & 7)) = *reinterpret_cast<const uint2*>(out + rr * kPitch + 4 * (t & 7));
}

template <int D, bool Q8>
cudaError_t launch_tree(const TreeParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, int grid,
                        cudaStream_t s) {
  auto kern = tree_kernel<D, Q8>;
  cudaError_t e = allow_smem<std::integer_sequence<int, 5, D, Q8>>(kern, TreeCfg<D, Q8>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_tree_kernel(kern, (unsigned)grid, TreeCfg<D, Q8>::kThreads, TreeCfg<D, Q8>::kSmem, s, tm_k, tm_v, p);
  if (e != cudaSuccess || !p.split) return e;
  // Groups of warps by the pieces that an item is likely to have: with 10 of them
  // (2048 rows of 128) a call took 58.0 us with four groups and 61.4 with one, with
  // 2.4 (6144 rows of 64) 39.6 and 37.8.
  const long long items = (long long)p.B * p.Hkv * p.rtiles;
  const unsigned parts = (unsigned)(items * ((p.ws_rows + 31) / 32) * (D / 32));
  return grid > 4 * items ? launch_tree_kernel(tree_join_kernel<D, Q8, 4>, parts, 1024, 0, s, p, grid)
                          : launch_tree_kernel(tree_join_kernel<D, Q8, 1>, parts, 256, 0, s, p, grid);
}

}  // namespace

cudaError_t launch_attention_tree(const TreeParams& p, bool q8, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                  int grid, cudaStream_t s) {
  // few rows: keys on the MMA's 128 lanes instead of rows (a 128-row tile costs
  // the same for any of them)
  if (p.N * p.G <= kTreeFewRows) return launch_attention_few(p, q8, tm_k, tm_v, grid, s);
  if (p.D == 64) return q8 ? launch_tree<64, true>(p, tm_k, tm_v, grid, s) : launch_tree<64, false>(p, tm_k, tm_v, grid, s);
  return q8 ? launch_tree<128, true>(p, tm_k, tm_v, grid, s) : launch_tree<128, false>(p, tm_k, tm_v, grid, s);
}

}  // namespace m4q
