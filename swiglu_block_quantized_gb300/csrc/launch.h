// launch.h -- host-side interface between the C ABI (api.cu) and the kernel
// translation units.  No kernel code here.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include <atomic>
#include <utility>

namespace m4q {

// One projection launch, already validated by the ABI layer.
struct ProjLaunch {
  const void* x;          // fp16 [M, K]
  const void* w0;         // packed weights (gate for SwiGLU)
  const void* w1;         // up weights (SwiGLU) or null
  void* y;                // fp16 [M, N]
  int M, N, K;
  long long row_bytes;
  bool swiglu;            // gated projection (gate and up weights)
  int act;                // gate activation: 0 SiLU, 1 GELU
  int head_dim;           // GEMM output: 0 row-major [M, N], else head-major [N / head_dim][M][head_dim]
  bool wtma;              // packed rows are 16-byte multiples: weights move by TMA (a
                          // last stage past the row end is zero-filled)
  uint32_t* status;       // device status word
  unsigned long long limit_ns;
  cudaStream_t stream;
  // tcgen05 path
  int nx;                 // activation rows per tile: 64, 128 or 256
  bool small;             // M <= 128 kernel (activations as the A operand, tc_small.cuh)
  int split;              // CTAs of a cluster splitting K for one tile (1, 2, 4, 8); the launcher
                          // lowers it until all clusters of the grid can be co-resident
  int sms;                // multiprocessors (persistent grid size, both paths)
  CUtensorMap tm_x, tm_w0, tm_w1, tm_y;
  // GEMV path
  int mt;                 // 1 (M <= 8) or 2 (M <= 16)
};

// Per-kernel, per-device "dynamic shared memory attribute set" flags.  An
// anonymous namespace gives them internal linkage, so two copies of the
// library loaded into one process never share them.
namespace {
template <typename Tag>
std::atomic<unsigned long long>& attr_flag() {
  static std::atomic<unsigned long long> f{0};
  return f;
}
}  // namespace

// Programmatic dependent launch of the projection kernels (on unless the
// environment sets M4Q_PDL=0): a kernel may be scheduled while the previous
// kernel of the stream finishes; it waits for that kernel (griddepcontrol)
// before its first global access.
inline bool pdl_enabled() {
  static const bool on = [] {
    const char* v = getenv("M4Q_PDL");
    return !(v && v[0] == '0');
  }();
  return on;
}

// Launch `kern` with the projection kernels' attributes: programmatic
// dependent launch, and a cluster of `cluster` CTAs along x when > 1.
template <typename... KArgs, typename... Args>
cudaError_t launch_proj(void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                        unsigned cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

cudaError_t launch_tc_q4_0(const ProjLaunch& L);
cudaError_t launch_tc_q8_0(const ProjLaunch& L);
cudaError_t launch_tc_q2_0(const ProjLaunch& L);
cudaError_t launch_tc_mlx4(const ProjLaunch& L);
cudaError_t launch_gemv(int codec, const ProjLaunch& L);

// attention.cu: attention of fp16 Q [H][M][D] over a KV cache [Hkv][T] of
// rows of D values (fp16, or Q8_0 blocks along D); O fp16 [M][H * D].
struct AttnParams {
  const __half* q;
  const uint8_t* k;
  const uint8_t* v;
  __half* o;
  float* ws_o;            // key splits: unnormalised O [nsplit][Hkv][rtiles * 64][D]
  float2* ws_ml;          // key splits: (max, sum) per row, same order
  int H, Hkv, G, M, T, D;
  long long kv_row_bytes; // bytes of one key row (2 D, or D / 32 * 34)
  int q_offset;           // causal: query i sees keys j <= q_offset + i
  int causal;
  float scale_log2;       // softmax scale * log2(e)
  int rtiles;             // ceil(M * G / 64) row tiles per KV head
  int nsplit, tsplit;     // key splits and keys per split (a multiple of 64)
  bool kv_vec16;          // every K/V tile start and T * kv_row_bytes are 16-byte aligned
  uint32_t* status;       // device status word (bounds-checked build)
  int nsm;                // SMs of the device (persistent grids)
};
cudaError_t launch_attention(const AttnParams& p, bool q8, cudaStream_t s);
// attention_tc.cu: the tcgen05 kernel for prefill-sized calls on an fp16 cache
// (tm_q: 3-D tensor map [H][M][D] of Q, boxes of [1][128 / G queries][64 d];
// tm_k, tm_v: [Hkv][T][D] of the caches, boxes of [1][128 keys][64 d]; all
// with the 128-byte swizzle)
bool attention_tc_shape(const AttnParams& p);                // the kernel takes the shape
bool attention_tc_applies(const AttnParams& p, bool q8);     // and is estimated faster than the split kernel
// Q8_0 caches K and V ([rows][D / 32 blocks]) decoded to fp16 kf, vf
// ([rows][D]), for the tensor-core path
cudaError_t launch_kv_q8_stage(const void* k, const void* v, long long rows, int D, void* kf, void* vf,
                               cudaStream_t s);
cudaError_t launch_attention_tc(const AttnParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                const CUtensorMap& tm_v, cudaStream_t s);

// kv_ops.cu: rotary positions and the KV cache's rows (fp16, or Q8_0 blocks
// along D), D = 64 or 128.
struct RowsView {         // fp16 rows [heads][M] of D values, strides in elements
  const __half* p;
  long long hs, rs;
};
struct KvOpsParams {
  RowsView q, k, v;       // Q rows (H of them a token, may be 0), K and V rows (Hkv, may be 0)
  __half* qo;             // rotated Q, strides qo_hs, qo_rs
  long long qo_hs, qo_rs;
  int H, Hkv, M, D;
  const int32_t* pos;     // [M], or [A][M] with axes
  const int64_t* freqs;   // [rot / 2] turns per position in units of 2^-64, or null: no rotation
  const int32_t* axes;    // [rot / 2] the axis of each pair (outside [0, A): not turned), or null: one axis
  int A;
  int rot, interleaved;
  float mscale;
  const int32_t* slots;   // [M] cache row b C + j of each token; outside [0, B C): not written
  uint8_t* kc;            // caches [B][Hkv][C] rows
  uint8_t* vc;
  int B, C;
  uint32_t* status;
  int nsm;
};
cudaError_t launch_rope_kv(const KvOpsParams& p, bool q8, cudaStream_t s);
struct KvReadParams {
  const uint8_t* kc;      // caches [B][Hkv][C] rows; either may be null
  const uint8_t* vc;
  __half* ko;             // [Hkv][n][D]
  __half* vo;
  const int32_t* slots;   // [n]
  int B, Hkv, C, D, n;
  uint32_t* status;
};
cudaError_t launch_kv_read(const KvReadParams& p, bool q8, cudaStream_t s);

// norm.cu: residual update and the norms on both sides of a block, one row of
// D values (D % 8 == 0) a group of warps.
struct NormParams {
  const __half* h;        // block output [M][D], or null: the residual is only normalised
  const void* r;          // residual stream [M][D], fp16 or fp32
  const __half* w_post;   // [D] or null
  const __half* gate;     // [D], [M][D] (gate_rows), or null
  const __half* w_pre;    // [D] or null (then no y)
  void* r_out;            // null: not written
  __half* y;
  long long M;
  int D;
  int gate_rows;
  float res_scale, branch_scale, eps;
  uint32_t* status;
};
cudaError_t launch_norm_residual(const NormParams& p, bool res32, cudaStream_t s);

// attention_tree.cu: attention of N drafted nodes of each of B sequences over
// its cache [Hkv][C] rows of D values.  One launch takes up to kTreeSeqs
// sequences (their tile counts stay in shared memory): sequences b0 .. b0 +
// B - 1 of the B_all of a call; the pointers are those of sequence b0, but for the
// caches', which are the call's.
constexpr int kTreeSeqs = 256;
// Nodes times query heads of a group up to which the kernel with the keys on the
// MMA's lanes takes a call (attention_few.cu).
constexpr int kTreeFewRows = 32;
// Items are cut when the longest, as often as an SM takes one, has `join` tiles
// more than the SM's share u of all tiles, and u / 2, at most `run`, more on top:
// otherwise the join, and the second run of a CTA, cost more than they save.  One bound
// for both head sizes and cache types, set at D = 64, fp16.  Measured, whole / cut, in
// us, 8 KV heads of 4 heads each, by tiles of a sequence:
//   8 sequences of 24 nodes (cut from 7 on)   4 tiles      6           8          10
//     D = 64, fp16                         9.7/11.9   11.7/12.8   13.6/15.0   15.4/15.7
//     D = 64, Q8_0                        12.8/12.5   14.9/13.9   17.1/16.5   19.2/16.8
//     D = 128, fp16                       13.0/13.5   16.5/18.4   20.0/21.1   22.7/22.2
//     D = 128, Q8_0                       17.1/15.7   19.8/17.6   22.4/20.7   25.4/21.7
//   one of 64 nodes (from 5 on)               3 tiles      4           6
//     D = 64, fp16                        11.3/13.2   12.1/12.1   14.1/12.5
//     D = 64, Q8_0                        14.2/14.1   15.1/13.0   17.3/13.4
//     D = 128, fp16                       14.2/14.9   14.8/13.2   17.6/13.5
//     D = 128, Q8_0                       19.2/17.4   20.9/14.8   23.6/15.1
//   few rows, 8 sequences of 4 (from 17 on)  16 tiles     20          24
//     D = 64, fp16                        16.4/18.2   19.4/20.1   21.9/21.8
//     D = 64, Q8_0                        19.9/20.0   23.0/20.9   26.2/22.9
//     D = 128, fp16                       18.9/22.7   21.8/25.8   24.5/28.4
//     D = 128, Q8_0                       23.0/24.7   26.8/27.2   30.5/29.4
//   few rows, one of one (from 7 on)          4 tiles      6           8
//     D = 64, fp16                          7.2/7.7     8.4/8.2     9.6/9.0
//     D = 64, Q8_0                          8.8/9.1    10.3/9.5    11.8/10.3
//     D = 128, fp16                         8.0/8.0     9.2/8.3    10.5/8.5
//     D = 128, Q8_0                        10.3/9.7   11.8/10.1    13.5/10.2
struct TreeWhole {
  float join, run;
};
constexpr TreeWhole kRowsWhole{4.f, 0.f}, kFewWhole{6.f, 4.f};
constexpr int kTreeLeast = 2;   // key tiles a CTA takes at least
struct TreeParams {
  const __half* q;        // [H][q_rows][D], row b N + i
  const uint8_t* k;       // [B_all][Hkv][C] rows
  const uint8_t* v;
  __half* o;              // [B N][H D]
  const int32_t* past;    // [B]
  const int32_t* parents; // [B][N]
  long long q_rows;       // B_all N
  int B, B_all, b0, H, Hkv, G, N, C, D;
  float scale_log2;       // softmax scale * log2(e)
  int rtiles;             // row tiles of an item's sequence and KV head: ceil(N G / 128)
  int split;              // tiles are dealt out evenly over the CTAs, pieces of items joined
                          // (unless, on the device, every item is short: tree_cut)
  TreeWhole whole;
  float share;            // an SM's share of a tile: 1 / SMs
  int waves;              // items an SM takes: ceil(B Hkv rtiles / SMs), of a full launch
  int ws_rows;            // rows of a piece: min(N G, 128)
  float2* ws_ml;          // [2 grid][ws_rows] (max, sum) of a piece
  float* ws_o;            // [2 grid][ws_rows][D] its unnormalised O
  uint32_t* status;
};
// tm_k, tm_v: [B_all Hkv][C][D] of fp16 caches, boxes of [1][128 keys][64 d],
// 128-byte swizzle (not read for Q8_0).
cudaError_t launch_attention_tree(const TreeParams& p, bool q8, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                  int grid, cudaStream_t s);
// attention_few.cu: the same for N G <= 32 rows an item
cudaError_t launch_attention_few(const TreeParams& p, bool q8, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                 int grid, cudaStream_t s);

// attention_paged.cu: attention of one new token of each of B sequences over the rows
// of a page pool [P][Hkv][page] that its table names.  One launch takes up to kPagedSeqs
// sequences (where their chunks of keys begin stays in shared memory); the pointers are
// those of the launch's first one.
constexpr int kPagedSeqs = 512;
struct PagedParams {
  const __half* q;        // [H][q_rows][D]
  const uint8_t* k;       // [P][Hkv][page] rows
  const uint8_t* v;
  __half* o;              // [B][H D]
  const int32_t* table;   // [B][W]
  const int32_t* lengths; // [B]
  long long q_rows;       // sequences of the call
  int B, H, Hkv, G, P, page, W, D;
  float scale_log2;       // softmax scale * log2(e)
  int rtiles;             // items of a sequence and KV head: ceil(G / rows of an item)
  int split;              // chunks may be dealt out evenly over the CTAs, pieces of items joined
  float waves, share, join;   // (on the device: where the longest item's cost times `waves`, the items a CTA
                          // takes, is more than `share` of all and `join` on top: PagedCut)
  int4* ws_cut;           // [grid] of the item cut whose first chunk is the CTA's: sequence, item, last CTA, 1
  float2* ws_ml;          // [2 grid][rows] (max, sum) of a piece
  float* ws_o;            // [2 grid][rows][D] its unnormalised O
  uint32_t* status;
};
// Query heads of an item, keys of a chunk (four warps' steps of 16 or 32 keys, 4 to 9 KB of
// rows each), and CTAs an SM.  Q8_0, 32 sequences: 16 keys a step and four CTAs took 62.5 us
// against 61.0 at D = 128, 64 keys and three CTAs 40.1 against 38.0 at D = 64.
constexpr int paged_rows(int G) { return G <= 8 ? 8 : 16; }
constexpr int paged_chunk(int D, bool q8) { return q8 ? 128 : 8192 / D; }
constexpr int paged_ctas(int G, int D, bool q8) { return G > 8 ? 2 : q8 && D == 64 ? 4 : 3; }
// Items are cut when the longest, as often as a CTA takes one, costs `share` times a CTA's
// part of all and `join` more: an item costs its chunks and one.  Measured, whole / cut, in
// us, 8 KV heads of 4 heads each, by keys of a sequence:
//   one sequence (cut from 640, 320, 512, 512)  256        384        512        1024
//     D = 64, fp16                            4.6/6.1    5.3/6.1    5.9/6.2    8.5/6.2
//     D = 128, fp16                           6.1/6.4    7.5/6.4    8.9/6.4   14.5/6.8
//     D = 64, Q8_0                            5.3/6.8    6.2/6.7    7.2/6.8   10.9/6.8
//     D = 128, Q8_0                           5.9/7.2    7.2/7.2    8.4/7.3   13.1/7.4
//   8 sequences (768, 384, 640, 640)          384        512        768        1024
//     D = 64, fp16                            5.7/7.5    6.3/7.8    7.7/7.9    9.1/8.6
//     D = 128, fp16                           8.0/8.4    9.5/9.0   12.4/9.4   15.2/10.9
//     D = 64, Q8_0                            6.7/8.3    7.7/8.3    9.7/8.7   11.6/9.3
//     D = 128, Q8_0                           7.7/9.0    8.9/9.6   11.3/9.8   13.7/11.1
//   32 sequences (1,792, 896, 768, 896)       512        1024       1536       2048
//     D = 64, fp16                            7.7/10.1  11.0/12.6  15.4/15.4  28.0/27.8
//     D = 128, fp16                          11.2/13.2  27.0/27.9  37.9/38.1  50.4/47.9
//     D = 64, Q8_0                           10.7/11.4  17.1/14.3  23.8/16.7  30.4/19.7
//     D = 128, Q8_0                          12.6/13.3  20.7/18.4  30.0/24.4  38.6/32.2
//   128 sequences (1,280, 640, 640, 384)      256        384        512        1024
//     D = 64, fp16                           13.1/14.3  17.5/17.8  26.6/28.1  46.7/48.9
//     D = 128, fp16                          27.2/28.1  37.4/38.7  47.2/48.4  85.2/87.6
//     D = 64, Q8_0                           13.5/16.0  16.9/20.0  20.5/22.3  36.8/37.0
//     D = 128, Q8_0                          20.1/21.3  28.3/29.0  35.0/34.3  59.4/53.9
// Of unequal lengths the longest decides, and cutting gains more.  The rule is one for both head
// dims, so it is not the faster side at every point: it cuts 8 sequences of 768 fp16 keys at D =
// 64, 32 of 1,024 and 1,536 at D = 128 and 128 of 384 Q8_0 keys at D = 128, for 1 to 3% more
// time.
// Short sequences under a wide table (a call's launches follow the table, whose lengths only the
// device knows): 300 keys of one sequence take 6.9 us of device time and 14 called under a table
// of 304 rows, 7.2 and 19 to 20 under one of 4,096 or 131,072 (Q8_0: 7.5 and 14, 9.3 and 19); 20
// keys 3.8 and 5.9.
struct PagedCut {
  float share, join;
};
constexpr PagedCut paged_cut(bool q8) { return q8 ? PagedCut{0.7f, 4.5f} : PagedCut{1.1f, 5.5f}; }
// tm_k, tm_v: [P Hkv][page][D] of fp16 pools, boxes of [1][8 rows][64 d], 128-byte swizzle
// (not read for Q8_0).
cudaError_t launch_attention_paged(const PagedParams& p, bool q8, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                   int grid, cudaStream_t s);

// page_plan.cu: pages handed to sequences and taken back, and the slots of a step's
// tokens.
constexpr int kPlanSeqs = 4096;
struct PlanParams {
  const int32_t* past;    // [B]
  const int32_t* fresh;   // [B] new tokens; below 0: ended
  int32_t* table;         // [B][W]
  int32_t* held;          // [B]
  int32_t* free_pages;    // [P]
  int32_t* n_free;        // [1]
  int32_t* slots;         // [T]
  int32_t* pos;           // [T]
  int32_t* lengths;       // [B]
  int32_t* starts;        // [B + 1]
  int B, W, P, page, T;
  int ctas;               // of the cluster: 1, 2, 4 or 8
  uint32_t* status;
};
cudaError_t launch_page_plan(const PlanParams& p, int threads, cudaStream_t s);

// verify.cu: drafted trees verified against the target's probabilities.
constexpr int kVerifyNodes = 256;
struct VerifyParams {
  const void* target;     // [B][N] rows of V probabilities, strides in elements
  const void* draft;
  long long t_bs, t_rs, d_bs, d_rs;
  const int32_t* tokens;  // [B][N]
  const int32_t* parents; // [B][N]
  const float* u;         // [B][N]
  int32_t* path;          // [B][N]
  int32_t* count;         // [B]
  int32_t* token;         // [B]
  int B, N, V;
  int ctas;               // of a sequence's cluster: 1 to 8, or 16
  uint32_t* status;
};
cudaError_t launch_verify(const VerifyParams& p, bool f16, cudaStream_t s);

// misc.cu
// Status bit of a failed bounds check (the kernels' kErrBounds), and the
// bounds-checked build switch (-DM4Q_BOUNDS=1).
constexpr uint32_t kErrBoundsBit = 4u;
#ifndef M4Q_BOUNDS
#define M4Q_BOUNDS 0
#endif
uint32_t* status_words();  // [0] wait/bounds status, [1] non-finite flag, [2] first bounds site; per current device
cudaError_t launch_dequant(int codec, const void* w, int N, int K, long long row_bytes, void* out,
                           cudaStream_t s);
cudaError_t launch_finite_check(const void* x, long long n, uint32_t* flag, cudaStream_t s);
cudaError_t launch_wait_selftest(uint32_t* status, unsigned long long limit_ns, cudaStream_t s);
cudaError_t launch_mlx4_pack(const void* words, const void* scales, const void* biases, int N, int K,
                             void* w, int sms, cudaStream_t s);
cudaError_t launch_repack(int codec, const void* w, long long blocks, void* out, int sms, cudaStream_t s);

}  // namespace m4q
