/*
 * m4q.h -- C ABI of the block-quantized projection library for one GB300
 * (sm_103a).  Shared object: swiglu_block_quantized_gb300/_build/libm4q.so.
 *
 * The operation (m4-prefill-engine pages):
 *  - "v0.1 vs v0.2 comparison", section 2.1, and the project page's Pillar 1
 *    (Bricks 1 and 2): the prefill projection Y[M,N] = X[M,K] * W^T with fp16
 *    activations and block-quantized weights unpacked inside the kernel.
 *  - "Releases", v0.3.0 (M4QuantizedLinear): one linear layer dispatches to a
 *    GEMV for decode-sized M and to a GEMM otherwise, across every codec.
 *  - "v0.1 vs v0.2 comparison", section 2.2 (Brick 3): the fused gate/up
 *    projection SiLU(X * Wg^T) x (X * Wu^T), computed on chip, writing only
 *    the final activation.  "Releases" v0.3.0 (TransformerBlock: SwiGLU /
 *    GeGLU activations) adds the GELU-gated form, GELU(g) = g * Phi(g).
 *  - "Releases", v0.3.0, PrismML Q2_0 codec: 128 weights in 34 bytes,
 *    w = (q - 1) * d with the reserved code 3 decoding to +2d.  Q4_0 and Q8_0
 *    are GGUF's 32-weight blocks: w = (q - 8) * d and w = q * d.
 *  - Project page, section 4 (v0.2.1) and Table B: MLX 4-bit weights, a
 *    20-byte block_mlx_4bit and its planar form.  Read as MLX's affine group
 *    quantization at group size 32: w = q * s + b with an fp16 scale s and
 *    bias b per group of 32 weights.
 *
 * Conventions common to every call:
 *  - Pointers X, W, Wg, Wu, Y, Wf16 are DEVICE pointers (cudaMalloc'd or from
 *    PyTorch).  The caller owns every buffer; the library allocates nothing
 *    during a call and keeps no pointer after it returns.
 *  - Layouts are row-major and dense.  X is fp16 [M, K]; Y is fp16 [M, N].
 *    W is [N rows][K / B blocks] of packed blocks (B = 32 for Q4_0, Q8_0 and
 *    MLX4, 128 for Q2_0), block bytes 18 / 34 / 34 / 20, each block a
 *    little-endian fp16 scale d followed by its codes:
 *      Q4_0: byte 2+j holds weight j in its low nibble, weight j+16 high;
 *      Q8_0: byte 2+i holds weight i as a signed byte;
 *      Q2_0: byte 2+i/4 holds weight i at bits 2*(i%4)..2*(i%4)+1;
 *      MLX4: bytes 2-3 hold the fp16 bias b, byte 4+i/2 holds weight i,
 *            even i in the low nibble (MLX's order; m4q_mlx4_pack builds
 *            these blocks from MLX's planar arrays).
 *  - Shapes: M >= 1, N >= 8 with N % 8 == 0, K >= B with K % B == 0.
 *    X, W, Wg, Wu, Y must be 16-byte aligned.
 *  - Arithmetic: every weight is decoded to fp16 as (q - z) * d (MLX4:
 *    q * s + b) rounded once to nearest even, products are accumulated in
 *    fp32, and each output is
 *    rounded once to fp16 (SiLU(g) * u or GELU(g) * u is formed in fp32
 *    first).
 *  - Asynchrony: calls enqueue work on `stream` and return; argument errors
 *    are returned before anything is enqueued.  Launch failures return
 *    M4Q_ERR_CUDA.  Device-side failures (a pipeline wait that gave up) are
 *    recorded in a device status word that m4q_check_device_status() reads.
 *  - Threading: calls may be made from several host threads.
 */
#ifndef M4Q_H_
#define M4Q_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t.  NULL means the legacy default stream. */
typedef struct CUstream_st* m4q_stream_t;

/* Weight codecs. */
enum m4q_codec { M4Q_Q4_0 = 0, M4Q_Q8_0 = 1, M4Q_Q2_0 = 2, M4Q_MLX4 = 3 };

/* Execution paths for m4q_gemm_ex / m4q_swiglu_ex. */
enum m4q_path {
  M4Q_PATH_AUTO = 0, /* M <= 16: streaming GEMV; otherwise the tensor-core GEMM */
  M4Q_PATH_GEMV = 1, /* weight-streaming GEMV (requires M <= 16) */
  M4Q_PATH_TC = 2    /* tcgen05 tensor-core GEMM (any M) */
};

/* Activations of the gated projection (m4q_glu_ex). */
enum m4q_act {
  M4Q_ACT_SILU = 0, /* SiLU(g) = g / (1 + e^-g): SwiGLU */
  M4Q_ACT_GELU = 1  /* GELU(g) = g * Phi(g) = g/2 * erfc(-g / sqrt 2): GeGLU */
};

/* Status codes returned by every call. */
enum m4q_status {
  M4Q_OK = 0,
  M4Q_ERR_INVALID_ARG = -1,        /* null pointer, M/N/K out of range, bad path */
  M4Q_ERR_UNSUPPORTED_CODEC = -2,  /* codec not one of enum m4q_codec */
  M4Q_ERR_BAD_SHAPE = -3,          /* K % B != 0 or N % 8 != 0 */
  M4Q_ERR_MISALIGNED = -4,         /* a pointer is not 16-byte aligned */
  M4Q_ERR_CUDA = -5,               /* a CUDA runtime call or launch failed */
  M4Q_ERR_NONFINITE = -6,          /* m4q_check_finite found NaN/Inf */
  M4Q_ERR_TIMEOUT = -7,            /* a device pipeline wait gave up */
  M4Q_ERR_UNSUPPORTED_DEVICE = -8, /* the current device is not sm_103 */
  M4Q_ERR_SCRATCH_LIMIT = -9,      /* m4q_mlp_noalloc: M * F above its fixed scratch */
  M4Q_ERR_BOUNDS = -10             /* bounds-checked build: an access was out of range */
};

/* Y = X * W^T.  Dispatch: M <= 16 takes the GEMV path, else the tcgen05
 * path.  Errors as listed in enum m4q_status. */
int m4q_gemm(const void* X, const void* W, int codec, int64_t M, int64_t N, int64_t K,
             void* Y, m4q_stream_t stream);

/* Y = SiLU(X * Wg^T) x (X * Wu^T); Wg and Wu share codec and shape [N, K].
 * Neither intermediate product is written to memory. */
int m4q_swiglu(const void* X, const void* Wg, const void* Wu, int codec, int64_t M,
               int64_t N, int64_t K, void* Y, m4q_stream_t stream);

/* Y = X * W^T written head-major: Y[h][m][d] = (X * W^T)[m][h * head_dim + d],
 * Y fp16 [N / head_dim][M][head_dim], so each head's [M, head_dim] block is
 * contiguous and attention reads it without a transpose ("v0.1 vs v0.2
 * comparison" section 4 and "Releases" v0.2.1: direct-head [H, M, D]
 * projection).  head_dim is 64 or 128 (else M4Q_ERR_INVALID_ARG) and must
 * divide N (else M4Q_ERR_BAD_SHAPE).  A fused Q/K/V projection is one call
 * on the row concatenation of Wq, Wk and Wv (packed rows are independent, so
 * concatenating the packed matrices concatenates the rows): the first
 * N_q / head_dim heads of Y are Q, then K, then V.  Otherwise as m4q_gemm. */
int m4q_gemm_heads(const void* X, const void* W, int codec, int64_t M, int64_t N, int64_t K,
                   int64_t head_dim, void* Y, m4q_stream_t stream);

/* Y = GELU(X * Wg^T) x (X * Wu^T) ("Releases" v0.3.0, GeGLU); otherwise as
 * m4q_swiglu. */
int m4q_geglu(const void* X, const void* Wg, const void* Wu, int codec, int64_t M,
              int64_t N, int64_t K, void* Y, m4q_stream_t stream);

/* As m4q_gemm / m4q_swiglu, with the path chosen by the caller (enum m4q_path). */
int m4q_gemm_ex(const void* X, const void* W, int codec, int64_t M, int64_t N, int64_t K,
                void* Y, int path, m4q_stream_t stream);
int m4q_swiglu_ex(const void* X, const void* Wg, const void* Wu, int codec, int64_t M,
                  int64_t N, int64_t K, void* Y, int path, m4q_stream_t stream);

/* The gated projection Y = act(X * Wg^T) x (X * Wu^T) with the activation
 * (enum m4q_act) and the path (enum m4q_path) chosen by the caller.  An
 * unknown act returns M4Q_ERR_INVALID_ARG. */
int m4q_glu_ex(const void* X, const void* Wg, const void* Wu, int codec, int64_t M, int64_t N,
               int64_t K, void* Y, int act, int path, m4q_stream_t stream);

/* The gated MLP block of a transformer layer ("Releases" v0.3.0:
 * TransformerBlock with SwiGLU / GeGLU activations):
 *     H = act(X * Wg^T) x (X * Wu^T)      fp16 [M, F]
 *     Y = H * Wd^T                         fp16 [M, D]
 * enqueued as two launches on `stream` (the gated projection, then the down
 * projection), each with the M <= 16 / tcgen05 dispatch of m4q_gemm.
 * X is fp16 [M, D]; Wg, Wu are packed [F, D] in codec_gu; Wd is packed
 * [D, F] in codec_d.  H is caller-provided device scratch of M * F fp16
 * (16-byte aligned) that receives the intermediate activation; it may be
 * reused once the call's work on `stream` has completed.  Shape rules of
 * m4q_gemm apply to both projections (D and F multiples of 8 and of the
 * block sizes).  act: enum m4q_act. */
int m4q_mlp(const void* X, const void* Wg, const void* Wu, const void* Wd, int codec_gu,
            int codec_d, int64_t M, int64_t D, int64_t F, void* H, void* Y, int act,
            m4q_stream_t stream);

/* m4q_mlp for callers that cannot allocate device memory (a runtime that
 * owns all device memory and gives plug-ins no allocator, or a loop that must
 * not call cudaMalloc, which may synchronize the device).  The pages have no
 * counterpart: this is a deployment variant of m4q_mlp.  Same arguments and
 * result as m4q_mlp without H: the fp16 intermediate is kept in one fixed
 * device array of the library, 1 << 20 elements (2 MiB, held on every GPU
 * that loads the library until the process exits).  M * F above that returns
 * M4Q_ERR_SCRATCH_LIMIT before anything is enqueued.  The call allocates
 * nothing.  The first call on a device checks that it is an sm_103 part
 * (else M4Q_ERR_UNSUPPORTED_DEVICE), looks up the array's device address
 * (cudaGetSymbolAddress) and keeps it for the life of the process; it should
 * come before any stream capture on that device.  cudaDeviceReset() on a
 * device makes the kept address stale: do not call this entry point on that
 * device afterwards.  All calls share the array: each one overwrites the part
 * it uses before reading it, but calls whose work overlaps on the GPU (no
 * stream order between them) race. */
int m4q_mlp_noalloc(const void* X, const void* Wg, const void* Wu, const void* Wd, int codec_gu,
                    int codec_d, int64_t M, int64_t D, int64_t F, void* Y, int act,
                    m4q_stream_t stream);

/* The projection of m4q_gemm (W1 == NULL) or the gated projection of
 * m4q_glu_ex (W1 != NULL, activation `act`) with the activations in host
 * memory and the result written to host memory: the end-to-end call of a
 * caller whose inputs arrive from the host.  M is cut into chunks of
 * `chunk_rows` rows (0: about a quarter of M, rounded up to 128 rows); each
 * chunk's activations are copied to the device on `h2d_stream`, projected on
 * `stream` (the dispatch of m4q_gemm / m4q_glu_ex with path AUTO) and
 * copied back on `d2h_stream`, so the copies of one chunk overlap the
 * kernels of its neighbours.  The copies overlap only if X_host and Y_host
 * are page-locked (cudaHostAlloc / pinned); otherwise the result is the same
 * and the copies serialize.
 *  - X_host: fp16 [M, K]; Y_host: fp16 [M, N] (host memory).
 *  - X_dev, Y_dev: device staging buffers of M * K and M * N fp16, 16-byte
 *    aligned, owned by the caller (the library allocates no memory).
 *  - W0, W1: packed device weights as for m4q_gemm / m4q_glu_ex.
 *  - Ordering: the copies start after the work already enqueued on
 *    `stream`, and `stream` waits for the last copy back, so work enqueued
 *    on `stream` after this call, and a synchronization of `stream`, see
 *    Y_host complete.  The three streams should be distinct for overlap.
 *  - The call records CUDA events of a per-device pool, created by the first
 *    call on a device; calls from several host threads are serialized while
 *    they enqueue.
 * Errors: those of m4q_gemm / m4q_glu_ex (checked before anything is
 * enqueued), M4Q_ERR_INVALID_ARG for a null host or staging pointer or a
 * negative chunk_rows, M4Q_ERR_MISALIGNED for unaligned staging buffers. */
int m4q_project_host(const void* X_host, const void* W0, const void* W1, int codec, int act, int64_t M,
                     int64_t N, int64_t K, void* Y_host, void* X_dev, void* Y_dev, int64_t chunk_rows,
                     m4q_stream_t stream, m4q_stream_t h2d_stream, m4q_stream_t d2h_stream);

/* Repack MLX 4-bit weights from MLX's planar arrays into MLX4 blocks
 * (project page, section 4: the deinterleaved "mlx_4bit_planar" layout of
 * the 20-byte block_mlx_4bit).  words: uint32 [N, K/8], code k of row n at
 * bits 4*(k%8) of word k/8 (little-endian); scales, biases: fp16 [N, K/32],
 * one per group of 32 weights.  W receives [N, K/32] 20-byte blocks
 * (m4q_weight_bytes(M4Q_MLX4, N, K) bytes) for any call above.  A one-time
 * layout step, not part of a projection: the tensor-core path moves whole
 * 160-byte stages of 8 blocks by TMA, so the 20-byte block stride never
 * splits a copy.  Requires N >= 1, K >= 32 with K % 32 == 0 (else
 * M4Q_ERR_BAD_SHAPE); words and W 16-byte aligned, scales and biases 2-byte
 * aligned (else M4Q_ERR_MISALIGNED).  Device pointers; enqueued on stream. */
int m4q_mlx4_pack(const void* words, const void* scales, const void* biases, int64_t N, int64_t K,
                  void* W, m4q_stream_t stream);

/* Split packed weights into planes ("v0.1 vs v0.2 comparison", section 4:
 * the v0.2.1 planar layout, which moves the codes of the 20-byte MLX 4-bit
 * blocks into their own 16-byte aligned array; the same split is offered for
 * every codec).  W: packed [N, K/B] blocks in `codec`.  Wplanar receives, back
 * to back with no padding, m4q_weight_bytes(codec, N, K) bytes in all:
 *   codes:  the code bytes of every block, unchanged, in row-major block
 *           order (16 bytes per block for Q4_0 and MLX4, 32 for Q8_0 and
 *           Q2_0), at offset 0;
 *   scales: fp16 [N, K/B], each block's scale d (MLX4: s), right after;
 *   biases: fp16 [N, K/B], MLX4 only, each block's bias b, after the scales.
 * For MLX4 the three arrays are MLX's own planar arrays (the inverse of
 * m4q_mlx4_pack).  The projections above read the packed blocks, never the
 * planes: this is an export for callers that store or hand on weights in
 * planar form.  Requires a known codec (else M4Q_ERR_UNSUPPORTED_CODEC),
 * N >= 1, K >= 1 (else M4Q_ERR_INVALID_ARG) with K % B == 0 (else
 * M4Q_ERR_BAD_SHAPE), W and Wplanar 16-byte aligned (else
 * M4Q_ERR_MISALIGNED) and not overlapping (not checked).  Device pointers;
 * enqueued on stream; the caller owns both buffers. */
int m4q_repack(const void* W, int codec, int64_t N, int64_t K, void* Wplanar, m4q_stream_t stream);

/* KV cache value formats for m4q_attention: fp16 values, or M4Q_Q8_0 blocks
 * along the head dimension. */
enum m4q_kv_codec { M4Q_KV_F16 = 16 };

/* Attention of fp16 queries over a KV cache ("v0.1 vs v0.2 comparison" 2.3:
 * FlashAttention with the Q8_0 KV cache dequantized on the fly; "Releases"
 * v0.3.0: grouped-query attention, causal masking with a sequence offset,
 * head dims 64 and 128; v0.2: chunked attention, running max and sum merged
 * exactly across key chunks):
 *   O[i, h*D + d] = sum_j softmax_j(scale * Q[h, i, :] . K[h / G, j, :]) V[h / G, j, d]
 * with G = H / Hkv, over keys j < T, and, when causal != 0, j <= q_offset + i.
 *  - Q: fp16 [H, M, D] (head-major, as m4q_gemm_heads writes it).
 *  - K, V: [Hkv, T] rows of D values: fp16 (kv_codec M4Q_KV_F16, 2 D bytes a
 *    row) or Q8_0 (kv_codec M4Q_Q8_0: D / 32 blocks of 34 bytes a row, the
 *    same block as the Q8_0 weights).  Each value enters the products as
 *    fp16 (Q8_0: RNE(q * d)).
 *  - O: fp16 [M, H * D] (token-major: the o-projection's input).
 *  - D is 64 or 128, H % Hkv == 0 (else M4Q_ERR_BAD_SHAPE); M, T >= 1,
 *    q_offset >= 0, scale finite (else M4Q_ERR_INVALID_ARG; the usual scale
 *    is 1 / sqrt(D)); Q, K, V, O and workspace 16-byte aligned.
 *  - Scores and the softmax are fp32; the probabilities are rounded to fp16
 *    for the P V product, which accumulates in fp32; O is rounded once.
 *  - workspace (m4q_attention_workspace() bytes of device memory, owned by
 *    the caller): when the query rows alone would leave SMs idle (decode),
 *    the keys are split across CTAs and merged by a second kernel, which
 *    keeps its partial results there; for a Q8_0 cache under a prefill-sized
 *    call (more than 16 rows per KV head) both caches are first decoded to
 *    fp16 there (RNE(q * d), as above), since every key tile is read by each
 *    row tile of its KV head, and the fp16 tensor-core path runs on them.
 *    NULL (or a smaller size) runs without either: the same result up to
 *    fp32 rounding, slower.  The library allocates nothing. */
int m4q_attention(const void* Q, const void* K, const void* V, int kv_codec, int64_t H, int64_t Hkv,
                  int64_t M, int64_t T, int64_t D, int64_t q_offset, int causal, float scale, void* O,
                  void* workspace, size_t workspace_bytes, m4q_stream_t stream);

/* Bytes of the key split's partial results m4q_attention keeps in its
 * workspace for this shape on the current device (0: no key split; also 0
 * for an invalid shape).  m4q_attention_workspace covers the Q8_0 staging
 * as well. */
size_t m4q_attention_workspace_bytes(int64_t H, int64_t Hkv, int64_t M, int64_t T, int64_t D);

/* Workspace bytes m4q_attention uses for this cache format and shape on the
 * current device: the key split's partial results, or for a Q8_0 cache
 * under a prefill-sized call 2 Hkv T D fp16 values (the decoded caches);
 * 0 when it uses none, or for an invalid shape. */
size_t m4q_attention_workspace(int kv_codec, int64_t H, int64_t Hkv, int64_t M, int64_t T, int64_t D);

/* ---------------------------------------------------------------------------
 * Between the projections and attention: rotary positions, the KV cache
 * written and read back, attention of drafted trees of tokens over a batch of
 * caches, and the norms around a block.  A decoder layer's step is
 *   m4q_norm_residual -> m4q_gemm_heads (Q, K, V) -> m4q_kv_write (with Q)
 *   -> m4q_attention_tree or m4q_attention -> m4q_gemm -> m4q_norm_residual
 *   -> m4q_mlp.
 *
 * A batch of caches: Kc, Vc hold [B][Hkv][C] rows of D values (D 64 or 128),
 * C the capacity in rows of every sequence; a row is fp16 (kv_codec
 * M4Q_KV_F16) or Q8_0 blocks along D (M4Q_Q8_0), as for m4q_attention, whose
 * caches are those of one sequence with T = C.  B * Hkv * C <= INT32_MAX, and
 * a Q8_0 cache is a multiple of 16 bytes (always so where C % 4 == 0), else
 * M4Q_ERR_BAD_SHAPE.  Row b * C + j of every KV head is cache row j of
 * sequence b: its "slot" is b * C + j.
 */

/* How rotary positions pair the first `rot` values of a row: value i with
 * value i + rot / 2, or value 2 i with value 2 i + 1. */
#define M4Q_ROPE_HALF 0
#define M4Q_ROPE_INTERLEAVED 1

/* Frequencies of m4q_rope_freqs, f_i = base^(-2 i / rot) radians a position:
 *  PLAIN   as they are;
 *  LINEAR  f_i / factor (positions interpolated);
 *  NTK     base * factor^(rot / (rot - 2)) for base (rot > 2);
 *  BANDS   by r_i = original f_i / (2 pi), the turns of pair i over the
 *          original length: f_i / factor where r_i <= low, f_i where r_i >=
 *          high, the linear mix in between;
 *  YARN    the same, with the magnitude factor 0.1 ln(factor) + 1.
 * BANDS and YARN mix by turns.  Models that were trained with a ramp over the pair
 * index i between two rounded indices (the turns beta_slow and beta_fast turned into
 * indices first) have other frequencies between the bands: give a table of one's
 * own for those. */
#define M4Q_ROPE_PLAIN 0
#define M4Q_ROPE_LINEAR 1
#define M4Q_ROPE_NTK 2
#define M4Q_ROPE_BANDS 3
#define M4Q_ROPE_YARN 4

/* Fills the frequency table of m4q_rope and m4q_kv_write: freqs (HOST memory,
 * rot / 2 entries) receives f_i as turns per position in units of 2^-64, i.e.
 * round(f_i / (2 pi) 2^64) mod 2^64 (any table of that form may be used), and
 * *mscale (HOST, may be NULL) the magnitude factor (1, or YARN's).  The
 * caller copies the table to the device once.  rot even and >= 2, base > 1,
 * factor >= 1 finite; BANDS and YARN: original > 0, 0 <= low < high, else
 * M4Q_ERR_INVALID_ARG.  Host work only. */
int m4q_rope_freqs(int64_t rot, double base, int scaling, double factor, double original, double low,
                   double high, int64_t* freqs, float* mscale);

/* Rotary positions: Y[h][m] = X[h][m] with each pair (a, b) of its first rot
 * values turned by pos[m] f_i: (a, b) -> mscale (a cos - b sin, b cos + a sin);
 * values from rot on are copied.
 *  - X, Y: fp16 rows of D values for H heads and M tokens; row (h, m) starts
 *    h * head_stride + m * row_stride elements in (strides multiples of 8,
 *    else M4Q_ERR_MISALIGNED): head-major as m4q_gemm_heads writes it, or the
 *    rows of m4q_gemm.  Y may be X (with X's strides), otherwise they do not
 *    overlap (not checked).
 *  - pos: int32 [M], any value (a negative position turns backwards).
 *  - freqs: the table of m4q_rope_freqs on the device; rot a multiple of 16,
 *    16 <= rot <= D; layout M4Q_ROPE_HALF or _INTERLEAVED.
 *  - The fraction of a turn pos f_i of the table's f_i is exact at every position and
 *    rounded by at most 2^-28 of a turn; sines, cosines and products are fp32, and each
 *    value is rounded once. */
int m4q_rope(const void* X, int64_t x_head_stride, int64_t x_row_stride, int64_t H, int64_t M, int64_t D,
             const int32_t* pos, const int64_t* freqs, int64_t rot, int layout, float mscale, void* Y,
             int64_t y_head_stride, int64_t y_row_stride, m4q_stream_t stream);

/* The same with positions of several axes (time, height and width of an image's or a
 * video's patches): pair i turns by pos[axes[i]][m] f_i.
 *  - pos: int32 [A][M], 1 <= A <= M4Q_ROPE_MAX_AXES (else M4Q_ERR_INVALID_ARG).
 *  - axes: int32 [rot / 2] on the device, the axis of each pair; a pair whose axis is
 *    outside [0, A) is not turned (position 0).  With every axis 0 the result is
 *    m4q_rope's, bit for bit. */
#define M4Q_ROPE_MAX_AXES 8
int m4q_rope_axes(const void* X, int64_t x_head_stride, int64_t x_row_stride, int64_t H, int64_t M, int64_t D,
                  const int32_t* pos, int64_t A, const int64_t* freqs, const int32_t* axes, int64_t rot, int layout,
                  float mscale, void* Y, int64_t y_head_stride, int64_t y_row_stride, m4q_stream_t stream);

/* Writes the K and V rows of M tokens to the caches, K turned as by m4q_rope
 * on the way (freqs NULL: as it is; pos, rot, layout and mscale are then not
 * read), and in the same launch turns the tokens' queries (Q NULL: none).
 *  - K, V: fp16 rows for Hkv heads and M tokens, strides as for m4q_rope.
 *  - slots: int32 [M], the cache row b * C + j of each token.  A slot outside
 *    [0, B * C) writes nothing (padding).  Two tokens of one call do not share
 *    a slot (not checked: the row would mix both).  Rows that no slot names
 *    are left as they are.  The caches overlap neither each other nor K, V, Q
 *    or Qout (not checked).
 *  - A Q8_0 block of 32 values x: d = max|x| / 127 rounded up to fp16, codes
 *    x / d to the nearest integer, ties to even (none exceeds 127); a block
 *    with an infinity or a NaN decodes to NaN.  K is quantised from the fp32
 *    results of its rotation.
 *  - Q: fp16 rows for H heads and the same M tokens; Qout fp16 [H][M][D], may
 *    be Q if Q has those strides.  Q needs freqs (else M4Q_ERR_INVALID_ARG).
 *    H + 2 Hkv <= 65535. */
int m4q_kv_write(const void* K, int64_t k_head_stride, int64_t k_row_stride, const void* V,
                 int64_t v_head_stride, int64_t v_row_stride, int64_t Hkv, int64_t M, int64_t D,
                 const int32_t* pos, const int64_t* freqs, int64_t rot, int layout, float mscale,
                 const int32_t* slots, void* Kc, void* Vc, int kv_codec, int64_t B, int64_t C, const void* Q,
                 int64_t q_head_stride, int64_t q_row_stride, int64_t H, void* Qout, m4q_stream_t stream);

/* The same with positions of several axes, as m4q_rope_axes (freqs and axes are
 * needed, else M4Q_ERR_INVALID_ARG). */
int m4q_kv_write_axes(const void* K, int64_t k_head_stride, int64_t k_row_stride, const void* V,
                      int64_t v_head_stride, int64_t v_row_stride, int64_t Hkv, int64_t M, int64_t D,
                      const int32_t* pos, int64_t A, const int64_t* freqs, const int32_t* axes, int64_t rot, int layout,
                      float mscale, const int32_t* slots, void* Kc, void* Vc, int kv_codec, int64_t B, int64_t C,
                      const void* Q, int64_t q_head_stride, int64_t q_row_stride, int64_t H, void* Qout,
                      m4q_stream_t stream);

/* Reads cache rows back: Kout, Vout fp16 [Hkv][n][D], row j the cache row
 * slots[j] (Q8_0: each value RNE(q d)); a slot outside [0, B * C) gives zeros,
 * and slots may repeat.  Kc with Kout, or Vc with Vout, may be NULL, not both.  Kout
 * and Vout overlap neither each other nor the caches (not checked). */
int m4q_kv_read(const void* Kc, const void* Vc, int kv_codec, int64_t B, int64_t Hkv, int64_t C, int64_t D,
                const int32_t* slots, int64_t n, void* Kout, void* Vout, m4q_stream_t stream);

/* Attention of N drafted nodes of each of B sequences over its cache (N = 1:
 * one new token a sequence).  Node i of sequence b sees the cache rows
 * j < past[b] and, at rows past[b] + a, its ancestors a and itself:
 *   O[b N + i, h D + d] = sum_j softmax_j(scale Q[h, b N + i] . K[b, h / G, j]) V[b, h / G, j, d]
 * with G = H / Hkv.  The nodes' own keys and values are in the cache already
 * (m4q_kv_write with slots b C + past[b] + i).
 *  - Q: fp16 [H][B N][D]; O: fp16 [B N][H D], which overlaps no other argument (not
 *    checked).
 *  - past: int32 [B] on the device (read by the kernel: a captured call
 *    follows its changes), clamped to [0, C]; a node whose row past[b] + i is
 *    not below C has no key of its own.
 *  - parents: int32 [B][N] on the device: -1 for a node that continues the
 *    cached context, else an earlier node (a < i).  Any other value, or a
 *    parent that is itself unused, marks the node as unused: its output row
 *    is zero and no node sees it.
 *  - Rows that a node does not see do not enter its result, whatever they
 *    hold (infinities and NaN included).
 *  - D is 64 or 128, H % Hkv == 0, Hkv ceil(N G / 128) ceil(C / 128) <=
 *    INT32_MAX (else M4Q_ERR_BAD_SHAPE); 1 <= N <= 256, B, C >= 1,
 *    B * N * H <= INT32_MAX, scale log2(e) finite in 32 bits (else
 *    M4Q_ERR_INVALID_ARG).
 *  - Arithmetic as m4q_attention.
 *  - workspace: m4q_attention_tree_workspace() bytes (not cleared before or
 *    after, 16-byte aligned) for the partial results of keys split across
 *    CTAs; NULL or a smaller size runs without a split, slower.  Calls whose
 *    work overlaps need a workspace each. */
int m4q_attention_tree(const void* Q, const void* Kc, const void* Vc, int kv_codec, int64_t B, int64_t H,
                       int64_t Hkv, int64_t N, int64_t C, int64_t D, const int32_t* past,
                       const int32_t* parents, float scale, void* O, void* workspace, size_t workspace_bytes,
                       m4q_stream_t stream);

/* Workspace bytes m4q_attention_tree uses for this shape on the current
 * device (0 when it uses none, or for an invalid shape). */
size_t m4q_attention_tree_workspace(int kv_codec, int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t C,
                                    int64_t D);

/* ---------------------------------------------------------------------------
 * A paged cache: pools Kc, Vc of P pages [P][Hkv][page] rows, shared by all sequences.
 * For m4q_kv_write and m4q_kv_read it is a batch of caches with B = P and C = page: row
 * r of page i has the slot i * page + r.  Each sequence has a row of the block table,
 * int32 [B][W]: its rows j lie at place j % page of page table[b][j / page].
 *
 * A step of one new token a sequence is m4q_page_plan -> (a layer: m4q_kv_write ->
 * m4q_attention_paged).  Where several tokens of a sequence attend (a prompt's, in every
 * layer but the last; a chain of drafted ones, before m4q_verify_tree) each of them is a
 * row of m4q_attention_paged of its own: its sequence's row of the table again, and a
 * length up to itself.  Each row reads its keys again, so the time grows with their
 * number.  The nodes of a drafted tree see keys that do not lie one behind the other:
 * m4q_kv_read brings the pages' rows into caches [B][Hkv][C] of fp16 rows, which
 * m4q_attention_tree takes.
 */

/* Pages and slots of a step, from lengths on the device (a captured call follows
 * them).  Sequence b has past[b] rows in the cache and gets fresh[b] tokens; fresh[b] <
 * 0 says that it has ended.
 *  - table int32 [B][W], held int32 [B], free_pages int32 [P], n_free int32 [1]: the
 *    state, on the device, updated.  held[b] entries of table[b] are pages of b (more
 *    than its rows need where drafted tokens were turned down); the first n_free
 *    entries of free_pages are free, the last of them handed out first.
 *  - b needs ceil((past[b] + fresh[b]) / page) pages, at most W, and is handed what it
 *    lacks, sequence by sequence; when the free ones run out the rest of the entries are
 *    -1.  An ended sequence's pages go on top of the free ones that are left (and are
 *    handed out from the next call on), its entries become -1 and held[b] 0.  Other
 *    entries of table and free_pages stay as they are.
 *  - A page is free or belongs to one sequence: among the free entries and those held no
 *    page is named twice (not checked), for one named twice goes back twice and is then
 *    handed to two sequences.  Sequences may share a prefix of whole pages all the same:
 *    one is given the prefix's entries as its first, held and past counting them, and
 *    before it ends its own entries move to the front of its row, held their number
 *    (the shared ones leave the row), so that the prefix goes back once, with the sequence
 *    that it came from, which ends after all that share it.
 *  - The tokens of all sequences lie one after the other in T places: starts int32
 *    [B + 1] is where each sequence's begin (starts[B]: their number; tokens behind the
 *    T-th are left out, as if fresh were smaller).  slots int32 [T], pos int32 [T]: the
 *    slot and the position past[b] + i of token i of b; the slot is -1 where b has no
 *    page for it.  Places behind the last token get slot -1 and position 0, so a padded
 *    m4q_kv_write of all T writes nothing for them.
 *  - lengths int32 [B]: the rows of b after the step, min(past[b] + fresh[b], held[b] *
 *    page), 0 for an ended one: what m4q_attention_paged reads.
 *  - Called again on its results with the same past and fresh it changes nothing, unless
 *    pages were missing or went back.
 *  - Values below 0 or above their range (past, held, n_free) count as the nearest in
 *    it; a table entry of b that is not a page gives slots of -1.
 *  - 1 <= B <= 4096, page, W, P, T >= 1, T <= INT32_MAX - 8192 (else
 *    M4Q_ERR_INVALID_ARG), P * page and W * page <= INT32_MAX (else
 *    M4Q_ERR_BAD_SHAPE).  The arrays do not overlap (not checked). */
int m4q_page_plan(const int32_t* past, const int32_t* fresh, int64_t B, int64_t page, int32_t* table, int64_t W,
                  int32_t* held, int32_t* free_pages, int64_t P, int32_t* n_free, int64_t T, int32_t* slots,
                  int32_t* pos, int32_t* lengths, int32_t* starts, m4q_stream_t stream);

/* Attention of one new token of each of B sequences over a paged cache:
 *   O[b, h D + d] = sum_{j < lengths[b]} softmax_j(scale Q[h, b] . K[b, h / G, j]) V[b, h / G, j, d]
 * with G = H / Hkv; the token's own row is one of them (lengths counts it).
 *  - Q: fp16 [H][B][D] (m4q_kv_write's Qout); O: fp16 [B][H D], which overlaps no other
 *    argument (not checked).
 *  - table int32 [B][W], lengths int32 [B] on the device, read by the kernel; lengths are
 *    clamped to [0, W * page].  Sequences may share pages, and several rows of a call may be
 *    tokens of one sequence (m4q_page_plan says how shared pages are given back).  Rows of
 *    an entry outside [0, P) are not seen; a sequence that sees no row gets zeros.
 *  - Rows behind the last do not enter the result, whatever they hold (infinities and
 *    NaN included).
 *  - D is 64 or 128, H % Hkv == 0, page % 8 == 0, W * page <= INT32_MAX, H (ceil(W page /
 *    64) + 1) <= INT32_MAX, the pools as for m4q_kv_write (else M4Q_ERR_BAD_SHAPE); B, H <=
 *    65535, scale log2(e) finite in 32 bits (else M4Q_ERR_INVALID_ARG).
 *  - A batch of caches [B][Hkv][C] (C % 8 == 0) is a pool of B pages of C rows, its table
 *    {{0}, {1}, ...}: for one new token a sequence m4q_attention_tree's result, up to
 *    roundings, in less time.
 *  - Arithmetic as m4q_attention (probabilities are rounded to fp16 before the product with
 *    V, 2^-11 of each, scores and sums are fp32), in runs of at most 2,048 keys a warp that are
 *    joined in fp32.  Within a run weights down to 2^-21 of its largest keep all of fp16's
 *    bits, those down to 2^-32 still count.
 *  - workspace: m4q_attention_paged_workspace() bytes (not cleared before or after,
 *    16-byte aligned) for the partial results of keys split across CTAs; NULL or a
 *    smaller size runs without a split, slower.  Calls whose work overlaps need a
 *    workspace each. */
int m4q_attention_paged(const void* Q, const void* Kc, const void* Vc, int kv_codec, int64_t B, int64_t H,
                        int64_t Hkv, int64_t P, int64_t page, int64_t D, const int32_t* table, int64_t W,
                        const int32_t* lengths, float scale, void* O, void* workspace, size_t workspace_bytes,
                        m4q_stream_t stream);

/* Workspace bytes m4q_attention_paged uses for this shape on the current device (0 when
 * it uses none, or for an invalid shape). */
size_t m4q_attention_paged_workspace(int kv_codec, int64_t B, int64_t H, int64_t Hkv, int64_t P, int64_t page,
                                     int64_t W, int64_t D);

/* Types of the probabilities of m4q_verify_tree. */
#define M4Q_PROB_F32 0
#define M4Q_PROB_F16 1

/* Drafted trees of tokens verified against the target's probabilities (speculative
 * sampling; siblings tried in turn), so that the tokens kept and the next one are
 * distributed as the target's own samples when each child was drawn from its parent's
 * draft distribution.
 *  - Node 0 of a sequence is its last known token (parents -1; any other value: an unused
 *    sequence, whose count is 0, token and path -1); node i > 0 is the drafted token
 *    tokens[b][i] behind node parents[b][i] in [0, i).  Nodes with other parents, or
 *    tokens outside [0, V), are unused.  (As m4q_attention_tree's nodes, with one root.)
 *  - target, draft: rows of V probabilities behind node i of sequence b, at
 *    b * seq_stride + i * row_stride elements, prob_type M4Q_PROB_F32 or _F16; p and q
 *    below.  Values that are not finite positive numbers count as 0; a row's sum is below
 *    2^120 (not checked).  draft may be NULL
 *    with N = 1: the next token is then a plain sample.
 *  - u: fp32 [B][N] in [0, 1): u[b][i] decides on node i, u[b][0] draws the next token.
 *  - From c = 0 on, with M = 0 and m = 1: the children of c in order of their index; x is
 *    taken, and becomes c, if u m q(x) < p(x) - M q(x); else M grows by m, and m becomes
 *    the sum of the rest r = max(p - M q, 0).  When no child is left the next token is
 *    the smallest x for which the sum of r up to x exceeds u[b][0] times the whole sum
 *    (M = 0: r = p).  Where r is 0 throughout (the draft covers the target, but for
 *    roundings) p stands for it; where p is 0 throughout the token is -1.
 *  - path int32 [B][N]: the nodes kept, 0 first, -1 behind them; count int32 [B]: their
 *    number; token int32 [B]: the next token.
 *  - A difference p - M q is formed to 2^-46 of p + M q.  A row's sum is formed to 2^-44 of
 *    it for rows of any one kind (softmaxes, equal or sorted values, up to 2^24 of them), and
 *    to 2^-34 whatever they hold (a thread's additions, up to 4,096 of 2^-47, all off to one
 *    side); neither is finer than 2^-146.  The order is fixed.
 *  - 1 <= N <= 256, 1 <= V <= 2^24 (else M4Q_ERR_INVALID_ARG).  The outputs overlap
 *    nothing (not checked). */
int m4q_verify_tree(const void* target, int64_t t_seq_stride, int64_t t_row_stride, const void* draft,
                    int64_t d_seq_stride, int64_t d_row_stride, int prob_type, int64_t B, int64_t N, int64_t V,
                    const int32_t* tokens, const int32_t* parents, const float* u, int32_t* path, int32_t* count,
                    int32_t* token, m4q_stream_t stream);

/* Types of the residual stream of m4q_norm_residual. */
#define M4Q_RES_F16 0
#define M4Q_RES_F32 1

/* The residual update and the norms after and before a block, one pass:
 *   u  = h / rms(h) * w_post                   (w_post NULL: u = h)
 *   r' = res_scale r + branch_scale gate u     (h NULL: r' = r)
 *   y  = r' / rms(r') * w_pre                  (w_pre and Y NULL: none)
 * for each of M rows of D values, rms(x) = sqrt(mean x^2 + eps).
 *  - h: fp16 [M][D], the block's output; R: the residual stream [M][D] in
 *    res_type; R_out: r' in res_type (NULL: not written; may be R); Y: fp16
 *    [M][D] (may be h, not R_out: M4Q_ERR_INVALID_ARG).  No other two arrays
 *    overlap (not checked).
 *  - w_post, w_pre: fp16 [D].  gate: fp16 [D] (gate_rows 0) or [M][D]
 *    (gate_rows 1), or NULL.
 *  - Sums, r' and products are fp32; r' is rounded where it is stored and y is
 *    formed from the unrounded r'.
 *  - D % 8 == 0 (else M4Q_ERR_BAD_SHAPE), 8 <= D <= 32768, eps >= 0, scales
 *    finite; w_post or gate without h, w_pre without Y or Y without w_pre, and
 *    a call that writes nothing are M4Q_ERR_INVALID_ARG.  16-byte aligned. */
int m4q_norm_residual(const void* h, const void* R, int res_type, const void* w_post, const void* gate,
                      int gate_rows, const void* w_pre, int64_t M, int64_t D, float res_scale,
                      float branch_scale, float eps, void* R_out, void* Y, m4q_stream_t stream);

/* Decode W [N, K] to fp16 Wf16 [N, K] (row-major): each weight (q - z) * d
 * (MLX4: q * s + b) rounded once to nearest even.  The test hook for
 * bit-exact decoding. */
int m4q_dequant(const void* W, int codec, int64_t N, int64_t K, void* Wf16,
                m4q_stream_t stream);

/* Bytes of a packed [N, K] weight matrix: N * (K / B) * block_bytes, or 0 for
 * an unknown codec or a K that is not a multiple of B. */
size_t m4q_weight_bytes(int codec, int64_t N, int64_t K);

/* NaN/Inf tripwire (the pages' "Releases" v0.3.0 bridge and the "v0.1 vs
 * v0.2 comparison" metrology table: a non-finite output is a hard failure).
 * Scans the device fp16 array x[n], synchronizes `stream` and returns
 * M4Q_ERR_NONFINITE if any element is NaN or +-Inf, M4Q_OK otherwise. */
int m4q_check_finite(const void* x, int64_t n, m4q_stream_t stream);

/* Synchronize `stream`, read and clear the current device's status word.
 * Returns M4Q_ERR_BOUNDS if, in a bounds-checked build, a kernel found an
 * index out of range since the last check (the site stays readable through
 * m4q_bounds_site until then), else M4Q_ERR_TIMEOUT if a kernel's bounded
 * pipeline wait gave up, else M4Q_OK. */
int m4q_check_device_status(m4q_stream_t stream);

/* Bounds-checked build (compiled with -DM4Q_BOUNDS=1, for tests): every
 * computed global access, every TMA coordinate and every computed
 * shared-memory staging offset of the projection and attention kernels is
 * tested against the extents the kernel was given before it is made; a
 * failing access is skipped and reported (M4Q_ERR_BOUNDS above) instead of
 * faulting.  m4q_build_flags() returns M4Q_BUILD_BOUNDS for such a build,
 * 0 for the normal one.  m4q_bounds_site() synchronizes `stream` and returns
 * the site number of the first failed check since the previous call (0: none;
 * the numbers are listed in the library source), clearing it; it returns
 * M4Q_ERR_CUDA (negative) if the status word cannot be read. */
#define M4Q_BUILD_BOUNDS 1
int m4q_build_flags(void);
int m4q_bounds_site(m4q_stream_t stream);

/* Self-test of the bounded wait: launches one block that waits on a barrier
 * nothing will complete, with a limit of `limit_ns` nanoseconds; the kernel
 * records the timeout in the status word and returns.  The caller then sees
 * M4Q_ERR_TIMEOUT from m4q_check_device_status().  Nothing faults or hangs. */
int m4q_selftest_wait_timeout(int64_t limit_ns, m4q_stream_t stream);

/* Human-readable text of a status code (static storage). */
const char* m4q_status_string(int status);

/* Library ABI version (major * 100 + minor). */
int m4q_version(void);

#ifdef __cplusplus
}
#endif

#endif /* M4Q_H_ */
