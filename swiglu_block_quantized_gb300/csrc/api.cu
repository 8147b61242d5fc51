// api.cu -- the C ABI declared in include/m4q.h: argument checks, path
// selection (GEMV for M <= 16, tcgen05 otherwise), TMA descriptor encoding
// and kernel launch on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include <cmath>
#include <mutex>

#include "../../include/m4q.h"
#include "launch.h"
#include "per_device.h"

namespace {

using m4q::ProjLaunch;

constexpr int kCodecs = 4;
constexpr int kBlock[kCodecs] = {32, 32, 128, 32};
constexpr int kBlockBytes[kCodecs] = {18, 34, 34, 20};
constexpr int kStageBytes[kCodecs] = {144, 272, 272, 160};    // bytes per packed stage

// Default limit of one device pipeline wait (ns); M4Q_WAIT_LIMIT_NS overrides.
unsigned long long wait_limit_ns() {
  static unsigned long long v = [] {
    const char* s = getenv("M4Q_WAIT_LIMIT_NS");
    unsigned long long x = s ? strtoull(s, nullptr, 10) : 0ull;
    return x ? x : 2000000000ull;
  }();
  return v;
}

// ------------------------------------------------------------ device facts

struct DevInfo {
  bool ok = false;
  bool sm103 = false;
  int sms = 0;
};

int current_device_info(DevInfo* out) {
  static std::mutex mu;
  static DevInfo cache[128];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return M4Q_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  DevInfo& d = cache[dev];
  if (!d.ok) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return M4Q_ERR_CUDA;
    d.sm103 = (major == 10 && minor == 3);
    d.sms = sms;
    d.ok = true;
  }
  *out = d;
  return M4Q_OK;
}

// ------------------------------------------------------------ tensor maps

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiledFn>(nullptr);
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// Cache of encoded tensor maps.  A map is a pure function of its
// description (element type, rank, base address, extents, pitches, box and
// swizzle), so a map found under an equal description is the one that
// encoding would produce, whatever happened to the memory in between; the
// cache holds no ownership of that memory.  Eager callers repeat the same
// few descriptions call after call (their weights and activation buffers),
// and a lookup costs far less than cuTensorMapEncodeTiled.  Direct-mapped,
// bounded, guarded by one mutex.
struct MapKey {
  uint32_t dt, rank, swz;
  uint64_t base;
  uint64_t dims[3], strides[2];
  uint32_t box[3];
  bool operator==(const MapKey& o) const {
    return dt == o.dt && rank == o.rank && swz == o.swz && base == o.base && dims[0] == o.dims[0] &&
           dims[1] == o.dims[1] && dims[2] == o.dims[2] && strides[0] == o.strides[0] &&
           strides[1] == o.strides[1] && box[0] == o.box[0] && box[1] == o.box[1] && box[2] == o.box[2];
  }
  uint64_t hash() const {
    uint64_t h = 0x9E3779B97F4A7C15ull;
    auto mix = [&h](uint64_t v) { h = (h ^ v) * 0xBF58476D1CE4E5B9ull; h ^= h >> 29; };
    mix(dt | ((uint64_t)rank << 8) | ((uint64_t)swz << 16));
    mix(base);
    for (int i = 0; i < 3; ++i) mix(dims[i]);
    for (int i = 0; i < 2; ++i) mix(strides[i]);
    mix(box[0] | ((uint64_t)box[1] << 20) | ((uint64_t)box[2] << 40));
    return h;
  }
};

struct MapSlot {
  bool used = false;
  MapKey key;
  CUtensorMap map;
};

constexpr int kMapSlots = 512;
std::mutex g_map_mu;
MapSlot g_maps[kMapSlots];

bool encode_cached(CUtensorMap* map, const MapKey& k, const cuuint32_t* estr, int rank) {
  const int slot = (int)(k.hash() % kMapSlots);
  {
    std::lock_guard<std::mutex> lock(g_map_mu);
    if (g_maps[slot].used && g_maps[slot].key == k) {
      *map = g_maps[slot].map;
      return true;
    }
  }
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {k.dims[0], k.dims[1], k.dims[2]};
  const cuuint64_t strides[2] = {k.strides[0], k.strides[1]};
  const cuuint32_t box[3] = {k.box[0], k.box[1], k.box[2]};
  if (fn(map, (CUtensorMapDataType)k.dt, rank, reinterpret_cast<void*>(k.base), dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, (CUtensorMapSwizzle)k.swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  std::lock_guard<std::mutex> lock(g_map_mu);
  g_maps[slot].used = true;
  g_maps[slot].key = k;
  g_maps[slot].map = *map;
  return true;
}

// 2-D map: inner extent `inner` elements, `outer` rows, row pitch in bytes.
bool encode_2d(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t inner,
               uint64_t outer, uint64_t pitch_bytes, uint32_t box_inner, uint32_t box_outer,
               CUtensorMapSwizzle swz) {
  MapKey k{};
  k.dt = (uint32_t)dt;
  k.rank = 2;
  k.swz = (uint32_t)swz;
  k.base = reinterpret_cast<uint64_t>(base);
  k.dims[0] = inner;
  k.dims[1] = outer;
  k.strides[0] = pitch_bytes;
  k.box[0] = box_inner;
  k.box[1] = box_outer;
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_cached(map, k, estr, 2);
}

// Head-major Y [N / hd][M][hd] as a 3-D tensor (d, m, head), boxes of
// [128 / hd heads][32 m][hd] (one staged GEMM chunk of 128 outputs).
bool encode_heads(CUtensorMap* map, const void* base, uint64_t M, uint64_t N, uint32_t hd) {
  MapKey k{};
  k.dt = (uint32_t)CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  k.rank = 3;
  k.swz = (uint32_t)CU_TENSOR_MAP_SWIZZLE_NONE;
  k.base = reinterpret_cast<uint64_t>(base);
  k.dims[0] = hd;
  k.dims[1] = M;
  k.dims[2] = N / hd;
  k.strides[0] = (uint64_t)hd * 2;
  k.strides[1] = (uint64_t)M * hd * 2;
  k.box[0] = hd;
  k.box[1] = 32;
  k.box[2] = 128 / hd;
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_cached(map, k, estr, 3);
}

// ------------------------------------------------------------ validation

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool known_codec(int codec) { return codec >= 0 && codec < kCodecs; }

int check_shape(int codec, int64_t M, int64_t N, int64_t K) {
  if (!known_codec(codec)) return M4Q_ERR_UNSUPPORTED_CODEC;
  if (M < 1 || N < 1 || K < 1) return M4Q_ERR_INVALID_ARG;
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return M4Q_ERR_INVALID_ARG;
  if (K % kBlock[codec] != 0 || N % 8 != 0) return M4Q_ERR_BAD_SHAPE;
  return M4Q_OK;
}

// ------------------------------------------------------------ host pipeline

// Events of m4q_project_host: per device, recorded and waited in stream
// order, so one pool serves every call; calls enqueue one at a time.
constexpr int kHostChunks = 16;
constexpr int kMaxEventDevices = 64;
struct HostEvents {
  bool ready = false;
  cudaEvent_t e[2 * kHostChunks + 2];
};
HostEvents g_host_events[kMaxEventDevices];
std::mutex g_host_mu[kMaxEventDevices];

// ------------------------------------------------------------ dispatch

int project(const void* X, const void* W0, const void* W1, int codec, int64_t M, int64_t N,
            int64_t K, void* Y, int path, bool swiglu, int act, m4q_stream_t stream,
            int64_t head_dim = 0) {
  if (!X || !W0 || !Y || (swiglu && !W1)) return M4Q_ERR_INVALID_ARG;
  if (act != M4Q_ACT_SILU && act != M4Q_ACT_GELU) return M4Q_ERR_INVALID_ARG;
  if (head_dim != 0 && (swiglu || (head_dim != 64 && head_dim != 128))) return M4Q_ERR_INVALID_ARG;
  if (head_dim != 0 && N % head_dim != 0) return M4Q_ERR_BAD_SHAPE;
  int rc = check_shape(codec, M, N, K);
  if (rc != M4Q_OK) return rc;
  if (path < M4Q_PATH_AUTO || path > M4Q_PATH_TC) return M4Q_ERR_INVALID_ARG;
  if (path == M4Q_PATH_GEMV && M > 16) return M4Q_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(W0) || !aligned16(Y) || (swiglu && !aligned16(W1)))
    return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  rc = current_device_info(&dev);
  if (rc != M4Q_OK) return rc;
  if (!dev.sm103) return M4Q_ERR_UNSUPPORTED_DEVICE;

  ProjLaunch L{};
  L.x = X;
  L.w0 = W0;
  L.w1 = swiglu ? W1 : nullptr;
  L.y = Y;
  L.M = (int)M;
  L.N = (int)N;
  L.K = (int)K;
  L.row_bytes = (K / kBlock[codec]) * (long long)kBlockBytes[codec];
  L.swiglu = swiglu;
  L.act = act;
  L.head_dim = (int)head_dim;
  // Rows that are 16-byte multiples move by TMA.  For the 18- and 34-byte
  // blocks that makes K a multiple of the packed stage; for MLX4 (20-byte
  // blocks) a multiple of 128, and the TMA box of the last stage of a row
  // then reads past the row end, which it fills with zeros (zero scale and
  // bias: zero weights, multiplied by zero-filled X columns).
  L.wtma = (L.row_bytes % 16) == 0;
  L.status = m4q::status_words();
  if (!L.status) return M4Q_ERR_CUDA;
  L.limit_ns = wait_limit_ns();
  L.stream = reinterpret_cast<cudaStream_t>(stream);

  const bool gemv = (path == M4Q_PATH_GEMV) || (path == M4Q_PATH_AUTO && M <= 16);
  cudaError_t e;
  if (gemv) {
    L.mt = M <= 8 ? 1 : 2;
    L.sms = dev.sms;
    e = m4q::launch_gemv(codec, L);
  } else {
    // Output tiles along N (64 outputs per tile for the gated projections).
    const int64_t out_rows = swiglu ? 64 : 128;
    const int64_t ntiles = (N + out_rows - 1) / out_rows;
    // M <= 128 with TMA-able rows and row-major output: the small-M kernel
    // (one activation tile of 128 rows as the A operand).
    // (Not for a plain GEMM with 272-byte packed stages above M = 64: its
    // 128-row X stages and 128-output Y tile do not fit shared memory.)
    L.small = L.wtma && head_dim == 0 && M <= 128 && !(kStageBytes[codec] > 160 && !swiglu && M > 64);
    int nx = 64;
    L.split = 1;
    if (L.small) {
      nx = M <= 32 ? 32 : (M <= 64 ? 64 : 128);   // X rows per stage of the small-M kernel
      // Few output tiles leave most SMs idle: split K over a cluster of up
      // to 8 CTAs per tile, each CTA taking a whole number of packed
      // stages, as long as every cluster of the grid can be resident at
      // once (clusters must fit inside one GPC, so fewer clusters of 8 than
      // SMs / 8 fit the GPU).
      const int64_t tiles = (N + out_rows - 1) / out_rows;
      const int64_t npk = (K + 8 * kBlock[codec] - 1) / (8 * kBlock[codec]);   // packed stages
      L.split = 8;
      while (L.split > 1 && (npk % L.split != 0 || tiles * L.split > dev.sms)) L.split /= 2;
    } else if (!L.wtma) {
      nx = 128;
    } else {
      // Tile width and K split with the least estimated time.  The
      // persistent CTAs take ceil(tiles / SMs) tiles each; a tile costs its
      // 64-k sub-steps (divided by the split) times a width factor, since a
      // sub-step costs about the same at every width except 256, about 12%
      // more (measured on the 8B, 1B and Q2_0 shapes); a split adds its
      // cross-CTA reduction, about 2.5 sub-steps.  Ties go to the wider tile
      // (less decode per FLOP).  A split needs every cluster of the grid
      // resident at once: tiles * split <= SMs here, and the launcher halves
      // it further if clusters of that size do not all fit.
      const int64_t nks = (K + 63) / 64;
      const int64_t npk = (K + 8 * kBlock[codec] - 1) / (8 * kBlock[codec]);   // packed stages
      double best = 1e300;
      for (int w = 256; w >= 64; w /= 2) {
        const int64_t t = ((M + w - 1) / w) * ntiles;
        for (int sp = 1; sp <= 8; sp *= 2) {
          if (sp > 1 && (w > 128 || head_dim != 0 || npk % sp != 0 || t * sp > dev.sms)) continue;
          const double waves = (double)((t * sp + dev.sms - 1) / dev.sms);
          const double est = waves * (double)nks / sp * (w == 256 ? 1.12 : 1.0) + (sp > 1 ? 2.5 : 0.0);
          if (est < best - 1e-9) {
            best = est;
            nx = w;
            L.split = sp;
          }
        }
      }
    }
    L.nx = nx;
    L.sms = dev.sms;
    if (!encode_2d(&L.tm_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, X, K, M, K * 2, 64, nx,
                   CU_TENSOR_MAP_SWIZZLE_128B))
      return M4Q_ERR_CUDA;
    // Y boxes: GEMM stages [32 m][128 n] chunks per warpgroup; SwiGLU stores
    // one [nx/2 m][16 n] slab per epilogue warp.
    if (L.small) {
      // [128 m][64 n] boxes in the 128-byte swizzled layout
      if (!encode_2d(&L.tm_y, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, Y, N, M, N * 2, 64, 128,
                     CU_TENSOR_MAP_SWIZZLE_128B))
        return M4Q_ERR_CUDA;
    } else if (head_dim != 0) {
      if (!encode_heads(&L.tm_y, Y, M, N, (uint32_t)head_dim)) return M4Q_ERR_CUDA;
    } else if (!encode_2d(&L.tm_y, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, Y, N, M, N * 2,
                          swiglu ? 16u : (uint32_t)out_rows, swiglu ? (uint32_t)(nx / 2) : 32u,
                          CU_TENSOR_MAP_SWIZZLE_NONE)) {
      return M4Q_ERR_CUDA;
    }
    L.tm_w0 = L.tm_x;
    L.tm_w1 = L.tm_x;
    if (L.wtma) {
      const uint32_t box_rows = swiglu ? 64 : 128;
      if (!encode_2d(&L.tm_w0, CU_TENSOR_MAP_DATA_TYPE_UINT16, W0, L.row_bytes / 2, N,
                     L.row_bytes, kStageBytes[codec] / 2, box_rows, CU_TENSOR_MAP_SWIZZLE_NONE))
        return M4Q_ERR_CUDA;
      if (swiglu && !encode_2d(&L.tm_w1, CU_TENSOR_MAP_DATA_TYPE_UINT16, W1, L.row_bytes / 2, N,
                               L.row_bytes, kStageBytes[codec] / 2, box_rows,
                               CU_TENSOR_MAP_SWIZZLE_NONE))
        return M4Q_ERR_CUDA;
    }
    switch (codec) {
      case M4Q_Q4_0: e = m4q::launch_tc_q4_0(L); break;
      case M4Q_Q8_0: e = m4q::launch_tc_q8_0(L); break;
      case M4Q_MLX4: e = m4q::launch_tc_mlx4(L); break;
      default: e = m4q::launch_tc_q2_0(L); break;
    }
  }
  return e == cudaSuccess ? M4Q_OK : M4Q_ERR_CUDA;
}

}  // namespace

extern "C" {

int m4q_gemm_ex(const void* X, const void* W, int codec, int64_t M, int64_t N, int64_t K, void* Y,
                int path, m4q_stream_t stream) {
  return project(X, W, nullptr, codec, M, N, K, Y, path, false, M4Q_ACT_SILU, stream);
}

int m4q_swiglu_ex(const void* X, const void* Wg, const void* Wu, int codec, int64_t M, int64_t N,
                  int64_t K, void* Y, int path, m4q_stream_t stream) {
  return project(X, Wg, Wu, codec, M, N, K, Y, path, true, M4Q_ACT_SILU, stream);
}

int m4q_gemm_heads(const void* X, const void* W, int codec, int64_t M, int64_t N, int64_t K,
                   int64_t head_dim, void* Y, m4q_stream_t stream) {
  if (head_dim == 0) return M4Q_ERR_INVALID_ARG;
  return project(X, W, nullptr, codec, M, N, K, Y, M4Q_PATH_AUTO, false, M4Q_ACT_SILU, stream, head_dim);
}

int m4q_glu_ex(const void* X, const void* Wg, const void* Wu, int codec, int64_t M, int64_t N,
               int64_t K, void* Y, int act, int path, m4q_stream_t stream) {
  return project(X, Wg, Wu, codec, M, N, K, Y, path, true, act, stream);
}

int m4q_geglu(const void* X, const void* Wg, const void* Wu, int codec, int64_t M, int64_t N,
              int64_t K, void* Y, m4q_stream_t stream) {
  return project(X, Wg, Wu, codec, M, N, K, Y, M4Q_PATH_AUTO, true, M4Q_ACT_GELU, stream);
}

int m4q_gemm(const void* X, const void* W, int codec, int64_t M, int64_t N, int64_t K, void* Y,
             m4q_stream_t stream) {
  return project(X, W, nullptr, codec, M, N, K, Y, M4Q_PATH_AUTO, false, M4Q_ACT_SILU, stream);
}

int m4q_swiglu(const void* X, const void* Wg, const void* Wu, int codec, int64_t M, int64_t N,
               int64_t K, void* Y, m4q_stream_t stream) {
  return project(X, Wg, Wu, codec, M, N, K, Y, M4Q_PATH_AUTO, true, M4Q_ACT_SILU, stream);
}

int m4q_mlp(const void* X, const void* Wg, const void* Wu, const void* Wd, int codec_gu,
            int codec_d, int64_t M, int64_t D, int64_t F, void* H, void* Y, int act,
            m4q_stream_t stream) {
  if (!H || !Wd) return M4Q_ERR_INVALID_ARG;
  // Validate both projections before enqueueing either.
  int rc = check_shape(codec_gu, M, F, D);
  if (rc != M4Q_OK) return rc;
  rc = check_shape(codec_d, M, D, F);
  if (rc != M4Q_OK) return rc;
  if (!aligned16(H) || !aligned16(Wd)) return M4Q_ERR_MISALIGNED;
  rc = project(X, Wg, Wu, codec_gu, M, F, D, H, M4Q_PATH_AUTO, true, act, stream);
  if (rc != M4Q_OK) return rc;
  return project(H, Wd, nullptr, codec_d, M, D, F, Y, M4Q_PATH_AUTO, false, M4Q_ACT_SILU, stream);
}

int m4q_project_host(const void* X_host, const void* W0, const void* W1, int codec, int act, int64_t M,
                     int64_t N, int64_t K, void* Y_host, void* X_dev, void* Y_dev, int64_t chunk_rows,
                     m4q_stream_t stream, m4q_stream_t h2d_stream, m4q_stream_t d2h_stream) {
  if (!X_host || !Y_host || !X_dev || !Y_dev || !W0 || chunk_rows < 0) return M4Q_ERR_INVALID_ARG;
  if (act != M4Q_ACT_SILU && act != M4Q_ACT_GELU) return M4Q_ERR_INVALID_ARG;
  int rc = check_shape(codec, M, N, K);
  if (rc != M4Q_OK) return rc;
  if (!aligned16(X_dev) || !aligned16(Y_dev) || !aligned16(W0) || (W1 && !aligned16(W1)))
    return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  rc = current_device_info(&dev);
  if (rc != M4Q_OK) return rc;
  if (!dev.sm103) return M4Q_ERR_UNSUPPORTED_DEVICE;
  int64_t rows = chunk_rows ? chunk_rows : ((M + 3) / 4 + 127) / 128 * 128;
  if (rows > M) rows = M;
  const int64_t chunks = (M + rows - 1) / rows;
  if (chunks > kHostChunks) rows = (M + kHostChunks - 1) / kHostChunks;   // at most kHostChunks chunks
  int dev_id = 0;
  if (cudaGetDevice(&dev_id) != cudaSuccess || dev_id < 0 || dev_id >= kMaxEventDevices) return M4Q_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_host_mu[dev_id]);
  HostEvents& ev = g_host_events[dev_id];
  if (!ev.ready) {
    for (int i = 0; i < 2 * kHostChunks + 2; ++i)
      if (cudaEventCreateWithFlags(&ev.e[i], cudaEventDisableTiming) != cudaSuccess) {
        (void)cudaGetLastError();
        return M4Q_ERR_CUDA;
      }
    ev.ready = true;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaStream_t sin = reinterpret_cast<cudaStream_t>(h2d_stream);
  cudaStream_t sout = reinterpret_cast<cudaStream_t>(d2h_stream);
  auto fail = [] { return M4Q_ERR_CUDA; };
  // Both copy streams start after the work already on `stream`.
  if (cudaEventRecord(ev.e[0], s) != cudaSuccess || cudaStreamWaitEvent(sin, ev.e[0], 0) != cudaSuccess ||
      cudaStreamWaitEvent(sout, ev.e[0], 0) != cudaSuccess)
    return fail();
  const uint8_t* xh = static_cast<const uint8_t*>(X_host);
  uint8_t* yh = static_cast<uint8_t*>(Y_host);
  uint8_t* xd = static_cast<uint8_t*>(X_dev);
  uint8_t* yd = static_cast<uint8_t*>(Y_dev);
  int c = 0;
  for (int64_t r0 = 0; r0 < M; r0 += rows, ++c) {
    const int64_t n = (M - r0) < rows ? (M - r0) : rows;
    const size_t xoff = (size_t)(r0 * K * 2), yoff = (size_t)(r0 * N * 2);
    cudaEvent_t in = ev.e[1 + 2 * c], done = ev.e[2 + 2 * c];
    if (cudaMemcpyAsync(xd + xoff, xh + xoff, (size_t)(n * K * 2), cudaMemcpyHostToDevice, sin) != cudaSuccess ||
        cudaEventRecord(in, sin) != cudaSuccess || cudaStreamWaitEvent(s, in, 0) != cudaSuccess)
      return fail();
    rc = project(xd + xoff, W0, W1, codec, n, N, K, yd + yoff, M4Q_PATH_AUTO, W1 != nullptr, act, stream);
    if (rc != M4Q_OK) return rc;
    if (cudaEventRecord(done, s) != cudaSuccess || cudaStreamWaitEvent(sout, done, 0) != cudaSuccess ||
        cudaMemcpyAsync(yh + yoff, yd + yoff, (size_t)(n * N * 2), cudaMemcpyDeviceToHost, sout) != cudaSuccess)
      return fail();
  }
  cudaEvent_t last = ev.e[2 * kHostChunks + 1];
  if (cudaEventRecord(last, sout) != cudaSuccess || cudaStreamWaitEvent(s, last, 0) != cudaSuccess) return fail();
  return M4Q_OK;
}

size_t m4q_weight_bytes(int codec, int64_t N, int64_t K) {
  if (!known_codec(codec) || N < 0 || K < 0 || K % kBlock[codec] != 0) return 0;
  return (size_t)N * (size_t)(K / kBlock[codec]) * (size_t)kBlockBytes[codec];
}

int m4q_dequant(const void* W, int codec, int64_t N, int64_t K, void* Wf16, m4q_stream_t stream) {
  if (!W || !Wf16) return M4Q_ERR_INVALID_ARG;
  if (!known_codec(codec)) return M4Q_ERR_UNSUPPORTED_CODEC;
  if (N < 1 || K < 1 || N > INT32_MAX || K > INT32_MAX) return M4Q_ERR_INVALID_ARG;
  if (K % kBlock[codec] != 0) return M4Q_ERR_BAD_SHAPE;
  if (!aligned16(W) || !aligned16(Wf16)) return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  int rc = current_device_info(&dev);
  if (rc != M4Q_OK) return rc;
  if (!dev.sm103) return M4Q_ERR_UNSUPPORTED_DEVICE;
  const long long row_bytes = (K / kBlock[codec]) * (long long)kBlockBytes[codec];
  return m4q::launch_dequant(codec, W, (int)N, (int)K, row_bytes, Wf16,
                             reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? M4Q_OK
             : M4Q_ERR_CUDA;
}

int m4q_mlx4_pack(const void* words, const void* scales, const void* biases, int64_t N, int64_t K,
                  void* W, m4q_stream_t stream) {
  if (!words || !scales || !biases || !W) return M4Q_ERR_INVALID_ARG;
  if (N < 1 || K < 1 || N > INT32_MAX || K > INT32_MAX) return M4Q_ERR_INVALID_ARG;
  if (K % 32 != 0) return M4Q_ERR_BAD_SHAPE;
  if (!aligned16(words) || !aligned16(W) || (reinterpret_cast<uintptr_t>(scales) & 1u) ||
      (reinterpret_cast<uintptr_t>(biases) & 1u))
    return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  int rc = current_device_info(&dev);
  if (rc != M4Q_OK) return rc;
  if (!dev.sm103) return M4Q_ERR_UNSUPPORTED_DEVICE;
  return m4q::launch_mlx4_pack(words, scales, biases, (int)N, (int)K, W, dev.sms,
                               reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? M4Q_OK
             : M4Q_ERR_CUDA;
}

int m4q_repack(const void* W, int codec, int64_t N, int64_t K, void* Wplanar, m4q_stream_t stream) {
  if (!W || !Wplanar) return M4Q_ERR_INVALID_ARG;
  if (!known_codec(codec)) return M4Q_ERR_UNSUPPORTED_CODEC;
  if (N < 1 || K < 1 || N > INT32_MAX || K > INT32_MAX) return M4Q_ERR_INVALID_ARG;
  if (K % kBlock[codec] != 0) return M4Q_ERR_BAD_SHAPE;
  if (!aligned16(W) || !aligned16(Wplanar)) return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  int rc = current_device_info(&dev);
  if (rc != M4Q_OK) return rc;
  if (!dev.sm103) return M4Q_ERR_UNSUPPORTED_DEVICE;
  const long long blocks = N * (K / kBlock[codec]);
  return m4q::launch_repack(codec, W, blocks, Wplanar, dev.sms, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? M4Q_OK
             : M4Q_ERR_CUDA;
}

// ------------------------------------------------------------ attention

}  // extern "C"

namespace {

// Key split of an attention call: CTAs = row tiles x KV heads; when that
// leaves the GPU under `per_sm` CTAs per SM (what the tiled kernel fits:
// two, for its registers or, decoding over an fp16 cache, its three-stage
// tile pipeline; three for the decode kernel over a Q8_0 cache), split the
// keys (tiles of 64) so the grid reaches about that, each split keeping at
// least two tiles.
struct AttnSplit {
  int rtiles, nsplit, tsplit;
  size_t ws_bytes;
};

AttnSplit attn_split(int64_t H, int64_t Hkv, int64_t M, int64_t T, int64_t D, int sms, int per_sm) {
  AttnSplit a;
  const int64_t R = M * (H / Hkv);
  a.rtiles = (int)((R + 63) / 64);
  const int64_t ctas = (int64_t)a.rtiles * Hkv;
  const int64_t ktiles = (T + 63) / 64;
  const int64_t target = (int64_t)per_sm * sms;
  int64_t ns = 1;
  if (ctas < target) {
    ns = (target + ctas - 1) / ctas;
    const int64_t most = ktiles / 2 > 1 ? ktiles / 2 : 1;
    if (ns > most) ns = most;
  }
  const int64_t per = (ktiles + ns - 1) / ns;     // key tiles per split
  a.tsplit = (int)(per * 64);
  a.nsplit = (int)((ktiles + per - 1) / per);
  a.ws_bytes = a.nsplit > 1 ? (size_t)a.nsplit * Hkv * a.rtiles * 64 * (size_t)(D * 4 + 8) : 0;
  return a;
}

// [heads][rows][D] fp16 as a 3-D tensor (d, row, head), boxes of
// [1][box_rows][64 d] with the 128-byte swizzle: the tcgen05 attention's Q,
// K and V tiles (rows past the extent read as zeros).
bool encode_kv(CUtensorMap* map, const void* base, uint64_t Hkv, uint64_t T, uint64_t D, uint32_t box_rows = 128) {
  MapKey k{};
  k.dt = (uint32_t)CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  k.rank = 3;
  k.swz = (uint32_t)CU_TENSOR_MAP_SWIZZLE_128B;
  k.base = reinterpret_cast<uint64_t>(base);
  k.dims[0] = D;
  k.dims[1] = T;
  k.dims[2] = Hkv;
  k.strides[0] = D * 2;
  k.strides[1] = T * D * 2;
  k.box[0] = 64;
  k.box[1] = box_rows;
  k.box[2] = 1;
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_cached(map, k, estr, 3);
}

// A Q8_0 cache can take the tcgen05 path after both caches are decoded to
// fp16 once (each key tile is read by every row tile of its KV head, so one
// decode replaces many): the staging needs 2 Hkv T D fp16 values.  False
// when the shape cannot take that path.
bool q8_staging_bytes(int64_t H, int64_t Hkv, int64_t M, int64_t T, int64_t D, size_t* bytes) {
  if (H < 1 || Hkv < 1 || M < 1 || T < 1 || H % Hkv != 0 || (D != 64 && D != 128)) return false;
  if (Hkv * T > INT32_MAX || M * (H / Hkv) > INT32_MAX) return false;
  m4q::AttnParams p{};
  p.H = (int)H;
  p.Hkv = (int)Hkv;
  p.G = (int)(H / Hkv);
  p.M = (int)M;
  p.D = (int)D;
  p.kv_row_bytes = 2 * D;
  if (!m4q::attention_tc_shape(p)) return false;
  *bytes = (size_t)2 * Hkv * T * D * 2;
  return true;
}

int check_attention(const void* Q, const void* K, const void* V, int kv_codec, int64_t H, int64_t Hkv,
                    int64_t M, int64_t T, int64_t D, int64_t q_offset, float scale, const void* O) {
  if (!Q || !K || !V || !O) return M4Q_ERR_INVALID_ARG;
  if (kv_codec != M4Q_KV_F16 && kv_codec != M4Q_Q8_0) return M4Q_ERR_UNSUPPORTED_CODEC;
  if (H < 1 || Hkv < 1 || M < 1 || T < 1 || q_offset < 0) return M4Q_ERR_INVALID_ARG;
  if (H > 65535 || M > INT32_MAX || T > INT32_MAX || q_offset > INT32_MAX || M * H > INT32_MAX)
    return M4Q_ERR_INVALID_ARG;
  if (!(scale == scale) || scale == INFINITY || scale == -INFINITY) return M4Q_ERR_INVALID_ARG;
  if (H % Hkv != 0 || (D != 64 && D != 128)) return M4Q_ERR_BAD_SHAPE;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return M4Q_ERR_MISALIGNED;
  return M4Q_OK;
}

}  // namespace

extern "C" {

size_t m4q_attention_workspace_bytes(int64_t H, int64_t Hkv, int64_t M, int64_t T, int64_t D) {
  if (H < 1 || Hkv < 1 || M < 1 || T < 1 || H % Hkv != 0 || (D != 64 && D != 128)) return 0;
  DevInfo dev;
  if (current_device_info(&dev) != M4Q_OK) return 0;
  // the larger of the two codecs' splits (a Q8_0 decode splits into more)
  return attn_split(H, Hkv, M, T, D, dev.sms, M * (H / Hkv) <= 16 ? 3 : 2).ws_bytes;
}

size_t m4q_attention_workspace(int kv_codec, int64_t H, int64_t Hkv, int64_t M, int64_t T, int64_t D) {
  // the path is chosen per call (the causal offset enters the estimate), so
  // the size covers both: the key split's results and a Q8_0 staging
  const size_t split = m4q_attention_workspace_bytes(H, Hkv, M, T, D);
  size_t stage = 0;
  if (kv_codec != M4Q_Q8_0 || !q8_staging_bytes(H, Hkv, M, T, D, &stage)) return split;
  return stage > split ? stage : split;
}

int m4q_attention(const void* Q, const void* K, const void* V, int kv_codec, int64_t H, int64_t Hkv,
                  int64_t M, int64_t T, int64_t D, int64_t q_offset, int causal, float scale, void* O,
                  void* workspace, size_t workspace_bytes, m4q_stream_t stream) {
  int rc = check_attention(Q, K, V, kv_codec, H, Hkv, M, T, D, q_offset, scale, O);
  if (rc != M4Q_OK) return rc;
  if (workspace && !aligned16(workspace)) return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  rc = current_device_info(&dev);
  if (rc != M4Q_OK) return rc;
  if (!dev.sm103) return M4Q_ERR_UNSUPPORTED_DEVICE;
  AttnSplit a = attn_split(H, Hkv, M, T, D, dev.sms, (M * (H / Hkv) <= 16 && kv_codec == M4Q_Q8_0) ? 3 : 2);
  if (a.nsplit > 1 && (!workspace || workspace_bytes < a.ws_bytes)) {
    a.nsplit = 1;   // no room for partial results: one CTA walks all keys
    a.tsplit = (int)(((T + 63) / 64) * 64);
  }
  m4q::AttnParams p{};
  p.q = static_cast<const __half*>(Q);
  p.k = static_cast<const uint8_t*>(K);
  p.v = static_cast<const uint8_t*>(V);
  p.o = static_cast<__half*>(O);
  p.H = (int)H;
  p.Hkv = (int)Hkv;
  p.G = (int)(H / Hkv);
  p.M = (int)M;
  p.T = (int)T;
  p.D = (int)D;
  p.kv_row_bytes = kv_codec == M4Q_KV_F16 ? 2 * D : (D / 32) * 34;
  p.kv_vec16 = (T * p.kv_row_bytes) % 16 == 0;   // K and V are 16-byte aligned (checked above)
  p.q_offset = (int)q_offset;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.rtiles = a.rtiles;
  p.nsplit = a.nsplit;
  p.tsplit = a.tsplit;
  p.status = m4q::status_words();
  if (!p.status) return M4Q_ERR_CUDA;
  p.nsm = dev.sms;
  if (a.nsplit > 1) {
    p.ws_o = static_cast<float*>(workspace);
    p.ws_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) +
                                         (size_t)a.nsplit * Hkv * a.rtiles * 64 * D * 4);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  size_t stage = 0;
  m4q::AttnParams pf = p;   // the same call on an fp16 cache (the staged form)
  pf.kv_row_bytes = 2 * D;
  if (kv_codec == M4Q_Q8_0 && workspace && q8_staging_bytes(H, Hkv, M, T, D, &stage) && workspace_bytes >= stage &&
      m4q::attention_tc_applies(pf, true)) {
    // decode both caches to fp16 in the workspace, then the fp16 path
    __half* kf = static_cast<__half*>(workspace);
    __half* vf = kf + (size_t)Hkv * T * D;
    if (m4q::launch_kv_q8_stage(K, V, (long long)Hkv * T, (int)D, kf, vf, s) != cudaSuccess) return M4Q_ERR_CUDA;
    K = kf;
    V = vf;
    p.k = reinterpret_cast<const uint8_t*>(kf);
    p.v = reinterpret_cast<const uint8_t*>(vf);
    p.kv_row_bytes = 2 * D;
    p.kv_vec16 = true;
    kv_codec = M4Q_KV_F16;
  }
  if (kv_codec == M4Q_KV_F16 && m4q::attention_tc_applies(p, false)) {
    // Q [H][M][D] takes the same form as the caches, in boxes of the
    // 128 / G queries a CTA takes of each head
    CUtensorMap tm_q, tm_k, tm_v;
    if (!encode_kv(&tm_q, Q, H, M, D, (uint32_t)(128 / p.G)) || !encode_kv(&tm_k, K, Hkv, T, D) ||
        !encode_kv(&tm_v, V, Hkv, T, D))
      return M4Q_ERR_CUDA;
    return m4q::launch_attention_tc(p, tm_q, tm_k, tm_v, s) == cudaSuccess ? M4Q_OK : M4Q_ERR_CUDA;
  }
  return m4q::launch_attention(p, kv_codec == M4Q_Q8_0, s) == cudaSuccess ? M4Q_OK : M4Q_ERR_CUDA;
}

// ------------------------------------------------------------ rotary positions, KV cache, norms

}  // extern "C"

namespace {

bool stride_ok(int64_t s) { return s % 8 == 0; }

// A batch of caches [B][Hkv][C] rows of D values.
int check_cache(int kv_codec, int64_t B, int64_t Hkv, int64_t C, int64_t D) {
  if (kv_codec != M4Q_KV_F16 && kv_codec != M4Q_Q8_0) return M4Q_ERR_UNSUPPORTED_CODEC;
  if (B < 1 || Hkv < 1 || C < 1) return M4Q_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return M4Q_ERR_BAD_SHAPE;
  if (B > INT32_MAX || Hkv > 65535 || C > INT32_MAX || B > INT32_MAX / (Hkv * C)) return M4Q_ERR_BAD_SHAPE;
  if (kv_codec == M4Q_Q8_0 && (B * Hkv * C * (D / 32 * 34)) % 16 != 0) return M4Q_ERR_BAD_SHAPE;
  return M4Q_OK;
}

int check_turn(const int32_t* pos, int64_t D, int64_t rot, int layout, float mscale) {
  if (!pos || (layout != M4Q_ROPE_HALF && layout != M4Q_ROPE_INTERLEAVED) || !(mscale - mscale == 0.f))
    return M4Q_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return M4Q_ERR_BAD_SHAPE;
  if (rot < 16 || rot > D || rot % 16 != 0) return M4Q_ERR_BAD_SHAPE;
  return M4Q_OK;
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The device's facts and status word, for the launches below (asked for once a device).
int ready(DevInfo* dev, uint32_t** status) {
  struct Facts {
    DevInfo dev;
    uint32_t* status = nullptr;
  };
  static m4q::PerDevice<Facts, 128> all;
  int id = 0;
  if (cudaGetDevice(&id) != cudaSuccess || id < 0 || id >= 128) return M4Q_ERR_CUDA;
  Facts f;
  const int rc = all.get(id, &f, [](Facts* k) -> int {
    const int e = current_device_info(&k->dev);
    if (e != M4Q_OK) return e;
    if (!k->dev.sm103) return M4Q_ERR_UNSUPPORTED_DEVICE;
    k->status = m4q::status_words();
    return k->status ? M4Q_OK : M4Q_ERR_CUDA;
  });
  if (rc != M4Q_OK) return rc;
  *dev = f.dev;
  *status = f.status;
  return M4Q_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? M4Q_OK : M4Q_ERR_CUDA; }

}  // namespace

extern "C" {

int m4q_rope_freqs(int64_t rot, double base, int scaling, double factor, double original, double low, double high,
                   int64_t* freqs, float* mscale) {
  if (!freqs || rot < 2 || rot % 2 != 0 || rot > 1 << 20) return M4Q_ERR_INVALID_ARG;
  if (scaling < M4Q_ROPE_PLAIN || scaling > M4Q_ROPE_YARN) return M4Q_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor)) return M4Q_ERR_INVALID_ARG;
  const bool bands = scaling == M4Q_ROPE_BANDS || scaling == M4Q_ROPE_YARN;
  if (bands && !(original > 0.0 && std::isfinite(original) && low >= 0.0 && high > low && std::isfinite(high)))
    return M4Q_ERR_INVALID_ARG;
  if (scaling == M4Q_ROPE_NTK) {
    if (rot == 2) return M4Q_ERR_INVALID_ARG;
    base *= std::pow(factor, (double)rot / (double)(rot - 2));
    if (!std::isfinite(base)) return M4Q_ERR_INVALID_ARG;
  }
  constexpr double kTurn = 6.283185307179586;
  for (int64_t i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * (double)i / (double)rot);
    if (scaling == M4Q_ROPE_LINEAR) f /= factor;
    if (bands) {
      const double r = original * f / kTurn;
      const double keep = r <= low ? 0.0 : r >= high ? 1.0 : (r - low) / (high - low);
      f = (1.0 - keep) * f / factor + keep * f;
    }
    freqs[i] = (int64_t)std::llround(std::ldexp(f / kTurn, 64));   // f <= 1: below 2^62
  }
  if (mscale) *mscale = scaling == M4Q_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return M4Q_OK;
}

}  // extern "C"

namespace {

// One axis: A = 1 and axes NULL.
int rope_call(const void* X, int64_t x_head_stride, int64_t x_row_stride, int64_t H, int64_t M, int64_t D,
              const int32_t* pos, int64_t A, const int64_t* freqs, const int32_t* axes, int64_t rot, int layout,
              float mscale, void* Y, int64_t y_head_stride, int64_t y_row_stride, m4q_stream_t stream) {
  if (!X || !Y || !freqs || A < 1 || A > M4Q_ROPE_MAX_AXES) return M4Q_ERR_INVALID_ARG;
  if (H < 1 || M < 1 || H > 65535 || M > INT32_MAX) return M4Q_ERR_INVALID_ARG;
  int rc = check_turn(pos, D, rot, layout, mscale);
  if (rc != M4Q_OK) return rc;
  if (!aligned_to(axes, 4)) return M4Q_ERR_MISALIGNED;
  if (!aligned16(X) || !aligned16(Y) || !aligned_to(pos, 4) || !aligned_to(freqs, 8) || !stride_ok(x_head_stride) ||
      !stride_ok(x_row_stride) || !stride_ok(y_head_stride) || !stride_ok(y_row_stride))
    return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  m4q::KvOpsParams p{};
  rc = ready(&dev, &p.status);
  if (rc != M4Q_OK) return rc;
  p.q = {static_cast<const __half*>(X), x_head_stride, x_row_stride};
  p.qo = static_cast<__half*>(Y);
  p.qo_hs = y_head_stride;
  p.qo_rs = y_row_stride;
  p.H = (int)H;
  p.M = (int)M;
  p.D = (int)D;
  p.pos = pos;
  p.freqs = freqs;
  p.axes = axes;
  p.A = (int)A;
  p.rot = (int)rot;
  p.interleaved = layout == M4Q_ROPE_INTERLEAVED;
  p.mscale = mscale;
  p.nsm = dev.sms;
  return done(m4q::launch_rope_kv(p, false, reinterpret_cast<cudaStream_t>(stream)));
}

int kv_write_call(const void* K, int64_t k_head_stride, int64_t k_row_stride, const void* V, int64_t v_head_stride,
                  int64_t v_row_stride, int64_t Hkv, int64_t M, int64_t D, const int32_t* pos, int64_t A,
                  const int64_t* freqs, const int32_t* axes, int64_t rot, int layout, float mscale,
                  const int32_t* slots, void* Kc, void* Vc, int kv_codec, int64_t B, int64_t C, const void* Q,
                  int64_t q_head_stride, int64_t q_row_stride, int64_t H, void* Qout, m4q_stream_t stream) {
  if (!K || !V || !slots || !Kc || !Vc || (Q && (!Qout || !freqs))) return M4Q_ERR_INVALID_ARG;
  if (freqs && (A < 1 || A > M4Q_ROPE_MAX_AXES)) return M4Q_ERR_INVALID_ARG;
  int rc = check_cache(kv_codec, B, Hkv, C, D);
  if (rc != M4Q_OK) return rc;
  if (M < 1 || M > INT32_MAX || (Q && H < 1) || (Q ? H : 0) + 2 * Hkv > 65535) return M4Q_ERR_INVALID_ARG;
  if (freqs) {
    rc = check_turn(pos, D, rot, layout, mscale);
    if (rc != M4Q_OK) return rc;
  }
  if (!aligned16(K) || !aligned16(V) || !aligned16(Kc) || !aligned16(Vc) || !aligned_to(slots, 4) ||
      !stride_ok(k_head_stride) || !stride_ok(k_row_stride) || !stride_ok(v_head_stride) || !stride_ok(v_row_stride) ||
      (freqs && (!aligned_to(pos, 4) || !aligned_to(freqs, 8) || !aligned_to(axes, 4))) ||
      (Q && (!aligned16(Q) || !aligned16(Qout) || !stride_ok(q_head_stride) || !stride_ok(q_row_stride))))
    return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  m4q::KvOpsParams p{};
  rc = ready(&dev, &p.status);
  if (rc != M4Q_OK) return rc;
  if (Q) {
    p.q = {static_cast<const __half*>(Q), q_head_stride, q_row_stride};
    p.qo = static_cast<__half*>(Qout);
    p.qo_hs = M * D;
    p.qo_rs = D;
    p.H = (int)H;
  }
  p.k = {static_cast<const __half*>(K), k_head_stride, k_row_stride};
  p.v = {static_cast<const __half*>(V), v_head_stride, v_row_stride};
  p.Hkv = (int)Hkv;
  p.M = (int)M;
  p.D = (int)D;
  if (freqs) {
    p.pos = pos;
    p.freqs = freqs;
    p.axes = axes;
    p.A = (int)A;
    p.rot = (int)rot;
    p.interleaved = layout == M4Q_ROPE_INTERLEAVED;
    p.mscale = mscale;
  }
  p.slots = slots;
  p.kc = static_cast<uint8_t*>(Kc);
  p.vc = static_cast<uint8_t*>(Vc);
  p.B = (int)B;
  p.C = (int)C;
  p.nsm = dev.sms;
  return done(m4q::launch_rope_kv(p, kv_codec == M4Q_Q8_0, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int m4q_rope(const void* X, int64_t x_head_stride, int64_t x_row_stride, int64_t H, int64_t M, int64_t D,
             const int32_t* pos, const int64_t* freqs, int64_t rot, int layout, float mscale, void* Y,
             int64_t y_head_stride, int64_t y_row_stride, m4q_stream_t stream) {
  return rope_call(X, x_head_stride, x_row_stride, H, M, D, pos, 1, freqs, nullptr, rot, layout, mscale, Y,
                   y_head_stride, y_row_stride, stream);
}

int m4q_rope_axes(const void* X, int64_t x_head_stride, int64_t x_row_stride, int64_t H, int64_t M, int64_t D,
                  const int32_t* pos, int64_t A, const int64_t* freqs, const int32_t* axes, int64_t rot, int layout,
                  float mscale, void* Y, int64_t y_head_stride, int64_t y_row_stride, m4q_stream_t stream) {
  if (!axes) return M4Q_ERR_INVALID_ARG;
  return rope_call(X, x_head_stride, x_row_stride, H, M, D, pos, A, freqs, axes, rot, layout, mscale, Y,
                   y_head_stride, y_row_stride, stream);
}

int m4q_kv_write(const void* K, int64_t k_head_stride, int64_t k_row_stride, const void* V, int64_t v_head_stride,
                 int64_t v_row_stride, int64_t Hkv, int64_t M, int64_t D, const int32_t* pos, const int64_t* freqs,
                 int64_t rot, int layout, float mscale, const int32_t* slots, void* Kc, void* Vc, int kv_codec,
                 int64_t B, int64_t C, const void* Q, int64_t q_head_stride, int64_t q_row_stride, int64_t H,
                 void* Qout, m4q_stream_t stream) {
  return kv_write_call(K, k_head_stride, k_row_stride, V, v_head_stride, v_row_stride, Hkv, M, D, pos, 1, freqs,
                       nullptr, rot, layout, mscale, slots, Kc, Vc, kv_codec, B, C, Q, q_head_stride, q_row_stride, H,
                       Qout, stream);
}

int m4q_kv_write_axes(const void* K, int64_t k_head_stride, int64_t k_row_stride, const void* V,
                      int64_t v_head_stride, int64_t v_row_stride, int64_t Hkv, int64_t M, int64_t D,
                      const int32_t* pos, int64_t A, const int64_t* freqs, const int32_t* axes, int64_t rot, int layout,
                      float mscale, const int32_t* slots, void* Kc, void* Vc, int kv_codec, int64_t B, int64_t C,
                      const void* Q, int64_t q_head_stride, int64_t q_row_stride, int64_t H, void* Qout,
                      m4q_stream_t stream) {
  if (!freqs || !axes) return M4Q_ERR_INVALID_ARG;
  return kv_write_call(K, k_head_stride, k_row_stride, V, v_head_stride, v_row_stride, Hkv, M, D, pos, A, freqs, axes,
                       rot, layout, mscale, slots, Kc, Vc, kv_codec, B, C, Q, q_head_stride, q_row_stride, H, Qout,
                       stream);
}

int m4q_kv_read(const void* Kc, const void* Vc, int kv_codec, int64_t B, int64_t Hkv, int64_t C, int64_t D,
                const int32_t* slots, int64_t n, void* Kout, void* Vout, m4q_stream_t stream) {
  if (!slots || (!Kc) != (!Kout) || (!Vc) != (!Vout) || (!Kc && !Vc)) return M4Q_ERR_INVALID_ARG;
  int rc = check_cache(kv_codec, B, Hkv, C, D);
  if (rc != M4Q_OK) return rc;
  if (n < 1 || n > INT32_MAX) return M4Q_ERR_INVALID_ARG;
  if ((Kc && (!aligned16(Kc) || !aligned16(Kout))) || (Vc && (!aligned16(Vc) || !aligned16(Vout))) ||
      !aligned_to(slots, 4))
    return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  m4q::KvReadParams p{};
  rc = ready(&dev, &p.status);
  if (rc != M4Q_OK) return rc;
  p.kc = static_cast<const uint8_t*>(Kc);
  p.vc = static_cast<const uint8_t*>(Vc);
  p.ko = static_cast<__half*>(Kout);
  p.vo = static_cast<__half*>(Vout);
  p.slots = slots;
  p.B = (int)B;
  p.Hkv = (int)Hkv;
  p.C = (int)C;
  p.D = (int)D;
  p.n = (int)n;
  return done(m4q::launch_kv_read(p, kv_codec == M4Q_Q8_0, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// How a tree attention call is laid out: persistent CTAs, and the workspace of
// the pieces that an even split of the key tiles leaves.
struct TreePlan {
  int rtiles, ws_rows, grid, seqs, waves;
  bool split;          // with a workspace
  m4q::TreeWhole whole;
  size_t ws_o, ws_bytes;
};

TreePlan tree_plan(int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t C, int64_t D, int sms) {
  TreePlan t;
  const int64_t rows = N * (H / Hkv);
  t.rtiles = (int)((rows + 127) / 128);
  t.ws_rows = (int)(rows < 128 ? rows : 128);
  const int64_t tiles = (C + 127) / 128;
  // sequences a launch: its unit count fits 31 bits (check_tree: that of one does)
  const int64_t fit = INT32_MAX / (Hkv * t.rtiles * tiles);
  int64_t seqs = B < m4q::kTreeSeqs ? B : m4q::kTreeSeqs;
  if (seqs > fit) seqs = fit;
  t.seqs = (int)seqs;
  const int64_t items = seqs * Hkv * t.rtiles;
  const int64_t most = items * tiles;
  const m4q::TreeWhole whole = rows <= m4q::kTreeFewRows ? m4q::kFewWhole : m4q::kRowsWhole;
  t.whole = whole;
  t.waves = (int)((items + sms - 1) / sms);
  t.split = (double)tiles * t.waves > whole.join;
  const int64_t want = t.split ? (most + m4q::kTreeLeast - 1) / m4q::kTreeLeast : items;
  t.grid = (int)(want < sms ? want : sms);
  t.ws_o = ((size_t)2 * t.grid * t.ws_rows * sizeof(float2) + 255) / 256 * 256;
  t.ws_bytes = t.split ? t.ws_o + (size_t)2 * t.grid * t.ws_rows * D * sizeof(float) : 0;
  return t;
}

int check_tree(int kv_codec, int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t C, int64_t D) {
  const int rc = check_cache(kv_codec, B, Hkv, C, D);
  if (rc != M4Q_OK) return rc;
  if (H < 1 || N < 1 || N > 256 || H > 65535 || B > INT32_MAX / (N * H)) return M4Q_ERR_INVALID_ARG;
  if (H % Hkv != 0) return M4Q_ERR_BAD_SHAPE;
  return (N * (H / Hkv) + 127) / 128 * Hkv <= INT32_MAX / ((C + 127) / 128) ? M4Q_OK : M4Q_ERR_BAD_SHAPE;
}

}  // namespace

extern "C" {

size_t m4q_attention_tree_workspace(int kv_codec, int64_t B, int64_t H, int64_t Hkv, int64_t N, int64_t C,
                                    int64_t D) {
  if (check_tree(kv_codec, B, H, Hkv, N, C, D) != M4Q_OK) return 0;
  DevInfo dev;
  if (current_device_info(&dev) != M4Q_OK) return 0;
  return tree_plan(B, H, Hkv, N, C, D, dev.sms).ws_bytes;
}

int m4q_attention_tree(const void* Q, const void* Kc, const void* Vc, int kv_codec, int64_t B, int64_t H, int64_t Hkv,
                       int64_t N, int64_t C, int64_t D, const int32_t* past, const int32_t* parents, float scale,
                       void* O, void* workspace, size_t workspace_bytes, m4q_stream_t stream) {
  const float scale_log2 = scale * 1.4426950408889634f;   // the kernels work in powers of 2
  if (!Q || !Kc || !Vc || !past || !parents || !O || !(scale_log2 - scale_log2 == 0.f)) return M4Q_ERR_INVALID_ARG;
  int rc = check_tree(kv_codec, B, H, Hkv, N, C, D);
  if (rc != M4Q_OK) return rc;
  if (!aligned16(Q) || !aligned16(Kc) || !aligned16(Vc) || !aligned16(O) || !aligned_to(past, 4) ||
      !aligned_to(parents, 4) || (workspace && !aligned16(workspace)))
    return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  m4q::TreeParams p{};
  rc = ready(&dev, &p.status);
  if (rc != M4Q_OK) return rc;
  TreePlan t = tree_plan(B, H, Hkv, N, C, D, dev.sms);
  if (!workspace || workspace_bytes < t.ws_bytes) t.split = false;
  p.q_rows = B * N;
  p.B_all = (int)B;
  p.H = (int)H;
  p.Hkv = (int)Hkv;
  p.G = (int)(H / Hkv);
  p.N = (int)N;
  p.C = (int)C;
  p.D = (int)D;
  p.scale_log2 = scale_log2;
  p.rtiles = t.rtiles;
  p.split = t.split ? 1 : 0;
  p.whole = t.whole;
  p.share = 1.f / (float)dev.sms;
  p.waves = t.waves;
  p.ws_rows = t.ws_rows;
  if (t.split) {
    char* ws = static_cast<char*>(workspace);
    p.ws_ml = reinterpret_cast<float2*>(ws);
    p.ws_o = reinterpret_cast<float*>(ws + t.ws_o);
  }
  const bool q8 = kv_codec == M4Q_Q8_0;
  CUtensorMap tm_k{}, tm_v{};
  if (!q8 && (!encode_kv(&tm_k, Kc, B * Hkv, C, D) || !encode_kv(&tm_v, Vc, B * Hkv, C, D))) return M4Q_ERR_CUDA;
  p.k = static_cast<const uint8_t*>(Kc);
  p.v = static_cast<const uint8_t*>(Vc);
  for (int64_t b0 = 0; b0 < B; b0 += t.seqs) {
    p.b0 = (int)b0;
    p.B = (int)(B - b0 < t.seqs ? B - b0 : t.seqs);
    p.q = static_cast<const __half*>(Q) + b0 * N * D;
    p.o = static_cast<__half*>(O) + b0 * N * H * D;
    p.past = past + b0;
    p.parents = parents + b0 * N;
    rc = done(m4q::launch_attention_tree(p, q8, tm_k, tm_v, t.grid, reinterpret_cast<cudaStream_t>(stream)));
    if (rc != M4Q_OK) return rc;
  }
  return M4Q_OK;
}

int m4q_page_plan(const int32_t* past, const int32_t* fresh, int64_t B, int64_t page, int32_t* table, int64_t W,
                  int32_t* held, int32_t* free_pages, int64_t P, int32_t* n_free, int64_t T, int32_t* slots,
                  int32_t* pos, int32_t* lengths, int32_t* starts, m4q_stream_t stream) {
  if (!past || !fresh || !table || !held || !free_pages || !n_free || !slots || !pos || !lengths || !starts)
    return M4Q_ERR_INVALID_ARG;
  if (B < 1 || B > m4q::kPlanSeqs || page < 1 || W < 1 || P < 1 || T < 1 || T > INT32_MAX - 8192)
    return M4Q_ERR_INVALID_ARG;
  if (page > INT32_MAX || P > INT32_MAX / page || W > INT32_MAX / page) return M4Q_ERR_BAD_SHAPE;
  const void* all[] = {past, fresh, table, held, free_pages, n_free, slots, pos, lengths, starts};
  for (const void* a : all)
    if (!aligned_to(a, 4)) return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  m4q::PlanParams p{};
  const int rc = ready(&dev, &p.status);
  if (rc != M4Q_OK) return rc;
  p.past = past;
  p.fresh = fresh;
  p.table = table;
  p.held = held;
  p.free_pages = free_pages;
  p.n_free = n_free;
  p.slots = slots;
  p.pos = pos;
  p.lengths = lengths;
  p.starts = starts;
  p.B = (int)B;
  p.W = (int)W;
  p.P = (int)P;
  p.page = (int)page;
  p.T = (int)T;
  // A token a thread up to eight CTAs of 1024 (and no more threads than there is work for).
  p.ctas = 1;
  while (p.ctas < 8 && T > 1024 * p.ctas) p.ctas *= 2;
  const int64_t work = T > B ? T : B;
  const int threads = work >= 1024 ? 1024 : (int)((work + 127) / 128 * 128);
  return done(m4q::launch_page_plan(p, threads, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// How a paged attention call is laid out: persistent CTAs, and the workspace of the
// pieces that an even split of the chunks leaves.
struct PagedPlan {
  int rtiles, seqs, grid, whole;   // whole: CTAs without a split
  bool split;
  float share, join;
  size_t ws_ml, ws_o, ws_bytes;
};

PagedPlan paged_plan(bool q8, int64_t B, int64_t H, int64_t Hkv, int64_t page, int64_t W, int64_t D, int sms) {
  PagedPlan t;
  const int G = (int)(H / Hkv), R = m4q::paged_rows(G);
  t.rtiles = (G + R - 1) / R;
  const int64_t chunk = m4q::paged_chunk((int)D, q8), chunks = (W * page + chunk - 1) / chunk;
  const int64_t fit = INT32_MAX / ((chunks + 1) * Hkv * t.rtiles);   // a launch's units fit 31 bits (check_paged: one sequence's do)
  t.seqs = (int)(B < m4q::kPagedSeqs ? B : m4q::kPagedSeqs);
  if (t.seqs > fit) t.seqs = (int)fit;
  const int64_t items = (int64_t)t.seqs * Hkv * t.rtiles;
  const int64_t most = (int64_t)sms * m4q::paged_ctas(G, (int)D, q8);
  const m4q::PagedCut cut = m4q::paged_cut(q8);
  t.join = cut.join;
  t.share = cut.share / (float)most;
  // Short tables stay whole by their width alone, two chunks past where a cut begins to pay
  // on the device: what the second launch and the workspace cost the host (4.5 us a call)
  // is more than it saves there (at most 2 us).
  t.split = (float)(chunks + 1) > cut.join + 2.f;
  t.whole = (int)(items < most ? items : most);
  t.grid = !t.split ? t.whole : (int)(chunks > most / items ? most : items * chunks);
  t.ws_ml = ((size_t)t.grid * sizeof(int4) + 255) / 256 * 256;
  t.ws_o = t.ws_ml + ((size_t)2 * t.grid * R * sizeof(float2) + 255) / 256 * 256;
  t.ws_bytes = t.split ? t.ws_o + (size_t)2 * t.grid * R * D * sizeof(float) : 0;
  return t;
}

int check_paged(int kv_codec, int64_t B, int64_t H, int64_t Hkv, int64_t P, int64_t page, int64_t W, int64_t D) {
  const int rc = check_cache(kv_codec, P, Hkv, page, D);
  if (rc != M4Q_OK) return rc;
  if (B < 1 || H < 1 || W < 1 || H > 65535 || B > 65535) return M4Q_ERR_INVALID_ARG;
  if (H % Hkv != 0 || page % 8 != 0 || W > INT32_MAX / page) return M4Q_ERR_BAD_SHAPE;
  // a sequence's chunks (of 64 keys or more) and one, times its items, fit 31 bits
  return (W * page + 127) / 64 <= INT32_MAX / H ? M4Q_OK : M4Q_ERR_BAD_SHAPE;
}

}  // namespace

extern "C" {

size_t m4q_attention_paged_workspace(int kv_codec, int64_t B, int64_t H, int64_t Hkv, int64_t P, int64_t page,
                                     int64_t W, int64_t D) {
  if (check_paged(kv_codec, B, H, Hkv, P, page, W, D) != M4Q_OK) return 0;
  DevInfo dev;
  if (current_device_info(&dev) != M4Q_OK) return 0;
  return paged_plan(kv_codec == M4Q_Q8_0, B, H, Hkv, page, W, D, dev.sms).ws_bytes;
}

int m4q_attention_paged(const void* Q, const void* Kc, const void* Vc, int kv_codec, int64_t B, int64_t H, int64_t Hkv,
                        int64_t P, int64_t page, int64_t D, const int32_t* table, int64_t W, const int32_t* lengths,
                        float scale, void* O, void* workspace, size_t workspace_bytes, m4q_stream_t stream) {
  const float scale_log2 = scale * 1.4426950408889634f;   // the kernels work in powers of 2
  if (!Q || !Kc || !Vc || !table || !lengths || !O || !(scale_log2 - scale_log2 == 0.f)) return M4Q_ERR_INVALID_ARG;
  int rc = check_paged(kv_codec, B, H, Hkv, P, page, W, D);
  if (rc != M4Q_OK) return rc;
  if (!aligned16(Q) || !aligned16(Kc) || !aligned16(Vc) || !aligned16(O) || !aligned_to(table, 4) ||
      !aligned_to(lengths, 4) || (workspace && !aligned16(workspace)))
    return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  m4q::PagedParams p{};
  rc = ready(&dev, &p.status);
  if (rc != M4Q_OK) return rc;
  const bool q8 = kv_codec == M4Q_Q8_0;
  PagedPlan t = paged_plan(q8, B, H, Hkv, page, W, D, dev.sms);
  CUtensorMap tm_k{}, tm_v{};
  if (!q8 && (!encode_kv(&tm_k, Kc, P * Hkv, page, D, 8) || !encode_kv(&tm_v, Vc, P * Hkv, page, D, 8)))
    return M4Q_ERR_CUDA;
  if (t.split && (!workspace || workspace_bytes < t.ws_bytes)) {
    t.split = false;
    t.grid = t.whole;
  }
  p.k = static_cast<const uint8_t*>(Kc);
  p.v = static_cast<const uint8_t*>(Vc);
  p.q_rows = B;
  p.H = (int)H;
  p.Hkv = (int)Hkv;
  p.G = (int)(H / Hkv);
  p.P = (int)P;
  p.page = (int)page;
  p.W = (int)W;
  p.D = (int)D;
  p.scale_log2 = scale_log2;
  p.rtiles = t.rtiles;
  p.split = t.split ? 1 : 0;
  p.share = t.share;
  p.join = t.join;
  if (t.split) {
    char* ws = static_cast<char*>(workspace);
    p.ws_cut = reinterpret_cast<int4*>(ws);
    p.ws_ml = reinterpret_cast<float2*>(ws + t.ws_ml);
    p.ws_o = reinterpret_cast<float*>(ws + t.ws_o);
  }
  for (int64_t b0 = 0; b0 < B; b0 += t.seqs) {
    p.B = (int)(B - b0 < t.seqs ? B - b0 : t.seqs);
    p.q = static_cast<const __half*>(Q) + b0 * D;
    p.o = static_cast<__half*>(O) + b0 * H * D;
    p.table = table + b0 * W;
    p.lengths = lengths + b0;
    p.waves = (float)((p.B * (int)Hkv * t.rtiles + t.grid - 1) / t.grid);
    rc = done(m4q::launch_attention_paged(p, q8, tm_k, tm_v, t.grid, reinterpret_cast<cudaStream_t>(stream)));
    if (rc != M4Q_OK) return rc;
  }
  return M4Q_OK;
}

int m4q_verify_tree(const void* target, int64_t t_seq_stride, int64_t t_row_stride, const void* draft,
                    int64_t d_seq_stride, int64_t d_row_stride, int prob_type, int64_t B, int64_t N, int64_t V,
                    const int32_t* tokens, const int32_t* parents, const float* u, int32_t* path, int32_t* count,
                    int32_t* token, m4q_stream_t stream) {
  if (!target || (!draft && N > 1) || !tokens || !parents || !u || !path || !count || !token)
    return M4Q_ERR_INVALID_ARG;
  if (prob_type != M4Q_PROB_F32 && prob_type != M4Q_PROB_F16) return M4Q_ERR_INVALID_ARG;
  if (B < 1 || B > INT32_MAX / m4q::kVerifyNodes || N < 1 || N > m4q::kVerifyNodes || V < 1 || V > 1 << 24)
    return M4Q_ERR_INVALID_ARG;
  const int size = prob_type == M4Q_PROB_F32 ? 4 : 2;
  if (!aligned_to(target, size) || !aligned_to(draft, size)) return M4Q_ERR_MISALIGNED;
  const void* all[] = {tokens, parents, u, path, count, token};
  for (const void* a : all)
    if (!aligned_to(a, 4)) return M4Q_ERR_MISALIGNED;
  DevInfo dev;
  m4q::VerifyParams p{};
  const int rc = ready(&dev, &p.status);
  if (rc != M4Q_OK) return rc;
  p.target = target;
  p.draft = draft;
  p.t_bs = t_seq_stride;
  p.t_rs = t_row_stride;
  p.d_bs = d_seq_stride;
  p.d_rs = d_row_stride;
  p.tokens = tokens;
  p.parents = parents;
  p.u = u;
  p.path = path;
  p.count = count;
  p.token = token;
  p.B = (int)B;
  p.N = (int)N;
  p.V = (int)V;
  // CTAs of a sequence: as many as fit the device at once, two an SM, each with at least
  // 4,096 values; up to 8, or 16 where that many fit (12.1 us with 16, 14.7 with 8 and 52.6
  // with 1 for one sequence over 128,000 values; 28.5 with 8, 38.5 with 4 and 37.1 with 16
  // for 32; 8.3 with 1, 9.0 with 2 for 16 over 4,000).
  int64_t ctas = 2 * dev.sms / B;
  if (ctas > V / 4096) ctas = V / 4096;
  p.ctas = ctas >= 16 ? 16 : ctas > 8 ? 8 : ctas < 1 ? 1 : (int)ctas;
  return done(m4q::launch_verify(p, prob_type == M4Q_PROB_F16, reinterpret_cast<cudaStream_t>(stream)));
}

int m4q_norm_residual(const void* h, const void* R, int res_type, const void* w_post, const void* gate, int gate_rows,
                      const void* w_pre, int64_t M, int64_t D, float res_scale, float branch_scale, float eps,
                      void* R_out, void* Y, m4q_stream_t stream) {
  if (!R || (res_type != M4Q_RES_F16 && res_type != M4Q_RES_F32)) return M4Q_ERR_INVALID_ARG;
  if (!h && (w_post || gate)) return M4Q_ERR_INVALID_ARG;
  if ((!w_pre) != (!Y) || (!R_out && !Y)) return M4Q_ERR_INVALID_ARG;
  if (M < 1 || M > INT32_MAX || D < 8 || D > 32768) return M4Q_ERR_INVALID_ARG;
  if (!(res_scale - res_scale == 0.f) || !(branch_scale - branch_scale == 0.f) || !(eps >= 0.f) ||
      !(eps - eps == 0.f))
    return M4Q_ERR_INVALID_ARG;
  if (D % 8 != 0) return M4Q_ERR_BAD_SHAPE;
  if (!aligned16(h) || !aligned16(R) || !aligned16(w_post) || !aligned16(gate) || !aligned16(w_pre) ||
      !aligned16(R_out) || !aligned16(Y))
    return M4Q_ERR_MISALIGNED;
  if (Y == R_out) return M4Q_ERR_INVALID_ARG;
  DevInfo dev;
  m4q::NormParams p{};
  const int rc = ready(&dev, &p.status);
  if (rc != M4Q_OK) return rc;
  p.h = static_cast<const __half*>(h);
  p.r = R;
  p.w_post = static_cast<const __half*>(w_post);
  p.gate = static_cast<const __half*>(gate);
  p.w_pre = static_cast<const __half*>(w_pre);
  p.r_out = R_out;
  p.y = static_cast<__half*>(Y);
  p.M = M;
  p.D = (int)D;
  p.gate_rows = gate_rows ? 1 : 0;
  p.res_scale = res_scale;
  p.branch_scale = branch_scale;
  p.eps = eps;
  return done(m4q::launch_norm_residual(p, res_type == M4Q_RES_F32, reinterpret_cast<cudaStream_t>(stream)));
}

int m4q_check_finite(const void* x, int64_t n, m4q_stream_t stream) {
  if (!x || n < 0) return M4Q_ERR_INVALID_ARG;
  if (!aligned16(x)) return M4Q_ERR_MISALIGNED;
  uint32_t* words = m4q::status_words();
  if (!words) return M4Q_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (m4q::launch_finite_check(x, n, words + 1, s) != cudaSuccess) return M4Q_ERR_CUDA;
  uint32_t flag = 0;
  if (cudaMemcpyAsync(&flag, words + 1, sizeof(flag), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return M4Q_ERR_CUDA;
  return flag ? M4Q_ERR_NONFINITE : M4Q_OK;
}

int m4q_check_device_status(m4q_stream_t stream) {
  uint32_t* words = m4q::status_words();
  if (!words) return M4Q_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t st = 0;
  if (cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpy(&st, words, sizeof(st), cudaMemcpyDeviceToHost) != cudaSuccess)
    return M4Q_ERR_CUDA;
  if (st) {
    if (cudaMemset(words, 0, sizeof(uint32_t)) != cudaSuccess) return M4Q_ERR_CUDA;
    return (st & m4q::kErrBoundsBit) ? M4Q_ERR_BOUNDS : M4Q_ERR_TIMEOUT;
  }
  return M4Q_OK;
}

int m4q_build_flags(void) {
#if M4Q_BOUNDS
  return M4Q_BUILD_BOUNDS;
#else
  return 0;
#endif
}

int m4q_bounds_site(m4q_stream_t stream) {
  uint32_t* words = m4q::status_words();
  if (!words) return M4Q_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t site = 0;
  if (cudaStreamSynchronize(s) != cudaSuccess ||
      cudaMemcpy(&site, words + 2, sizeof(site), cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemset(words + 2, 0, sizeof(uint32_t)) != cudaSuccess)
    return M4Q_ERR_CUDA;
  return (int)site;
}

int m4q_selftest_wait_timeout(int64_t limit_ns, m4q_stream_t stream) {
  if (limit_ns < 1000 || limit_ns > 1000000000) return M4Q_ERR_INVALID_ARG;
  uint32_t* words = m4q::status_words();
  if (!words) return M4Q_ERR_CUDA;
  return m4q::launch_wait_selftest(words, (unsigned long long)limit_ns,
                                   reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? M4Q_OK
             : M4Q_ERR_CUDA;
}

const char* m4q_status_string(int status) {
  switch (status) {
    case M4Q_OK: return "ok";
    case M4Q_ERR_INVALID_ARG: return "invalid argument";
    case M4Q_ERR_UNSUPPORTED_CODEC: return "unsupported codec";
    case M4Q_ERR_BAD_SHAPE: return "bad shape (K must be a multiple of the block, N of 8)";
    case M4Q_ERR_MISALIGNED: return "pointer not aligned (16 bytes; fp16 scale and bias arrays 2 bytes)";
    case M4Q_ERR_CUDA: return "CUDA error";
    case M4Q_ERR_NONFINITE: return "non-finite values found";
    case M4Q_ERR_TIMEOUT: return "a device pipeline wait gave up";
    case M4Q_ERR_UNSUPPORTED_DEVICE: return "device is not sm_103";
    case M4Q_ERR_SCRATCH_LIMIT: return "M * F exceeds the fixed scratch of m4q_mlp_noalloc (1 << 20 fp16)";
    case M4Q_ERR_BOUNDS: return "an access was out of range (bounds-checked build)";
    default: return "unknown status";
  }
}

int m4q_version(void) { return 100; }

}  // extern "C"
