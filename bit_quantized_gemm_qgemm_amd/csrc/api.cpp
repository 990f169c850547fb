// libqgemm C ABI: argument checks, dispatch by format and M, launch on the
// caller's stream.  Every check that needs no device runs first, so a bad
// call returns its status without touching the HIP runtime.
#include <hip/hip_runtime.h>

#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "../../include/qgemm.h"
#include "qgemm_common.h"

namespace {

using qgemm::PackGeom;
using qgemm::pack_geom;
using qgemm::grouped_geom;

constexpr int64_t kMaxIndex = (int64_t)1 << 31;   // kernels index with 32-bit ints
// The weight-only GEMMs take the 256 x 256 tiled kernel from M = 256 on once
// its grid fills three quarters of the CUs (192 tiles), or from M = 640 with
// at least 48 tiles; otherwise the small-M kernel.  A round of tiles costs
// about the same whatever M is, while the small-M kernel's time grows with M.
// Measured on MI355X (us, small-M kernel / tiled kernel):
//   W8A16 K = 4096 N = 11008 (43 tile columns): M = 512 114 / 132, 768 189 / 134
//   W4A16 K = 8192 N = 28672 (112): M = 256 177 / 219, 384 267 / 223
//   W8A16 K = 4096 N = 4096 (16): M = 512 75 / 132, 768 165 / 132
//   grouped W4A16 g128 K = 8192 N = 28672: M = 256 214 / 257, 384 318 / 258
//   grouped W8A16 g128 K = 4096 N = 11008: M = 512 115 / 151, 768 186 / 153
//   NVFP4 K = 8192 N = 28672: M = 256 198 / 247, 384 303 / 249
constexpr int64_t kWeightOnlyTileMinM = 256;
constexpr int64_t kWeightOnlyTileFullGrid = 192;
constexpr int64_t kWeightOnlyTileLongM = 640;
constexpr int64_t kWeightOnlyTileLongMinTiles = 48;
bool weight_only_tiled(int64_t M, int64_t N) {
  if (M < kWeightOnlyTileMinM || N <= 128) return false;
  const int64_t tiles = qgemm::cdiv(M, 256) * qgemm::cdiv(N, 256);
  return tiles >= kWeightOnlyTileFullGrid ||
         (M >= kWeightOnlyTileLongM && tiles >= kWeightOnlyTileLongMinTiles);
}
// FP8 and MXFP4 GEMMs take the small-M kernel (16-row slabs, up to four per
// workgroup) up to M = 64; from 65 to 128 rows unless N is wide (FP8 N >=
// 24576, MXFP4 N >= 16384), where one row of 256 x 256 tiles is faster; and
// above that while the tiled kernels' grid stays small: FP8 up to M = 512
// while M * N <= 2.6e6 (5 * 2^19), MXFP4 up to M = 256 while M * N <= 2^21.
// Otherwise the tile kernels.  The small-M kernel's time grows with M * N * K,
// while the tiled kernels take about one 256 x 256 x K tile per CU whatever M
// is.  Measured on MI355X (us, small-M kernel / tile kernels):
//   FP8 K = N = 8192:   M = 128 30 / 68, 144 47 / 69, 256 48 / 73, 384 71 / 70,
//                       512 95 / 73
//   FP8 K = N = 4096:   M = 512 37 / 40, 768 54 / 40
//   FP8 K = 8192, N = 28672: M = 72 92 / 78, 128 86 / 72, 144 123 / 80
//   FP8 K = 4096, N = 16384: M = 96 28 / 38
//   MXFP4 K = N = 8192: M = 128 27 / 44, 192 39 / 50, 256 49 / 56, 384 70 / 46
//   MXFP4 K = N = 4096: M = 256 24 / 26, 384 34 / 25
//   MXFP4 K = 8192, N = 28672: M = 72 87 / 48, 128 85 / 51, 144 117 / 52
//   MXFP4 K = 4096, N = 16384: M = 72 27.6 / 24.7, 128 27.8 / 27.0
bool scaled_small_m(int fmt, int64_t M, int64_t N) {
  if (M <= 64) return true;
  if (M <= 128) return N < (fmt == QGEMM_FP8 ? 24576 : 16384);
  if (fmt == QGEMM_FP8) return M <= 512 && M * N <= 2621440;
  return M <= 256 && M * N <= 2097152;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// formats of qgemm_prepack (the grouped ones have their own prepack)
bool valid_format(int fmt) {
  return (fmt >= QGEMM_W4A16 && fmt <= QGEMM_FP8) || fmt == QGEMM_NVFP4;
}

// K constraints per format (see qgemm.h).
bool k_ok(int fmt, int64_t K) {
  switch (fmt) {
    case QGEMM_W4A16: return K % 2 == 0;
    case QGEMM_W8A16: return true;
    case QGEMM_MXFP4: return K % 32 == 0;
    case QGEMM_FP8: return K % 16 == 0;
    case QGEMM_NVFP4: return K % 16 == 0;
    default: return false;
  }
}

// Sizes must be non-negative and every array the kernels index must stay
// addressable with 32-bit element offsets.
int check_sizes(int fmt, int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return QGEMM_ERR_SHAPE;
  if (!k_ok(fmt, K)) return QGEMM_ERR_SHAPE;
  if (M >= kMaxIndex || N >= kMaxIndex || K >= kMaxIndex) return QGEMM_ERR_SHAPE;
  if (M * K * 2 >= kMaxIndex * 2 || M * N >= kMaxIndex || K * N >= kMaxIndex * 2)
    return QGEMM_ERR_SHAPE;
  return QGEMM_OK;
}

// Device architecture check, cached per device ordinal.  The environment
// variable QGEMM_ARCH_OVERRIDE, when set, stands in for the current device's
// architecture name and no device is queried (host-side tests of the
// ERR_ARCH path on machines without the GPU).
int check_device() {
  if (const char* forced = std::getenv("QGEMM_ARCH_OVERRIDE"))
    return std::strncmp(forced, "gfx950", 6) == 0 ? QGEMM_OK : QGEMM_ERR_ARCH;
  static std::mutex mu;
  static int cached[64];
  static bool init = false;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return QGEMM_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(mu);
  if (!init) {
    for (int& c : cached) c = 1;  // 1 = unknown
    init = true;
  }
  if (dev < 0 || dev >= 64) return QGEMM_ERR_DEVICE;
  if (cached[dev] == 1) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return QGEMM_ERR_DEVICE;
    cached[dev] = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? QGEMM_OK : QGEMM_ERR_ARCH;
  }
  return cached[dev];
}

int launched(hipError_t e) { return e == hipSuccess ? QGEMM_OK : QGEMM_ERR_LAUNCH; }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// A pointer may be NULL only when its array holds no elements.
bool present(const void* p, int64_t elems) { return p != nullptr || elems == 0; }

// The kernel a GEMM call of format fmt launches (M, N, K and group_k already
// validated): the one dispatch every entry point and qgemm_dispatch_kernel
// apply.  The fused-quantization calls dispatch as their GEMM format.
int kernel_for(int fmt, int64_t M, int64_t N, int64_t K, int64_t group_k) {
  if (M == 0 || N == 0) return QGEMM_KERNEL_NONE;
  switch (fmt) {
    case QGEMM_W4A16:
    case QGEMM_W8A16:   // fp16 X rows of the tile kernel must be 16-byte aligned
      return weight_only_tiled(M, N) && K > 0 && K % 8 == 0 &&
                     qgemm::pipe_fits(fmt, M, N, K, 0)
                 ? QGEMM_KERNEL_WEIGHT_ONLY_256
                 : QGEMM_KERNEL_SMALL_M;
    case QGEMM_NVFP4:   // K % 16 == 0
      return weight_only_tiled(M, N) && K > 0 && qgemm::pipe_fits(fmt, M, N, K, 0)
                 ? QGEMM_KERNEL_WEIGHT_ONLY_256
                 : QGEMM_KERNEL_SMALL_M;
    case QGEMM_W4A16_GROUPED:
    case QGEMM_W8A16_GROUPED:   // K % 32 == 0
      return weight_only_tiled(M, N) && K > 0 && qgemm::pipe_fits(fmt, M, N, K, group_k)
                 ? QGEMM_KERNEL_WEIGHT_ONLY_256
                 : QGEMM_KERNEL_SMALL_M;
    case QGEMM_MXFP4:
    case QGEMM_FP8:
      if (scaled_small_m(fmt, M, N)) return QGEMM_KERNEL_SMALL_M;
      if (!qgemm::tile_is_big(fmt, M, N, K)) return QGEMM_KERNEL_TILE_128;
      return fmt == QGEMM_MXFP4 ? QGEMM_KERNEL_MXFP4_256 : QGEMM_KERNEL_FP8_256;
    default:
      return QGEMM_ERR_FORMAT;
  }
}

int weight_only(int fmt, const void* x, const void* w_packed, const void* scales, void* y,
                int64_t M, int64_t N, int64_t K, void* stream) {
  int st = check_sizes(fmt, M, N, K);
  if (st != QGEMM_OK) return st;
  if (!present(x, M * K) || !present(w_packed, K * N) || !present(scales, N) ||
      !present(y, M * N))
    return QGEMM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w_packed, 16) || !aligned(scales, 16) || !aligned(y, 16))
    return QGEMM_ERR_ALIGN;
  if (M == 0 || N == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  // Large M: LDS-tiled matrix-core kernel (each weight byte is read once per
  // 256 rows).  Otherwise the register-dequant kernel in 16-row slabs, the
  // bandwidth path of decode.
  if (kernel_for(fmt, M, N, K, 0) == QGEMM_KERNEL_WEIGHT_ONLY_256)
    return launched(qgemm::launch_weight_only_tile(fmt, x, w_packed, scales, y, M, N, K,
                                                   as_stream(stream)));
  return launched(qgemm::launch_decode_gemm(fmt, x, w_packed, scales, nullptr, nullptr, y, M, N,
                                            K, as_stream(stream)));
}

// Grouped weight-only formats: K and group_k multiples of 32 (a 32-element
// matrix step never straddles two groups), the sizes of the per-column format.
int check_grouped(int fmt, int64_t M, int64_t N, int64_t K, int64_t group_k) {
  if (fmt != QGEMM_W4A16_GROUPED && fmt != QGEMM_W8A16_GROUPED) return QGEMM_ERR_FORMAT;
  if (group_k <= 0 || group_k % 32 != 0 || K % 32 != 0) return QGEMM_ERR_SHAPE;
  if (group_k >= kMaxIndex) return QGEMM_ERR_SHAPE;
  return check_sizes(fmt == QGEMM_W4A16_GROUPED ? QGEMM_W4A16 : QGEMM_W8A16, M, N, K);
}

int grouped_gemm(int fmt, const void* x, const void* w_packed, void* y, int64_t M, int64_t N,
                 int64_t K, int64_t group_k, void* stream) {
  int st = check_grouped(fmt, M, N, K, group_k);
  if (st != QGEMM_OK) return st;
  if (!present(x, M * K) || !present(w_packed, K * N) || !present(y, M * N))
    return QGEMM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w_packed, 16) || !aligned(y, 16)) return QGEMM_ERR_ALIGN;
  if (M == 0 || N == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  // K % 32 == 0 here, so fp16 X rows are 16-byte aligned
  if (kernel_for(fmt, M, N, K, group_k) == QGEMM_KERNEL_WEIGHT_ONLY_256)
    return launched(qgemm::launch_weight_only_tile_grouped(fmt, x, w_packed, y, M, N, K, group_k,
                                                           as_stream(stream)));
  return launched(qgemm::launch_decode_grouped(fmt, x, w_packed, y, M, N, K, group_k,
                                               as_stream(stream)));
}

// ---- FP8 GEMM with fp32 A quantized on the device --------------------------

// Checks shared by qgemm_fp8_act and qgemm_fp8_act_noalloc (everything but
// the workspace).
int check_fp8_act(const float* a, const void* b_packed, const float* scale_b, void* c,
                  int64_t M, int64_t N, int64_t K) {
  int st = check_sizes(QGEMM_FP8, M, N, K);
  if (st != QGEMM_OK) return st;
  if (!present(a, M * K) || !present(b_packed, K * N) || !present(c, M * N) || !scale_b)
    return QGEMM_ERR_NULL;
  if (!aligned(a, 16) || !aligned(b_packed, 16) || !aligned(c, 16) || !aligned(scale_b, 4))
    return QGEMM_ERR_ALIGN;
  return QGEMM_OK;
}

// Quantize A into ws (codes [M*K], the fp32 scale at round_up(M*K, 16), the
// partial maxima 16 bytes after it), then the GEMM; everything on `stream`.
int fp8_act_run(const float* a, const void* b_packed, const float* scale_b, void* c, uint8_t* ws,
                int64_t M, int64_t N, int64_t K, void* stream) {
  uint8_t* codes = ws;
  float* scale_a = reinterpret_cast<float*>(codes + qgemm::cdiv(M * K, 16) * 16);
  float* partials = scale_a + 4;
  // an empty A still gets its scale (1.0, the all-zero rule); K % 16 == 0,
  // so A is whole 16-byte pieces
  int st = launched(
      qgemm::launch_quantize_fp8_ws(a, M * K, codes, scale_a, partials, as_stream(stream)));
  if (st != QGEMM_OK || N == 0) return st;
  if (kernel_for(QGEMM_FP8, M, N, K, 0) == QGEMM_KERNEL_SMALL_M)
    return launched(qgemm::launch_decode_gemm(QGEMM_FP8, codes, b_packed, nullptr, scale_a,
                                              scale_b, c, M, N, K, as_stream(stream)));
  return launched(qgemm::launch_tile_gemm(QGEMM_FP8, codes, nullptr, b_packed, scale_a, scale_b,
                                          c, M, N, K, as_stream(stream)));
}

// Fixed scratch of qgemm_fp8_act_noalloc, one copy per GPU, held from the
// moment the code object is loaded on that GPU until the process ends: the
// codes of A (at most QGEMM_FP8_ACT_NOALLOC_MAX_ELEMS bytes), 16 bytes holding
// the fp32 scale, then the partial maxima of the quantizer.  Every call on a
// GPU shares that GPU's copy.  Nothing in it needs to start at zero: each
// call writes every byte it later reads.
constexpr int64_t kNoAllocScratchBytes =
    QGEMM_FP8_ACT_NOALLOC_MAX_ELEMS + 16 + 4 * qgemm::kFp8Partials;
static __device__ __align__(256) uint8_t scratch[kNoAllocScratchBytes];

// The device address of this GPU's copy of `scratch`.  In host code the
// array's name is only a host-side stand-in, so kernels receive the address
// hipGetSymbolAddress returns, looked up once per device with that device
// current.
int scratch_of_current_device(uint8_t** out) {
  static std::mutex mu;
  static void* addr[64] = {};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return QGEMM_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p)
      return QGEMM_ERR_DEVICE;
    addr[dev] = p;
  }
  *out = static_cast<uint8_t*>(addr[dev]);
  return QGEMM_OK;
}

// ---- paged key-value cache ---------------------------------------------------

constexpr int64_t kMaxStride = (int64_t)1 << 40;   // elements; keeps offsets far from 2^63

bool below(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v < hi; }

// Types of the cache calls: 16-bit elements, pools of the same type or e4m3
// with both scale arrays (and only then).
int check_kv_types(int dtype, int cache_dtype, const float* k_scale, const float* v_scale,
                   int64_t kv_heads) {
  if (dtype != QGEMM_F16 && dtype != QGEMM_BF16) return QGEMM_ERR_FORMAT;
  if (cache_dtype != dtype && cache_dtype != QGEMM_E4M3) return QGEMM_ERR_FORMAT;
  if (cache_dtype == QGEMM_E4M3) {
    if (!present(k_scale, kv_heads) || !present(v_scale, kv_heads)) return QGEMM_ERR_NULL;
    if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return QGEMM_ERR_ALIGN;
  } else if (k_scale || v_scale) {
    return QGEMM_ERR_FORMAT;
  }
  return QGEMM_OK;
}

bool kv_dim_ok(int64_t dim) { return dim >= 16 && dim <= 256 && dim % 16 == 0; }

// Rows of the pools counted in 32 bits (see KvPool).
int check_kv_pool(int64_t kv_heads, int64_t dim, int64_t pages, int64_t page_size,
                  int64_t page_stride, int64_t head_stride, int64_t token_stride,
                  qgemm::KvPool* pool) {
  if (!kv_dim_ok(dim)) return QGEMM_ERR_SHAPE;
  if (!below(kv_heads, 0, kMaxIndex) || !below(pages, 0, kMaxIndex) ||
      !below(page_size, 1, kMaxIndex) || pages * page_size >= kMaxIndex)
    return QGEMM_ERR_SHAPE;
  for (int64_t st : {page_stride, head_stride, token_stride})
    if (!below(st, 0, kMaxIndex * dim) || st % dim != 0) return QGEMM_ERR_SHAPE;
  const int64_t pr = page_stride / dim, hr = head_stride / dim, tr = token_stride / dim;
  if (pages > 0 && kv_heads > 0) {   // each product is below 2^62
    const int64_t a = (pages - 1) * pr, b = (kv_heads - 1) * hr, c = (page_size - 1) * tr;
    if (a >= kMaxIndex || b >= kMaxIndex || c >= kMaxIndex || a + b + c >= kMaxIndex)
      return QGEMM_ERR_SHAPE;
  }
  *pool = qgemm::KvPool{(int)pages, (int)page_size, (int)pr, (int)hr, (int)tr};
  return QGEMM_OK;
}

// Entries of 4 bytes from `at` on.
struct Span {
  uintptr_t at;
  int64_t n;
  Span(const void* p, int64_t entries) : at(reinterpret_cast<uintptr_t>(p)), n(entries) {}
  bool meets(const Span& o) const {   // one begins within the other
    return n > 0 && o.n > 0 && (at - o.at < 4 * (uintptr_t)o.n || o.at - at < 4 * (uintptr_t)n);
  }
};

// Whether x meets a row of a table: rows of `width` entries, `stride` apart.
bool meets_rows(const Span& x, const void* table, int64_t rows, int64_t width, int64_t stride) {
  const Span all(table, rows > 0 && width > 0 ? (rows - 1) * stride + width : 0);
  if (!x.meets(all)) return false;
  if (rows == 1 || x.at < all.at) return true;
  const int64_t from = (int64_t)((x.at - all.at) / 4), row = from / stride;   // stride >= width
  return from - row * stride < width || from + x.n > (row + 1) * stride;
}

// ---- int8 x int8 products, dense and by expert ------------------------------

// Bytes at `at`; whether two such stretches share any.
struct Bytes {
  uintptr_t at;
  uint64_t n;
  Bytes(const void* p, int64_t bytes) : at(reinterpret_cast<uintptr_t>(p)), n((uint64_t)bytes) {}
  bool meets(const Bytes& o) const {
    return n > 0 && o.n > 0 && (at - o.at < o.n || o.at - at < n);
  }
};

// Whether an output shares memory with an input or with another output.
int check_apart(std::initializer_list<Bytes> outputs, std::initializer_list<Bytes> inputs) {
  for (const Bytes& x : outputs) {
    for (const Bytes& y : inputs)
      if (x.meets(y)) return QGEMM_ERR_OVERLAP;
    for (const Bytes& y : outputs)
      if (&x != &y && x.meets(y)) return QGEMM_ERR_OVERLAP;
  }
  return QGEMM_OK;
}

// The sum of K products of two codes stays within 32 bits: 2^14 K < 2^31.
constexpr int64_t kMaxInt8K = 131056;
// Rows of a product: a launch has less than 2^32 threads.
constexpr int64_t kMaxInt8Rows = (int64_t)1 << 28;

// One packed weight stays below 2^31 bytes (32-bit offsets within it), all of
// them below 2^41.
int check_w8a8_weight(int64_t experts, int64_t K, int64_t N, int gated) {
  if (!below(experts, 1, qgemm::kMaxExperts + 1) || !below(K, 0, kMaxInt8K + 1) || K % 16 != 0 ||
      !below(N, 0, kMaxIndex) || (gated != 0 && gated != 1) || (gated && N % 2 != 0))
    return QGEMM_ERR_SHAPE;
  if ((N + 32) * qgemm::cdiv(K > 0 ? K : 1, 128) * 128 >= kMaxIndex) return QGEMM_ERR_SHAPE;
  return QGEMM_OK;
}

// Checks and the launch shared by qgemm_w8a8 (experts = 0) and qgemm_w8a8_experts.
int w8a8(int dtype, const int8_t* a, const float* a_scale, const void* w_packed,
         const float* w_scale, const int32_t* offsets, const int32_t* rows, void* out,
         int64_t a_rows, int64_t M, int64_t N, int64_t K, int64_t experts, int gated, void* stream) {
  if (dtype != QGEMM_F16 && dtype != QGEMM_BF16) return QGEMM_ERR_FORMAT;
  const bool grouped = experts != 0;
  const int64_t weights = grouped ? experts : 1;
  int st = check_w8a8_weight(weights, K, N, gated);
  if (st != QGEMM_OK) return st;
  const int64_t out_n = gated ? N / 2 : N;
  if (!below(M, 0, kMaxInt8Rows) || !below(a_rows, 0, kMaxIndex) || a_rows * K >= kMaxIndex ||
      M * N >= kMaxIndex || (!rows && M > 0 && a_rows != M))
    return QGEMM_ERR_SHAPE;
  const bool some = M > 0 && N > 0;
  if (!present(a, a_rows * K) || !present(a_scale, a_rows) || !present(w_packed, K * N) ||
      !present(w_scale, N) || !present(out, M * out_n) || (grouped && !offsets))
    return QGEMM_ERR_NULL;
  if (!aligned(a, 16) || !aligned(w_packed, 16) || !aligned(out, 16) || !aligned(a_scale, 4) ||
      !aligned(w_scale, 4) || !aligned(offsets, 4) || !aligned(rows, 4))
    return QGEMM_ERR_ALIGN;
  const qgemm::W8a8Geom geom = qgemm::w8a8_geom(K, N, gated);
  if ((st = check_apart({{out, 2 * M * out_n}},
                        {{a, a_rows * K}, {a_scale, 4 * a_rows}, {w_packed, weights * geom.bytes},
                         {w_scale, 4 * weights * N}, {offsets, grouped ? 4 * (experts + 1) : 0},
                         {rows, rows ? 4 * M : 0}})) != QGEMM_OK)
    return st;
  if (!some) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  qgemm::W8a8 p{};
  p.a = a;
  p.a_scale = a_scale;
  p.w = static_cast<const uint8_t*>(w_packed);
  p.w_scale = w_scale;
  p.offsets = offsets;
  p.rows = rows;
  p.out = static_cast<uint16_t*>(out);
  p.a_rows = a_rows;
  p.M = M;
  p.N = N;
  p.K = K;
  p.experts = weights;
  p.gated = gated != 0;
  p.bf16 = dtype == QGEMM_BF16;
  return launched(qgemm::launch_w8a8(p, as_stream(stream)));
}

bool kv_view_ok(int64_t outer, int64_t inner) {   // strides of q, k, v: whole 16-byte pieces
  return below(outer, 0, kMaxStride) && below(inner, 0, kMaxStride) && outer % 8 == 0 &&
         inner % 8 == 0;
}

}  // namespace

extern "C" {

const char* qgemm_status_string(int status) {
  switch (status) {
    case QGEMM_OK: return "ok";
    case QGEMM_ERR_NULL: return "a required pointer is NULL";
    case QGEMM_ERR_SHAPE: return "invalid shape (negative, K not a multiple the format needs, or too large)";
    case QGEMM_ERR_ALIGN: return "pointer not aligned (16 bytes for arrays, 4 for scalar scales)";
    case QGEMM_ERR_ARCH: return "current device is not gfx950";
    case QGEMM_ERR_LAUNCH: return "kernel launch failed";
    case QGEMM_ERR_FORMAT: return "unknown format id";
    case QGEMM_ERR_DEVICE: return "no HIP device available";
    case QGEMM_ERR_TOO_LARGE: return "input larger than the entry point's fixed scratch";
    case QGEMM_ERR_OVERLAP: return "buffers share memory that must not";
    default: return "unknown status";
  }
}

int qgemm_abi_version(void) { return 103; }

int qgemm_dispatch_kernel(int fmt, int64_t M, int64_t N, int64_t K, int64_t group_k) {
  int st;
  if (fmt == QGEMM_W4A16_GROUPED || fmt == QGEMM_W8A16_GROUPED)
    st = check_grouped(fmt, M, N, K, group_k);
  else if (valid_format(fmt))
    st = check_sizes(fmt, M, N, K);
  else
    return QGEMM_ERR_FORMAT;
  if (st != QGEMM_OK) return st;
  return kernel_for(fmt, M, N, K, group_k);
}

int64_t qgemm_prepack_bytes(int fmt, int64_t K, int64_t N) {
  if (!valid_format(fmt)) return QGEMM_ERR_FORMAT;
  const int st = check_sizes(fmt, 0, N, K);
  if (st != QGEMM_OK) return st;
  return pack_geom(fmt, K, N).total;
}

int qgemm_prepack(int fmt, const void* w, const void* w_scales, void* w_packed, int64_t K,
                  int64_t N, void* stream) {
  if (!valid_format(fmt)) return QGEMM_ERR_FORMAT;
  if (!w_packed) return QGEMM_ERR_NULL;
  int st = check_sizes(fmt, 0, N, K);
  if (st != QGEMM_OK) return st;
  const bool empty = (K == 0 || N == 0);
  if (!empty && !w) return QGEMM_ERR_NULL;
  if ((fmt == QGEMM_MXFP4 || fmt == QGEMM_NVFP4) && !empty && !w_scales) return QGEMM_ERR_NULL;
  if (!aligned(w_packed, 16)) return QGEMM_ERR_ALIGN;
  if (pack_geom(fmt, K, N).total == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  return launched(qgemm::launch_prepack(fmt, w, w_scales, w_packed, K, N, as_stream(stream)));
}

int64_t qgemm_prepack_grouped_bytes(int fmt, int64_t K, int64_t N, int64_t group_k) {
  const int st = check_grouped(fmt, 0, N, K, group_k);
  if (st != QGEMM_OK) return st;
  return grouped_geom(fmt, K, N, group_k).total;
}

int qgemm_prepack_grouped(int fmt, const void* w, const void* scales, const void* zeros,
                          int64_t group_k, int64_t group_n, void* w_packed, int64_t K,
                          int64_t N, void* stream) {
  int st = check_grouped(fmt, 0, N, K, group_k);
  if (st != QGEMM_OK) return st;
  if (group_n < 1 || group_n >= kMaxIndex) return QGEMM_ERR_SHAPE;
  if (!w_packed) return QGEMM_ERR_NULL;
  const bool empty = (K == 0 || N == 0);
  if (!empty && (!w || !scales)) return QGEMM_ERR_NULL;
  if (!aligned(w_packed, 16) || !aligned(w, 16) || !aligned(scales, 16) || !aligned(zeros, 16))
    return QGEMM_ERR_ALIGN;
  if (grouped_geom(fmt, K, N, group_k).total == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  return launched(qgemm::launch_prepack_grouped(fmt, w, scales, zeros, group_k, group_n,
                                                w_packed, K, N, as_stream(stream)));
}

int qgemm_nvfp4(const void* x, const void* w_packed, const float* global_scale, void* y,
                int64_t M, int64_t N, int64_t K, void* stream) {
  int st = check_sizes(QGEMM_NVFP4, M, N, K);
  if (st != QGEMM_OK) return st;
  if (!present(x, M * K) || !present(w_packed, K * N) || !present(y, M * N) || !global_scale)
    return QGEMM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w_packed, 16) || !aligned(y, 16) || !aligned(global_scale, 4))
    return QGEMM_ERR_ALIGN;
  if (M == 0 || N == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  // K % 16 == 0 here, so fp16 X rows are 16-byte aligned
  if (kernel_for(QGEMM_NVFP4, M, N, K, 0) == QGEMM_KERNEL_WEIGHT_ONLY_256)
    return launched(qgemm::launch_weight_only_tile_nvfp4(x, w_packed, global_scale, y, M, N, K,
                                                         as_stream(stream)));
  return launched(qgemm::launch_decode_nvfp4(x, w_packed, global_scale, y, M, N, K,
                                             as_stream(stream)));
}

int qgemm_w4a16_grouped(const void* x, const void* w_packed, void* y, int64_t M, int64_t N,
                        int64_t K, int64_t group_k, void* stream) {
  return grouped_gemm(QGEMM_W4A16_GROUPED, x, w_packed, y, M, N, K, group_k, stream);
}

int qgemm_w8a16_grouped(const void* x, const void* w_packed, void* y, int64_t M, int64_t N,
                        int64_t K, int64_t group_k, void* stream) {
  return grouped_gemm(QGEMM_W8A16_GROUPED, x, w_packed, y, M, N, K, group_k, stream);
}

int qgemm_quantize_mxfp4(const float* x, int64_t rows, int64_t K, uint8_t* codes, uint8_t* e8m0,
                         void* stream) {
  if (rows < 0 || K < 0 || K % 32 != 0) return QGEMM_ERR_SHAPE;
  if (!present(x, rows * K) || !present(codes, rows * K) || !present(e8m0, rows * K))
    return QGEMM_ERR_NULL;
  if (rows >= kMaxIndex || K >= kMaxIndex || rows * K >= kMaxIndex * 4) return QGEMM_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(codes, 16)) return QGEMM_ERR_ALIGN;
  if (rows == 0 || K == 0) return QGEMM_OK;
  int st = check_device();
  if (st != QGEMM_OK) return st;
  return launched(qgemm::launch_quantize_mxfp4(x, rows, K, codes, e8m0, as_stream(stream)));
}

int qgemm_quantize_fp8(const float* x, int64_t count, uint8_t* codes, float* scale,
                       void* stream) {
  if (!scale) return QGEMM_ERR_NULL;
  if (count < 0) return QGEMM_ERR_SHAPE;
  if (count > 0 && (!x || !codes)) return QGEMM_ERR_NULL;
  if (!aligned(scale, 4)) return QGEMM_ERR_ALIGN;
  int st = check_device();
  if (st != QGEMM_OK) return st;
  return launched(qgemm::launch_quantize_fp8(x, count, codes, scale, as_stream(stream)));
}

int qgemm_w4a16(const void* x, const void* w_packed, const void* scales, void* y, int64_t M,
                int64_t N, int64_t K, void* stream) {
  return weight_only(QGEMM_W4A16, x, w_packed, scales, y, M, N, K, stream);
}

int qgemm_w8a16(const void* x, const void* w_packed, const void* scales, void* y, int64_t M,
                int64_t N, int64_t K, void* stream) {
  return weight_only(QGEMM_W8A16, x, w_packed, scales, y, M, N, K, stream);
}

int qgemm_mxfp4(const void* a_codes, const void* a_e8m0, const void* w_packed, void* c,
                int64_t M, int64_t N, int64_t K, void* stream) {
  int st = check_sizes(QGEMM_MXFP4, M, N, K);
  if (st != QGEMM_OK) return st;
  if (!present(a_codes, M * K) || !present(a_e8m0, M * K) || !present(w_packed, K * N) ||
      !present(c, M * N))
    return QGEMM_ERR_NULL;
  if (!aligned(a_codes, 16) || !aligned(w_packed, 16) || !aligned(c, 16)) return QGEMM_ERR_ALIGN;
  if (M == 0 || N == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  if (kernel_for(QGEMM_MXFP4, M, N, K, 0) == QGEMM_KERNEL_SMALL_M)
    return launched(qgemm::launch_decode_gemm(QGEMM_MXFP4, a_codes, w_packed, a_e8m0, nullptr,
                                              nullptr, c, M, N, K, as_stream(stream)));
  return launched(qgemm::launch_tile_gemm(QGEMM_MXFP4, a_codes, a_e8m0, w_packed, nullptr,
                                          nullptr, c, M, N, K, as_stream(stream)));
}

int qgemm_fp8(const void* a, const void* b_packed, const float* scale_a, const float* scale_b,
              void* c, int64_t M, int64_t N, int64_t K, void* stream) {
  int st = check_sizes(QGEMM_FP8, M, N, K);
  if (st != QGEMM_OK) return st;
  if (!present(a, M * K) || !present(b_packed, K * N) || !present(c, M * N) || !scale_a ||
      !scale_b)
    return QGEMM_ERR_NULL;
  if (!aligned(a, 16) || !aligned(b_packed, 16) || !aligned(c, 16)) return QGEMM_ERR_ALIGN;
  if (!aligned(scale_a, 4) || !aligned(scale_b, 4)) return QGEMM_ERR_ALIGN;
  if (M == 0 || N == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  if (kernel_for(QGEMM_FP8, M, N, K, 0) == QGEMM_KERNEL_SMALL_M)
    return launched(qgemm::launch_decode_gemm(QGEMM_FP8, a, b_packed, nullptr, scale_a, scale_b,
                                              c, M, N, K, as_stream(stream)));
  return launched(qgemm::launch_tile_gemm(QGEMM_FP8, a, nullptr, b_packed, scale_a, scale_b, c, M,
                                          N, K, as_stream(stream)));
}

// ---- activation quantization enqueued before the GEMM ----------------------

int64_t qgemm_act_workspace_bytes(int fmt, int64_t M, int64_t K) {
  if (fmt != QGEMM_MXFP4 && fmt != QGEMM_FP8) return QGEMM_ERR_FORMAT;
  if (M < 0 || K < 0 || !k_ok(fmt, K)) return QGEMM_ERR_SHAPE;
  if (M >= kMaxIndex || K >= kMaxIndex || M * K >= kMaxIndex * 2) return QGEMM_ERR_SHAPE;
  if (fmt == QGEMM_MXFP4) return qgemm::cdiv(M * K / 2, 16) * 16 + M * (K / 32);
  return qgemm::cdiv(M * K, 16) * 16 + 16 + 4 * qgemm::kFp8Partials;
}

int qgemm_mxfp4_act(const float* a, const void* w_packed, void* c, void* workspace, int64_t M,
                    int64_t N, int64_t K, void* stream) {
  int st = check_sizes(QGEMM_MXFP4, M, N, K);
  if (st != QGEMM_OK) return st;
  if (!present(a, M * K) || !present(w_packed, K * N) || !present(c, M * N) ||
      !present(workspace, M * K))
    return QGEMM_ERR_NULL;
  if (!aligned(a, 16) || !aligned(w_packed, 16) || !aligned(c, 16) || !aligned(workspace, 16))
    return QGEMM_ERR_ALIGN;
  if (M == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  uint8_t* e8m0 = codes + qgemm::cdiv(M * K / 2, 16) * 16;
  if (K > 0) {
    st = launched(qgemm::launch_quantize_mxfp4(a, M, K, codes, e8m0, as_stream(stream)));
    if (st != QGEMM_OK) return st;
  }
  if (N == 0) return QGEMM_OK;
  if (kernel_for(QGEMM_MXFP4, M, N, K, 0) == QGEMM_KERNEL_SMALL_M)
    return launched(qgemm::launch_decode_gemm(QGEMM_MXFP4, codes, w_packed, e8m0, nullptr,
                                              nullptr, c, M, N, K, as_stream(stream)));
  return launched(qgemm::launch_tile_gemm(QGEMM_MXFP4, codes, e8m0, w_packed, nullptr, nullptr, c,
                                          M, N, K, as_stream(stream)));
}

int qgemm_fp8_act(const float* a, const void* b_packed, const float* scale_b, void* c,
                  void* workspace, int64_t M, int64_t N, int64_t K, void* stream) {
  int st = check_fp8_act(a, b_packed, scale_b, c, M, N, K);
  if (st != QGEMM_OK) return st;
  if (!workspace) return QGEMM_ERR_NULL;
  if (!aligned(workspace, 16)) return QGEMM_ERR_ALIGN;
  if (M == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  return fp8_act_run(a, b_packed, scale_b, c, static_cast<uint8_t*>(workspace), M, N, K, stream);
}

int qgemm_fp8_act_noalloc(const float* a, const void* b_packed, const float* scale_b, void* c,
                          int64_t M, int64_t N, int64_t K, void* stream) {
  int st = check_fp8_act(a, b_packed, scale_b, c, M, N, K);
  if (st != QGEMM_OK) return st;
  if (M * K > QGEMM_FP8_ACT_NOALLOC_MAX_ELEMS) return QGEMM_ERR_TOO_LARGE;
  if (M == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  uint8_t* ws = nullptr;
  if ((st = scratch_of_current_device(&ws)) != QGEMM_OK) return st;
  return fp8_act_run(a, b_packed, scale_b, c, ws, M, N, K, stream);
}

// ---- paged key-value cache ---------------------------------------------------

int qgemm_kv_plan(int32_t* table, const int32_t* cached, const int32_t* added,
                  const int32_t* free_pages, int32_t* lens, int32_t* cu_tokens,
                  int32_t* cu_pages, int64_t* slots, int64_t batch, int64_t width,
                  int64_t table_stride, int64_t num_free, int64_t page_size, int64_t tokens,
                  void* stream) {
  if (!below(batch, 0, kMaxIndex) || !below(width, 0, kMaxIndex) ||
      !below(num_free, 0, kMaxIndex) || !below(page_size, 1, kMaxIndex) ||
      !below(tokens, 0, kMaxIndex) || !below(table_stride, 0, kMaxStride) ||
      (batch > 1 && table_stride < width) ||
      (table_stride > 0 && batch > ((int64_t)1 << 60) / table_stride))   // no such table
    return QGEMM_ERR_SHAPE;
  if (!present(table, batch * width) || !present(cached, batch) || !present(added, batch) ||
      !present(free_pages, num_free) || !present(lens, batch) || !cu_tokens || !cu_pages ||
      !present(slots, tokens))
    return QGEMM_ERR_NULL;
  for (const void* p : {(const void*)table, (const void*)cached, (const void*)added,
                        (const void*)free_pages, (const void*)lens, (const void*)cu_tokens,
                        (const void*)cu_pages})
    if (!aligned(p, 4)) return QGEMM_ERR_ALIGN;
  if (!aligned(slots, 8)) return QGEMM_ERR_ALIGN;
  int st = check_device();
  if (st != QGEMM_OK) return st;
  // The workgroups read the inputs at any time of the launch, so nothing that it
  // writes may lie there: but lens on cached is kept apart by the launch.
  const Span in[] = {{cached, batch}, {added, batch}, {free_pages, num_free}};
  const Span made[] = {{lens, batch}, {cu_tokens, batch + 1}, {cu_pages, batch + 1}, {slots, 2 * tokens}};
  for (const Span& x : in)
    if (meets_rows(x, table, batch, width, table_stride)) return QGEMM_ERR_OVERLAP;
  for (const Span& x : made) {
    if (meets_rows(x, table, batch, width, table_stride)) return QGEMM_ERR_OVERLAP;
    for (const Span& y : in)
      if (x.meets(y) && !(&x == made && &y == in && lens == cached)) return QGEMM_ERR_OVERLAP;
    for (const Span& y : made)
      if (&x != &y && x.meets(y)) return QGEMM_ERR_OVERLAP;
  }
  return launched(qgemm::launch_kv_plan(
      qgemm::KvPlan{table, cached, added, free_pages, lens, cu_tokens, cu_pages, slots, batch,
                    width, table_stride, num_free, page_size, tokens},
      as_stream(stream)));
}

int qgemm_kv_append(int dtype, int cache_dtype, const void* k, const void* v,
                    const int64_t* slots, void* k_cache, void* v_cache, const float* k_scale,
                    const float* v_scale, int64_t tokens, int64_t kv_heads, int64_t dim,
                    int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                    int64_t v_head_stride, int64_t pages, int64_t page_size, int64_t page_stride,
                    int64_t head_stride, int64_t token_stride, void* stream) {
  int st = check_kv_types(dtype, cache_dtype, k_scale, v_scale, kv_heads);
  if (st != QGEMM_OK) return st;
  qgemm::KvPool pool;
  if ((st = check_kv_pool(kv_heads, dim, pages, page_size, page_stride, head_stride, token_stride,
                          &pool)) != QGEMM_OK)
    return st;
  // a thread takes 8 elements; a launch has fewer than 2^32 threads
  if (!below(tokens, 0, kMaxIndex) || tokens * kv_heads >= kMaxIndex / (dim / 8) ||
      !kv_view_ok(k_token_stride, k_head_stride) || !kv_view_ok(v_token_stride, v_head_stride))
    return QGEMM_ERR_SHAPE;
  const bool some = tokens > 0 && kv_heads > 0;
  if (!present(k, some) || !present(v, some) || !present(slots, tokens) ||
      !present(k_cache, some && pages > 0) || !present(v_cache, some && pages > 0))
    return QGEMM_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16))
    return QGEMM_ERR_ALIGN;
  if (!some || pages == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  qgemm::KvAppend a{};
  a.x[0] = k;
  a.x[1] = v;
  a.cache[0] = k_cache;
  a.cache[1] = v_cache;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.token_stride[0] = k_token_stride;
  a.token_stride[1] = v_token_stride;
  a.head_stride[0] = k_head_stride;
  a.head_stride[1] = v_head_stride;
  a.slots = slots;
  a.tokens = tokens;
  a.kv_heads = (int)kv_heads;
  a.dim = (int)dim;
  a.pool = pool;
  return launched(qgemm::launch_kv_append(dtype, cache_dtype, a, as_stream(stream)));
}

int64_t qgemm_paged_attention_workspace_bytes(int64_t batch, int64_t heads, int64_t kv_heads,
                                              int64_t dim, int64_t max_len, int64_t window) {
  if (!below(batch, 0, kMaxIndex) || !below(heads, 0, kMaxIndex) ||
      !below(kv_heads, 1, kMaxIndex) || heads % kv_heads != 0 || !kv_dim_ok(dim) ||
      !below(max_len, 0, kMaxIndex / 2) || !below(window, 0, kMaxIndex) ||
      batch * heads >= kMaxIndex / 256 || batch * qgemm::cdiv(max_len, 32) >= kMaxIndex)
    return QGEMM_ERR_SHAPE;
  return qgemm::paged_attention_workspace(batch, heads, kv_heads, dim, max_len, window);
}

int qgemm_paged_attention(int dtype, int cache_dtype, const void* q, const void* k_cache,
                          const void* v_cache, const int32_t* table, const int32_t* lens,
                          const float* k_scale, const float* v_scale, void* out,
                          void* workspace, int64_t batch, int64_t heads, int64_t kv_heads,
                          int64_t dim, int64_t q_batch_stride, int64_t q_head_stride,
                          int64_t pages, int64_t page_size, int64_t page_stride,
                          int64_t head_stride, int64_t token_stride, int64_t width,
                          int64_t table_stride, int64_t max_len, int64_t window, float scale,
                          void* stream) {
  int st = check_kv_types(dtype, cache_dtype, k_scale, v_scale, kv_heads);
  if (st != QGEMM_OK) return st;
  const int64_t need =
      qgemm_paged_attention_workspace_bytes(batch, heads, kv_heads, dim, max_len, window);
  if (need < 0) return (int)need;
  qgemm::KvPool pool;
  if ((st = check_kv_pool(kv_heads, dim, pages, page_size, page_stride, head_stride, token_stride,
                          &pool)) != QGEMM_OK)
    return st;
  if (!kv_view_ok(q_batch_stride, q_head_stride) || !below(width, 0, kMaxIndex) ||
      !below(table_stride, 0, kMaxStride) || (batch > 1 && table_stride < width))
    return QGEMM_ERR_SHAPE;
  const int64_t rows = batch * heads;
  if (!present(q, rows) || !present(out, rows) || !present(lens, rows) ||
      !present(table, rows > 0 ? width : 0) || !present(k_cache, rows > 0 ? pages : 0) ||
      !present(v_cache, rows > 0 ? pages : 0) || !present(workspace, need))
    return QGEMM_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(workspace, 16) || !aligned(table, 4) || !aligned(lens, 4))
    return QGEMM_ERR_ALIGN;
  if (rows == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  qgemm::PagedAttention a{};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.table = table;
  a.lens = lens;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.out = out;
  a.workspace = workspace;
  a.q_batch_stride = q_batch_stride;
  a.q_head_stride = q_head_stride;
  a.table_stride = table_stride;
  a.batch = (int)batch;
  a.heads = (int)heads;
  a.kv_heads = (int)kv_heads;
  a.dim = (int)dim;
  a.pool = pool;
  a.max_len = max_len;
  a.limit = max_len < width * page_size ? max_len : width * page_size;
  if (pages == 0) a.limit = 0;   // every page is missing
  a.window = window;
  a.scale = scale;
  return launched(qgemm::launch_paged_attention(dtype, cache_dtype, a, as_stream(stream)));
}

// ---- int8 x int8 products, dense and by expert ------------------------------

int qgemm_quantize_int8(int dtype, const void* x, int8_t* codes, float* scale, int64_t rows,
                        int64_t K, int64_t row_stride, void* stream) {
  if (dtype != QGEMM_F16 && dtype != QGEMM_BF16 && dtype != QGEMM_F32) return QGEMM_ERR_FORMAT;
  const int64_t size = dtype == QGEMM_F32 ? 4 : 2;
  if (!below(rows, 0, kMaxIndex) || !below(K, 0, kMaxInt8K + 1) || K % 16 != 0 ||
      !below(row_stride, 0, kMaxStride) || (K > 0 && row_stride * size % 16 != 0) ||
      (row_stride > 0 && rows > ((int64_t)1 << 60) / row_stride))   // no such array
    return QGEMM_ERR_SHAPE;
  if (!present(x, rows * K) || !present(codes, rows * K) || !present(scale, rows))
    return QGEMM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scale, 4)) return QGEMM_ERR_ALIGN;
  if (rows == 0) return QGEMM_OK;
  const int64_t reach = K > 0 ? size * ((rows - 1) * row_stride + K) : 0;
  int st = check_apart({{codes, rows * K}, {scale, 4 * rows}}, {{x, reach}});
  if (st != QGEMM_OK) return st;
  if ((st = check_device()) != QGEMM_OK) return st;
  return launched(qgemm::launch_quantize_int8(dtype, x, row_stride, codes, scale, rows, K,
                                              as_stream(stream)));
}

int64_t qgemm_prepack_w8a8_bytes(int64_t experts, int64_t K, int64_t N, int gated) {
  const int st = check_w8a8_weight(experts, K, N, gated);
  if (st != QGEMM_OK) return st;
  return experts * qgemm::w8a8_geom(K, N, gated).bytes;
}

int qgemm_prepack_w8a8(const int8_t* w, void* w_packed, int64_t experts, int64_t K, int64_t N,
                       int gated, void* stream) {
  int st = check_w8a8_weight(experts, K, N, gated);
  if (st != QGEMM_OK) return st;
  const int64_t bytes = experts * qgemm::w8a8_geom(K, N, gated).bytes;
  if (!present(w, K * N) || !present(w_packed, bytes)) return QGEMM_ERR_NULL;
  if (!aligned(w, 16) || !aligned(w_packed, 16)) return QGEMM_ERR_ALIGN;
  if ((st = check_apart({{w_packed, bytes}}, {{w, experts * K * N}})) != QGEMM_OK) return st;
  if (bytes == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  return launched(qgemm::launch_prepack_w8a8(w, w_packed, experts, K, N, gated != 0, as_stream(stream)));
}

int qgemm_w8a8(int dtype, const int8_t* a, const float* a_scale, const void* w_packed,
               const float* w_scale, void* out, int64_t M, int64_t N, int64_t K, int gated,
               void* stream) {
  return w8a8(dtype, a, a_scale, w_packed, w_scale, nullptr, nullptr, out, M, M, N, K, 0, gated, stream);
}

int qgemm_w8a8_experts(int dtype, const int8_t* a, const float* a_scale, const void* w_packed,
                       const float* w_scale, const int32_t* offsets, const int32_t* rows, void* out,
                       int64_t a_rows, int64_t M, int64_t N, int64_t K, int64_t experts, int gated,
                       void* stream) {
  if (experts < 1) return QGEMM_ERR_SHAPE;
  return w8a8(dtype, a, a_scale, w_packed, w_scale, offsets, rows, out, a_rows, M, N, K, experts, gated,
              stream);
}

int qgemm_w8a8_tile(int64_t M, int64_t N, int64_t K, int64_t experts, int gated, int64_t* rows,
                    int64_t* cols, int64_t* k_split) {
  const int st = check_w8a8_weight(experts == 0 ? 1 : experts, K, N, gated);
  if (st != QGEMM_OK) return st;
  if (!below(M, 0, kMaxInt8Rows) || M * N >= kMaxIndex) return QGEMM_ERR_SHAPE;
  if (!rows || !cols || !k_split) return QGEMM_ERR_NULL;
  static const int32_t some = 0;
  qgemm::W8a8 p{};
  p.offsets = experts == 0 ? nullptr : &some;   // not read
  p.M = M;
  p.N = N;
  p.K = K;
  p.experts = experts == 0 ? 1 : experts;
  p.gated = gated != 0;
  const qgemm::W8a8Tile t = qgemm::w8a8_tile(p);
  *rows = t.rows;
  *cols = t.cols;
  *k_split = t.k_split;
  return QGEMM_OK;
}

int64_t qgemm_expert_plan_workspace_bytes(int64_t pairs, int64_t experts) {
  if (!below(pairs, 0, qgemm::kMaxPairs + 1) || !below(experts, 1, qgemm::kMaxExperts + 1))
    return QGEMM_ERR_SHAPE;
  return qgemm::expert_plan_workspace(pairs, experts);
}

int qgemm_expert_plan(int id_bytes, const void* ids, int32_t* offsets, int32_t* rows,
                      int32_t* places, void* workspace, int64_t tokens, int64_t top,
                      int64_t experts, void* stream) {
  if (id_bytes != 4 && id_bytes != 8) return QGEMM_ERR_FORMAT;
  if (!below(tokens, 0, kMaxIndex) || !below(top, 0, kMaxIndex)) return QGEMM_ERR_SHAPE;
  const int64_t pairs = tokens * top;
  const int64_t need = qgemm_expert_plan_workspace_bytes(pairs, experts);
  if (need < 0) return (int)need;
  if (!present(ids, pairs) || !offsets || !present(rows, pairs) || !present(places, pairs) ||
      !present(workspace, need))
    return QGEMM_ERR_NULL;
  if (!aligned(ids, (uintptr_t)id_bytes) || !aligned(offsets, 4) || !aligned(rows, 4) ||
      !aligned(places, 4) || !aligned(workspace, 16))
    return QGEMM_ERR_ALIGN;
  // ids are read while the outputs are written
  int st = check_apart({{offsets, 4 * (experts + 1)}, {rows, 4 * pairs}, {places, 4 * pairs},
                        {workspace, need}},
                       {{ids, id_bytes * pairs}});
  if (st != QGEMM_OK) return st;
  if ((st = check_device()) != QGEMM_OK) return st;
  return launched(qgemm::launch_expert_plan(
      qgemm::ExpertPlan{ids, id_bytes == 8, offsets, rows, places, static_cast<int32_t*>(workspace),
                        pairs, (int)top, (int)experts},
      as_stream(stream)));
}

int qgemm_expert_combine(int dtype, const void* y, const int32_t* places, const float* gates,
                         void* out, int64_t rows, int64_t tokens, int64_t top, int64_t N,
                         void* stream) {
  if (dtype != QGEMM_F16 && dtype != QGEMM_BF16) return QGEMM_ERR_FORMAT;
  if (!below(rows, 0, kMaxIndex) || !below(tokens, 0, kMaxIndex) || !below(top, 0, kMaxIndex) ||
      !below(N, 0, kMaxIndex) || rows * N >= kMaxIndex || tokens * N >= kMaxIndex ||
      tokens * top >= kMaxIndex)
    return QGEMM_ERR_SHAPE;
  if (!present(y, rows * N) || !present(places, tokens * top) || !present(gates, tokens * top) ||
      !present(out, tokens * N))
    return QGEMM_ERR_NULL;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(places, 4) || !aligned(gates, 4))
    return QGEMM_ERR_ALIGN;
  int st = check_apart({{out, 2 * tokens * N}},
                       {{y, 2 * rows * N}, {places, 4 * tokens * top}, {gates, 4 * tokens * top}});
  if (st != QGEMM_OK) return st;
  if (tokens == 0 || N == 0) return QGEMM_OK;
  if ((st = check_device()) != QGEMM_OK) return st;
  return launched(qgemm::launch_expert_combine(
      dtype,
      qgemm::ExpertCombine{static_cast<const uint16_t*>(y), places, gates, static_cast<uint16_t*>(out),
                           (uint32_t)rows, (uint32_t)tokens, (uint32_t)N, (int)top},
      as_stream(stream)));
}

int qgemm_read_probe(const void* buf, int64_t bytes, uint32_t* sink, int64_t workgroups,
                     void* stream) {
  if (bytes < 0 || bytes % 16 != 0 || workgroups < 1 || workgroups > (1 << 20))
    return QGEMM_ERR_SHAPE;
  if (!present(buf, bytes) || !sink) return QGEMM_ERR_NULL;
  if (!aligned(buf, 16) || !aligned(sink, 4)) return QGEMM_ERR_ALIGN;
  int st = check_device();
  if (st != QGEMM_OK) return st;
  return launched(qgemm::launch_read_probe(buf, bytes, sink, workgroups, as_stream(stream)));
}

int qgemm_mfma_probe(int fmt, const void* operands, int64_t iters, float* sink,
                     int64_t workgroups, void* stream) {
  if (fmt != QGEMM_MXFP4 && fmt != QGEMM_FP8) return QGEMM_ERR_FORMAT;
  if (iters < 0 || workgroups < 1 || workgroups > (1 << 20)) return QGEMM_ERR_SHAPE;
  if (!operands || !sink) return QGEMM_ERR_NULL;
  if (!aligned(operands, 16) || !aligned(sink, 4)) return QGEMM_ERR_ALIGN;
  int st = check_device();
  if (st != QGEMM_OK) return st;
  return launched(qgemm::launch_mfma_probe(fmt == QGEMM_MXFP4, operands, iters, sink, workgroups,
                                           as_stream(stream)));
}

}  // extern "C"
