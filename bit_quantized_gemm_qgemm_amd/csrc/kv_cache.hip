// Writing side of the paged key-value cache: block tables and slots of the
// tokens that enter a step, and the tokens' keys and values into their slots.
#include "qgemm_common.h"

namespace qgemm {
namespace {

// ---------------------------------------------------------------------------
// Plan: two running sums over the requests (tokens gained, pages gained), then
// one slot per token.
// ---------------------------------------------------------------------------
// The workgroup walks the requests 256 at a time, one per thread, carrying
// the sums of the tiles before; a tile's sums stay in LDS, where each token of
// the tile finds its request by binary search.  A page that a request gains
// starts at one of its new tokens (the first position that the held pages do
// not cover is not before the first new one), so the thread of the token at a
// page's first position writes the table entry, and every thread takes the
// number of a new page from the free list itself: nothing is read that this
// launch writes.
constexpr int kPlanThreads = 256;

struct PlanTile {
  int64_t tok[kPlanThreads + 1];    // tokens of the requests before, within all
  int64_t page[kPlanThreads];       // pages gained by the requests before
  int cached[kPlanThreads];
  int have[kPlanThreads];
  int64_t wave[2][kPlanThreads / kWave];
};

__global__ __launch_bounds__(kPlanThreads) void kv_plan_kernel(const KvPlan p) {
  __shared__ PlanTile s;
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t capacity = p.width * p.page_size;
  int64_t tok0 = 0, page0 = 0;
  for (int64_t b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
    const int64_t b = b0 + tid;
    int64_t cached = 0, added = 0, have = 0, take = 0;
    if (b < p.batch) {
      cached = p.cached[b] > 0 ? p.cached[b] : 0;
      added = p.added[b] > 0 ? p.added[b] : 0;
      const int64_t len = cached + added < capacity ? cached + added : capacity;
      have = cdiv(cached, p.page_size);
      have = have < p.width ? have : p.width;
      take = cdiv(len, p.page_size) - have;
      take = take > 0 ? take : 0;
      p.lens[b] = (int32_t)len;
    }
    int64_t tok = added, page = take;   // inclusive sums over the wave, then the tile
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int64_t t = __shfl_up(tok, off, kWave), q = __shfl_up(page, off, kWave);
      if (lane >= off) {
        tok += t;
        page += q;
      }
    }
    if (lane == 63) {
      s.wave[0][wave] = tok;
      s.wave[1][wave] = page;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
      tok += s.wave[0][w];
      page += s.wave[1][w];
    }
    s.tok[tid + 1] = tok0 + tok;
    s.page[tid] = page0 + page - take;
    s.cached[tid] = (int)cached;
    s.have[tid] = (int)have;
    if (tid == 0) s.tok[0] = tok0;
    if (b < p.batch) {
      p.cu_tokens[b] = (int32_t)(tok0 + tok - added);
      p.cu_pages[b] = (int32_t)(page0 + page - take);
    }
    if (tid == kPlanThreads - 1) s.wave[1][0] = page;   // the tile's pages, read after the barrier
    __syncthreads();
    const int64_t tile_pages = s.wave[1][0], tok_end = s.tok[kPlanThreads];
    for (int64_t t = tok0 + tid; t < tok_end; t += kPlanThreads) {
      int lo = 0, hi = kPlanThreads;   // the last request whose first token is not past t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.tok[mid] <= t) lo = mid; else hi = mid;
      }
      const int64_t pos = s.cached[lo] + (t - s.tok[lo]);
      int64_t slot = -1;
      if (pos < capacity) {
        const int64_t pi = pos / p.page_size, off = pos - pi * p.page_size;
        int32_t* entry = p.table + (b0 + lo) * p.table_stride + pi;
        int32_t page_no;
        if (pi < s.have[lo]) {
          page_no = *entry;
        } else {
          const int64_t f = s.page[lo] + pi - s.have[lo];
          page_no = f < p.num_free ? p.free_pages[f] : -1;
          if (off == 0) *entry = page_no;
        }
        if (page_no >= 0) slot = (int64_t)page_no * p.page_size + off;
      }
      if (t < p.tokens) p.slots[t] = slot;
    }
    tok0 = tok_end;
    page0 += tile_pages;
    __syncthreads();   // the tile is rewritten next
  }
  if (tid == 0) {
    p.cu_tokens[p.batch] = (int32_t)tok0;
    p.cu_pages[p.batch] = (int32_t)page0;
  }
  for (int64_t t = tok0 + tid; t < p.tokens; t += kPlanThreads) p.slots[t] = -1;
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
// fp32 -> e4m3fn: nearest even, saturated at +-448, NaN kept.
__device__ __forceinline__ uint32_t e4m3_code(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v), sign = (u >> 24) & 0x80u;
  const float a = fabsf(v);
  if (!(a == a)) return sign | 0x7fu;
  if (a >= 448.0f) return sign | 0x7eu;
  if (a < 0.015625f) return sign | (uint32_t)__builtin_rintf(a * 512.0f);   // step 2^-9
  const uint32_t ua = __builtin_bit_cast(uint32_t, a);
  return sign | (((ua + 0x7ffffu + ((ua >> 20) & 1u)) >> 20) - (120u << 3));
}

template <int DT>
__device__ __forceinline__ float to_float(uint16_t bits) {
  if constexpr (DT == 1) return (float)__builtin_bit_cast(_Float16, bits);
  return __builtin_bit_cast(float, (uint32_t)bits << 16);
}

// One thread per 8 elements of one row (token, kv head), for keys
// (blockIdx.y = 0) and values (1).
template <int DT, bool E4M3>
__global__ __launch_bounds__(256) void kv_append_kernel(const KvAppend a) {
  const int part = (int)blockIdx.y;
  const int chunks = a.dim / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.tokens * a.kv_heads * chunks) return;
  const int c = (int)(i % chunks);
  const int h = (int)(i / chunks % a.kv_heads);
  const int64_t t = i / chunks / a.kv_heads;
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= (int64_t)a.pool.pages * a.pool.page_size) return;
  const int64_t page = slot / a.pool.page_size, off = slot - page * a.pool.page_size;
  const int64_t row = page * a.pool.page_rows + (int64_t)h * a.pool.head_rows +
                      off * a.pool.token_rows;
  const uint16_t* x = static_cast<const uint16_t*>(a.x[part]) + t * a.token_stride[part] +
                      h * a.head_stride[part] + 8 * c;
  const uintx4 v = *reinterpret_cast<const uintx4*>(x);
  if constexpr (!E4M3) {
    uint16_t* y = static_cast<uint16_t*>(a.cache[part]) + row * a.dim + 8 * c;
    *reinterpret_cast<uintx4*>(y) = v;
  } else {
    const float scale = a.scale[part][h];
    uintx2 w = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = to_float<DT>((uint16_t)(v[j >> 1] >> (16 * (j & 1))));
      w[j >> 2] |= e4m3_code(f / scale) << (8 * (j & 3));
    }
    uint8_t* y = static_cast<uint8_t*>(a.cache[part]) + row * a.dim + 8 * c;
    *reinterpret_cast<uintx2*>(y) = w;
  }
}

}  // namespace

hipError_t launch_kv_plan(const KvPlan& p, hipStream_t stream) {
  hipLaunchKernelGGL(kv_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_kv_append(int dtype, int cache_dtype, const KvAppend& a, hipStream_t stream) {
  const dim3 grid((unsigned)cdiv(a.tokens * a.kv_heads * (a.dim / 8), 256), 2), block(256);
  const bool e4m3 = cache_dtype == 3;
  auto kernel = dtype == 1 ? (e4m3 ? kv_append_kernel<1, true> : kv_append_kernel<1, false>)
                           : (e4m3 ? kv_append_kernel<2, true> : kv_append_kernel<2, false>);
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace qgemm
