// Writing side of the paged key-value cache: block tables and slots of the
// tokens that enter a step, and the tokens' keys and values into their slots.
#include "qgemm_common.h"

namespace qgemm {
namespace {

// ---------------------------------------------------------------------------
// Plan: two running sums over the requests (tokens gained, pages gained), then
// one slot per token.
// ---------------------------------------------------------------------------
// A workgroup walks the requests a tile at a time, one per thread, carrying
// the sums of the tiles before; a tile's sums stay in LDS, where each token of
// the tile finds its request by binary search.  A page that a request gains
// starts at one of its new tokens (the first position that the held pages do
// not cover is not before the first new one), so the thread of the token at a
// page's first position writes the table entry, and every thread takes the
// number of a new page from the free list itself: nothing is read that this
// launch writes.  (Lengths updated in place would be, by the other workgroups: a
// lone one reads each count once, in the thread that then writes it; for more,
// kv_lens_kernel writes them in a launch of its own, 1.6 us for 3000 requests.)
//
// Several workgroups share the tokens in equal slices.  Each forms the sums
// itself (8 bytes a request, from L2) up to the end of its slice, so none
// waits for another; the first also writes them out.  The slices end at the
// host's count of tokens: where the device's sum is past it, the last workgroup
// writes the pages that begin there, page by page, so the time is bounded by
// the table whatever the counts say.
//
// All of it is latency: a tile costs two loads one after the other, two
// barriers and the search.  So one tile and one token per thread where that is
// possible: 1000 requests of a token each take one tile of 1024 instead of four
// of 256, 131K tokens one token a thread instead of four.  Up to 256 of both
// keep the smaller workgroup (8 requests: 3.3 us, 4.6 with 1024 threads).  Then
// LDS: sums by moves between lanes and a token that tries its own request first
// took 1000 requests from 6.0 to 4.7 us, 131K tokens from 5.8 to 5.0, 8 requests
// from 3.3 to 3.0.
constexpr int kPlanThreadsSmall = 256, kPlanThreads = 1024;
constexpr int kPlanGroups = 256;       // workgroups at most, one a CU

// x of the lane that a DPP control names, 0 where it names none or the row is
// masked out.  VALU moves: as shuffles through LDS the 16 waves' sums stood in
// line there for a third of a tile's time.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ int64_t moved(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, CTRL, ROWS, 0xf, false);
  const uint32_t hi =
      __builtin_amdgcn_update_dpp(0, (int)(uint32_t)((uint64_t)x >> 32), CTRL, ROWS, 0xf, false);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Inclusive sums over 16 lanes, by shifts of 1, 2, 4 and 8 within the row.
__device__ __forceinline__ int64_t sums_of_row(int64_t x) {
  x += moved<0x111>(x);
  x += moved<0x112>(x);
  x += moved<0x114>(x);
  x += moved<0x118>(x);
  return x;
}

// Over the wave: the last lane of a row goes to the next one (rows 1 and 3),
// then lane 31 to the upper half.
__device__ __forceinline__ int64_t sums_of_wave(int64_t x) {
  x = sums_of_row(x);
  x += moved<0x142, 0xa>(x);
  x += moved<0x143, 0xc>(x);
  return x;
}

__device__ __forceinline__ int64_t lane_of(int64_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)x, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)x >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Tokens of a request after the step.
__device__ __forceinline__ int64_t length_after(int64_t cached, int64_t added, int64_t capacity) {
  return cached + added < capacity ? cached + added : capacity;
}

__device__ __forceinline__ int64_t count_of(const int32_t* counts, int64_t b) {
  return counts[b] > 0 ? counts[b] : 0;
}

template <int THREADS>
struct PlanTile {
  int64_t tok[THREADS + 1];    // tokens of the requests before, within all
  int64_t page[THREADS];       // pages gained by the requests before
  int cached[THREADS];
  int have[THREADS];
  int64_t wave[2][THREADS / kWave];   // 16 waves at most
  int64_t pages;               // of the whole tile
};

template <int THREADS>
__global__ __launch_bounds__(THREADS) void kv_plan_kernel(const KvPlan p, int64_t slice) {
  __shared__ PlanTile<THREADS> s;
  constexpr int kWaves = THREADS / kWave;
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t capacity = p.width * p.page_size;
  const uint32_t P = (uint32_t)p.page_size;
  const bool first = blockIdx.x == 0, last = blockIdx.x == gridDim.x - 1;
  const int64_t from = blockIdx.x * slice, to = from + slice < p.tokens ? from + slice : p.tokens;
  int64_t tok0 = 0, page0 = 0;
  for (int64_t b0 = 0; b0 < p.batch && (first || last || tok0 < to); b0 += THREADS) {
    const int64_t b = b0 + tid;
    int64_t cached = 0, added = 0, have = 0, take = 0;
    if (b < p.batch) {
      cached = count_of(p.cached, b);
      added = count_of(p.added, b);
      const int64_t len = length_after(cached, added, capacity);
      // both counts are below 2^32, so the pages are too
      have = ((uint32_t)cached + (P - 1)) / P;
      have = have < p.width ? have : p.width;
      take = (int64_t)(((uint64_t)len + (P - 1)) / P) - have;
      take = take > 0 ? take : 0;
      if (first && p.lens) p.lens[b] = (int32_t)len;
    }
    int64_t tok = sums_of_wave(added), page = sums_of_wave(take);
    if (lane == 63) {
      s.wave[0][wave] = tok;
      s.wave[1][wave] = page;
    }
    __syncthreads();
    if (wave > 0) {   // lane w brings wave w's total
      const bool some = (lane & 15) < kWaves;
      tok += lane_of(sums_of_row(some ? s.wave[0][lane & 15] : 0), wave - 1);
      page += lane_of(sums_of_row(some ? s.wave[1][lane & 15] : 0), wave - 1);
    }
    s.tok[tid + 1] = tok0 + tok;
    s.page[tid] = page0 + page - take;
    s.cached[tid] = (int)cached;
    s.have[tid] = (int)have;
    if (tid == 0) s.tok[0] = tok0;
    if (tid == THREADS - 1) s.pages = page;
    if (first && b < p.batch) {
      p.cu_tokens[b] = (int32_t)(tok0 + tok - added);
      p.cu_pages[b] = (int32_t)(page0 + page - take);
    }
    __syncthreads();
    const int64_t tile_pages = s.pages, tok_end = s.tok[THREADS];
    const int64_t t1 = tok_end < to ? tok_end : to;
    const int filled = p.batch - b0 < THREADS ? (int)(p.batch - b0) : THREADS;
    for (int64_t t = (tok0 > from ? tok0 : from) + tid; t < t1; t += THREADS) {
      // the last request whose first token is not past t; where every request
      // gains one token it is this thread's own
      int lo = 0, hi = filled;
      if (tid < filled && s.tok[tid] <= t && t < s.tok[tid + 1]) {
        lo = tid;
        hi = tid + 1;
      }
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.tok[mid] <= t) lo = mid; else hi = mid;
      }
      const int64_t pos = s.cached[lo] + (t - s.tok[lo]);   // below 2^32
      int64_t slot = -1;
      if (pos < capacity) {
        const uint32_t pi = (uint32_t)pos / P, off = (uint32_t)pos - pi * P;
        int32_t* entry = p.table + (b0 + lo) * p.table_stride + pi;
        int32_t page_no;
        if (pi < (uint32_t)s.have[lo]) {
          page_no = *entry;
        } else {
          const int64_t f = s.page[lo] + pi - s.have[lo];
          page_no = f < p.num_free ? p.free_pages[f] : -1;
          if (off == 0) *entry = page_no;
        }
        if (page_no >= 0) slot = (int64_t)page_no * p.page_size + off;
      }
      p.slots[t] = slot;
    }
    if (last && tok_end > p.tokens) {
      for (int64_t x = tid; x < tile_pages; x += THREADS) {
        const int64_t f = page0 + x;
        int lo = 0, hi = filled;   // the last request whose first page is not past f
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s.page[mid] <= f) lo = mid; else hi = mid;
        }
        const int64_t pi = s.have[lo] + (f - s.page[lo]);
        if (s.tok[lo] + pi * p.page_size - s.cached[lo] >= p.tokens)
          p.table[(b0 + lo) * p.table_stride + pi] = f < p.num_free ? p.free_pages[f] : -1;
      }
    }
    tok0 = tok_end;
    page0 += tile_pages;
    __syncthreads();   // the tile is rewritten next
  }
  if (first && tid == 0) {
    p.cu_tokens[p.batch] = (int32_t)tok0;
    p.cu_pages[p.batch] = (int32_t)page0;
  }
  // slots past the last token (the sums are complete where this runs at all)
  for (int64_t t = (tok0 > from ? tok0 : from) + tid; t < to; t += THREADS) p.slots[t] = -1;
}

__global__ __launch_bounds__(256) void kv_lens_kernel(const KvPlan p) {
  const int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (b < p.batch)
    p.lens[b] = (int32_t)length_after(count_of(p.cached, b), count_of(p.added, b), p.width * p.page_size);
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
// fp32 x / s of one divisor for many x, correctly rounded.  With r the rounded
// reciprocal, q = x r is within two steps of x / s; one fused correction by the
// remainder x - q s brings it within one, and a second, whose remainder is then
// exact, rounds as the division would: 5 instructions where the division takes
// 10, which bounded the append (8192 tokens of 8 x 128: 16.9 -> 11.6 us, the
// hardware's conversion included).  That holds while no remainder underflows and
// nothing overflows: for |s| in 2^-60 .. 2^60 wherever the quotient reaches
// 2^-11 (below it the code is 0) and stays below 512 (above it the code is
// 448's).  Any other s divides.
struct Divisor {
  float s, r;
  bool usual;
  __device__ __forceinline__ explicit Divisor(float scale)
      : s(scale), r(1.0f / scale), usual(fabsf(scale) >= 0x1p-60f && fabsf(scale) <= 0x1p60f) {}
};

__device__ __forceinline__ float quotient(float x, const Divisor& d) {
  const float far = x * d.r;
  float q = __builtin_fmaf(__builtin_fmaf(-far, d.s, x), d.r, far);
  q = __builtin_fmaf(__builtin_fmaf(-q, d.s, x), d.r, q);
  return fabsf(far) < 512.0f ? __builtin_copysignf(q, far) : far;   // far: also NaN and infinities
}

// Held to +-448, NaN kept: what the conversion takes without overflow.
__device__ __forceinline__ float saturated(float q) {
  return q == q ? __builtin_amdgcn_fmed3f(q, -448.0f, 448.0f) : q;
}

template <int DT>
__device__ __forceinline__ float to_float(uint16_t bits) {
  if constexpr (DT == 1) return (float)__builtin_bit_cast(_Float16, bits);
  return __builtin_bit_cast(float, (uint32_t)bits << 16);
}

// A thread moves 8 elements of one row (token, kv head), of the keys and of
// the values: the row's number, its slot and its place in the pool are found
// once for both, and two 16-byte loads are in flight.
template <int DT, bool E4M3>
__global__ __launch_bounds__(256) void kv_append_kernel(const KvAppend a, int rows_per_group) {
  const int chunks = a.dim / 8;
  const int local = (int)threadIdx.x / chunks, c = (int)threadIdx.x - local * chunks;
  const int64_t rows = a.tokens * a.kv_heads;   // below 2^31
  const int64_t n = (int64_t)blockIdx.x * rows_per_group + local;
  if (local >= rows_per_group || n >= rows) return;
  const uint32_t t = (uint32_t)n / (uint32_t)a.kv_heads;
  const int h = (int)((uint32_t)n - t * (uint32_t)a.kv_heads);
  uintx4 v[2];
#pragma unroll
  for (int part = 0; part < 2; ++part)
    v[part] = *reinterpret_cast<const uintx4*>(static_cast<const uint16_t*>(a.x[part]) +
                                               t * a.token_stride[part] +
                                               h * a.head_stride[part] + 8 * c);
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= (int64_t)a.pool.pages * a.pool.page_size) return;
  const uint32_t page = (uint32_t)slot / (uint32_t)a.pool.page_size;
  const uint32_t off = (uint32_t)slot - page * (uint32_t)a.pool.page_size;
  const int64_t at = (int64_t)(page * (uint32_t)a.pool.page_rows +
                               (uint32_t)h * (uint32_t)a.pool.head_rows +
                               off * (uint32_t)a.pool.token_rows) * a.dim + 8 * c;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    if constexpr (!E4M3) {
      *reinterpret_cast<uintx4*>(static_cast<uint16_t*>(a.cache[part]) + at) = v[part];
    } else {
      const Divisor d(a.scale[part][h]);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = to_float<DT>((uint16_t)(v[part][j >> 1] >> (16 * (j & 1))));
      if (d.usual) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = quotient(f[j], d);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] /= d.s;
      }
      uintx2 w;
#pragma unroll
      for (int j = 0; j < 2; ++j) {   // the conversion rounds to nearest even
        int x = __builtin_amdgcn_cvt_pk_fp8_f32(saturated(f[4 * j]), saturated(f[4 * j + 1]), 0, false);
        x = __builtin_amdgcn_cvt_pk_fp8_f32(saturated(f[4 * j + 2]), saturated(f[4 * j + 3]), x, true);
        w[j] = (uint32_t)x;
      }
      *reinterpret_cast<uintx2*>(static_cast<uint8_t*>(a.cache[part]) + at) = w;
    }
  }
}

}  // namespace

hipError_t launch_kv_plan(const KvPlan& p, hipStream_t stream) {
  const bool small = p.batch <= kPlanThreadsSmall && p.tokens <= kPlanThreadsSmall;
  int64_t groups = small ? 1 : cdiv(p.tokens, kPlanThreads);
  groups = groups < 1 ? 1 : groups < kPlanGroups ? groups : kPlanGroups;
  const dim3 grid((unsigned)groups);
  KvPlan q = p;
  const bool lens_after = groups > 1 && p.lens == p.cached;
  if (lens_after) q.lens = nullptr;
  if (small)
    hipLaunchKernelGGL((kv_plan_kernel<kPlanThreadsSmall>), grid, dim3(kPlanThreadsSmall), 0, stream,
                       q, p.tokens);
  else
    hipLaunchKernelGGL((kv_plan_kernel<kPlanThreads>), grid, dim3(kPlanThreads), 0, stream, q,
                       cdiv(p.tokens, groups));
  if (lens_after && p.batch > 0)
    hipLaunchKernelGGL(kv_lens_kernel, dim3((unsigned)cdiv(p.batch, 256)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_kv_append(int dtype, int cache_dtype, const KvAppend& a, hipStream_t stream) {
  const int rows = 256 / (a.dim / 8);   // whole rows of a workgroup
  const dim3 grid((unsigned)cdiv(a.tokens * a.kv_heads, rows)), block(256);
  const bool e4m3 = cache_dtype == 3;
  auto kernel = dtype == 1 ? (e4m3 ? kv_append_kernel<1, true> : kv_append_kernel<1, false>)
                           : (e4m3 ? kv_append_kernel<2, true> : kv_append_kernel<2, false>);
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, a, rows);
  return hipGetLastError();
}

}  // namespace qgemm
