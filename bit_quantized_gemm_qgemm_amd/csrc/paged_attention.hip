// Attention of one new token per request over the paged key-value cache.
#include "qgemm_common.h"

namespace qgemm {
namespace {

constexpr int kAttnWaves = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int DT>
__device__ __forceinline__ float to_float(uint16_t bits) {
  if constexpr (DT == 1) return (float)__builtin_bit_cast(_Float16, bits);
  return __builtin_bit_cast(float, (uint32_t)bits << 16);
}

// e4m3fn code -> its value: the seven low bits read as an fp16 (bias 15
// instead of 7) are value * 2^-8, subnormals included
__device__ __forceinline__ float e4m3_value(uint8_t code) {
  const uint32_t m = code & 0x7fu;
  if (m == 0x7fu) return __builtin_nanf("");
  const float v = (float)__builtin_bit_cast(_Float16, (uint16_t)(m << 7)) * 256.0f;
  return code & 0x80u ? -v : v;
}

template <int DT, bool E4M3>
__device__ __forceinline__ float cache_value(const void* cache, int64_t i) {
  if constexpr (E4M3) return e4m3_value(static_cast<const uint8_t*>(cache)[i]);
  return to_float<DT>(static_cast<const uint16_t*>(cache)[i]);
}

// One workgroup per (head, request); its waves take tokens in turn, a lane
// holding the elements lane + 64 j of the row.  Each wave keeps the running
// maximum m, the sum l of exp(s - m) and the weighted sum of the values; the
// waves are joined through LDS at the end.
template <int DT, bool E4M3>
__global__ __launch_bounds__(64 * kAttnWaves) void paged_attention_kernel(const PagedAttention a) {
  __shared__ float sm[kAttnWaves], sl[kAttnWaves], so[kAttnWaves][256];
  const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
  const int head = (int)blockIdx.x, b = (int)blockIdx.y;
  const int kvh = head / (a.heads / a.kv_heads);
  int64_t n = a.lens[b];
  n = n < 0 ? 0 : (n < a.limit ? n : a.limit);
  const int64_t first = a.window > 0 && n > a.window ? n - a.window : 0;
  const float kscale = (E4M3 ? a.k_scale[kvh] : 1.0f) * a.scale * kLog2e;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + b * a.q_batch_stride +
                      head * a.q_head_stride;
  float qv[4], o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) qv[j] = lane + 64 * j < a.dim ? to_float<DT>(q[lane + 64 * j]) : 0.f;
  float m = -INFINITY, l = 0.f;
  for (int64_t t = first + wave; t < n; t += kAttnWaves) {
    const int64_t pi = t / a.pool.page_size, off = t - pi * a.pool.page_size;
    const int32_t page = a.table[b * a.table_stride + pi];
    if (page < 0 || page >= a.pool.pages) continue;
    const int64_t row = (int64_t)page * a.pool.page_rows + (int64_t)kvh * a.pool.head_rows +
                        off * a.pool.token_rows;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 64 * j < a.dim)
        s += qv[j] * cache_value<DT, E4M3>(a.k_cache, row * a.dim + lane + 64 * j);
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) s += __shfl_xor(s, x, 64);
    s *= kscale;
    const float top = fmaxf(m, s);
    const float base = top == -INFINITY ? 0.f : top;
    const float shrink = exp2f(m - base), p = exp2f(s - base);
    m = top;
    l = l * shrink + p;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 64 * j < a.dim)
        o[j] = o[j] * shrink + p * cache_value<DT, E4M3>(a.v_cache, row * a.dim + lane + 64 * j);
  }
  if (lane == 0) {
    sm[wave] = m;
    sl[wave] = l;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) so[wave][lane + 64 * j] = o[j];
  __syncthreads();
  const int d = (int)threadIdx.x;
  if (d >= a.dim) return;
  float top = -INFINITY;
  for (int w = 0; w < kAttnWaves; ++w) top = fmaxf(top, sm[w]);
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc = 0.f;
  for (int w = 0; w < kAttnWaves; ++w) {
    const float f = exp2f(sm[w] - base);
    sum += f * sl[w];
    acc += f * so[w][d];
  }
  const float y = sum == 0.f ? 0.f : acc / sum * (E4M3 ? a.v_scale[kvh] : 1.0f);
  static_cast<uint16_t*>(a.out)[((int64_t)b * a.heads + head) * a.dim + d] =
      DT == 1 ? f32_to_f16_bits(y) : f32_to_bf16_rne(y);
}

}  // namespace

int64_t paged_attention_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) {
  return 0;
}

hipError_t launch_paged_attention(int dtype, int cache_dtype, const PagedAttention& a,
                                  hipStream_t stream) {
  const dim3 grid((unsigned)a.heads, (unsigned)a.batch), block(64 * kAttnWaves);
  const bool e4m3 = cache_dtype == 3;
  auto kernel =
      dtype == 1 ? (e4m3 ? paged_attention_kernel<1, true> : paged_attention_kernel<1, false>)
                 : (e4m3 ? paged_attention_kernel<2, true> : paged_attention_kernel<2, false>);
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace qgemm
