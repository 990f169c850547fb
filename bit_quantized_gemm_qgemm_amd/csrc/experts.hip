// Routing around the products grouped by expert: the order of a batch's rows,
// and the sum of each token's expert outputs.
#include "qgemm_common.h"

namespace qgemm {
namespace {

// ---------------------------------------------------------------------------
// Plan
// ---------------------------------------------------------------------------
// A stable counting sort of the pairs (token, choice) by their expert.  A wave
// takes 64 pairs at a time, in order.  The lanes that hold the same expert find
// each other by one ballot for each bit of its number; a pair's place among the
// wave's pairs of its expert is the count so far plus the lanes before it, and
// the first of the lanes adds them to the count.  So each wave keeps counts of
// its own and nothing is added by more than one lane: no atomics, and the order
// is the pairs' own.  The counts of the waves (and of the workgroups before, which
// a launch of its own has left in the workspace) then become places.
constexpr int kPlanRounds = 8;   // pairs of a lane, kept in registers

template <int THREADS>
struct PlanState {
  static constexpr int kWaves = THREADS / 64;
  int e[kPlanRounds];      // expert, or -1
  int at[kPlanRounds];     // place among the wave's pairs of that expert
};

// counts[wave][experts] in LDS; pair (wave * kPlanRounds + r) * 64 + lane of the
// workgroup's share
template <int THREADS>
__device__ __forceinline__ void count_pairs(PlanState<THREADS>& s, const ExpertPlan& p, int64_t first,
                                            int* counts) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < PlanState<THREADS>::kWaves * p.experts; i += THREADS) counts[i] = 0;
  const int bits = 32 - __builtin_clz(p.experts);   // of 0 .. experts
#pragma unroll
  for (int r = 0; r < kPlanRounds; ++r) {
    const int64_t i = first + (wave * kPlanRounds + r) * 64 + lane;
    int64_t id = -1;
    if (i < p.pairs)
      id = p.wide ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
    s.e[r] = id >= 0 && id < p.experts ? (int)id : -1;
  }
  __syncthreads();
  volatile int* mine = counts + wave * p.experts;
#pragma unroll
  for (int r = 0; r < kPlanRounds; ++r) {
    const bool some = s.e[r] >= 0;
    uint64_t same = __ballot(some);
    if (same == 0) {   // the wave's share has ended
      s.at[r] = 0;
      continue;
    }
    for (int b = 0; b < bits; ++b) {
      const bool bit = (s.e[r] >> b) & 1;
      const uint64_t set = __ballot(bit);
      same &= bit ? set : ~set;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    int so_far = 0;
    if (some) so_far = mine[s.e[r]];
    s.at[r] = so_far + before;
    __builtin_amdgcn_wave_barrier();   // all lanes have read
    if (some && before == 0) mine[s.e[r]] = so_far + __popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
}

template <int THREADS, int EXPERTS>
__global__ __launch_bounds__(THREADS) void expert_count_kernel(const ExpertPlan p) {
  __shared__ int counts[PlanState<THREADS>::kWaves * EXPERTS];
  PlanState<THREADS> s;
  count_pairs<THREADS>(s, p, (int64_t)blockIdx.x * THREADS * kPlanRounds, counts);
  for (int e = threadIdx.x; e < p.experts; e += THREADS) {
    int n = 0;
    for (int w = 0; w < PlanState<THREADS>::kWaves; ++w) n += counts[w * p.experts + e];
    p.counts[(int64_t)blockIdx.x * p.experts + e] = n;
  }
}

template <int THREADS, int EXPERTS>
__global__ __launch_bounds__(THREADS) void expert_place_kernel(const ExpertPlan p) {
  constexpr int kWaves = PlanState<THREADS>::kWaves;
  __shared__ int counts[kWaves * EXPERTS];
  __shared__ int wave_sum[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t first = (int64_t)blockIdx.x * THREADS * kPlanRounds;
  PlanState<THREADS> s;
  count_pairs<THREADS>(s, p, first, counts);

  // sums over the experts, THREADS of them at a time
  int before = 0;   // pairs of the experts of the rounds before
  for (int e0 = 0; e0 < p.experts; e0 += THREADS) {
    const int e = e0 + tid;
    int own = 0, earlier = 0, all = 0;   // this workgroup's, those of the ones before it, everyone's
    if (e < p.experts) {
      for (int w = 0; w < kWaves; ++w) own += counts[w * p.experts + e];
      all = own;
      if (gridDim.x > 1) {
        all = 0;
        for (int b = 0; b < (int)gridDim.x; ++b) {
          const int n = p.counts[(int64_t)b * p.experts + e];
          all += n;
          if (b < (int)blockIdx.x) earlier += n;
        }
      }
    }
    int upto = all;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    if (lane == 63) wave_sum[wave] = upto;
    __syncthreads();
    int base = before;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) base += wave_sum[w];
      before += wave_sum[w];
    }
    if (e < p.experts) {
      int at = base + upto - all;
      if (blockIdx.x == 0) p.offsets[e] = at;
      at += earlier;
      for (int w = 0; w < kWaves; ++w) {
        const int n = counts[w * p.experts + e];
        counts[w * p.experts + e] = at;
        at += n;
      }
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.experts] = before;
#pragma unroll
  for (int r = 0; r < kPlanRounds; ++r) {
    const int64_t i = first + (wave * kPlanRounds + r) * 64 + lane;
    if (i >= p.pairs) break;
    int place = -1;
    if (s.e[r] >= 0) {
      place = counts[wave * p.experts + s.e[r]] + s.at[r];
      p.rows[place] = (int32_t)((uint32_t)i / (uint32_t)p.top);
    }
    p.places[i] = place;
    if (i >= before) p.rows[i] = -1;   // past the last row
  }
}

// ---------------------------------------------------------------------------
// Combine
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ float to_float(uint16_t bits) {
  if constexpr (DT == 1) return (float)__builtin_bit_cast(_Float16, bits);
  return __builtin_bit_cast(float, (uint32_t)bits << 16);
}

template <int DT>
__device__ __forceinline__ uint16_t from_float(float v) {
  return DT == 1 ? f32_to_f16_bits(v) : f32_to_bf16_rne(v);
}

// out[t, n] = sum_j gates[t, j] * y[places[t, j], n] in fp32, in the order of j;
// one element a thread.
template <int DT>
__global__ __launch_bounds__(256) void expert_combine_kernel(const ExpertCombine p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.tokens * p.N) return;
  const int64_t t = i / p.N, n = i - t * p.N;
  float sum = 0.f;
  for (int j = 0; j < p.top; ++j) {
    const int place = p.places[t * p.top + j];
    if (place >= 0 && place < p.rows)
      sum = __builtin_fmaf(p.gates[t * p.top + j], to_float<DT>(p.y[place * p.N + n]), sum);
  }
  p.out[i] = from_float<DT>(sum);
}

template <int THREADS, int EXPERTS>
hipError_t launch_plan(const ExpertPlan& p, hipStream_t stream) {
  const int64_t groups = cdiv(p.pairs, THREADS * kPlanRounds);
  const dim3 grid((unsigned)(groups > 0 ? groups : 1));
  if (groups > 1)
    hipLaunchKernelGGL((expert_count_kernel<THREADS, EXPERTS>), grid, dim3(THREADS), 0, stream, p);
  hipLaunchKernelGGL((expert_place_kernel<THREADS, EXPERTS>), grid, dim3(THREADS), 0, stream, p);
  return hipGetLastError();
}

constexpr int kPlanThreads = 1024;

}  // namespace

int64_t expert_plan_workspace(int64_t pairs, int64_t experts) {
  const int64_t groups = cdiv(pairs, kPlanThreads * kPlanRounds);
  return groups > 1 ? groups * experts * (int64_t)sizeof(int) : 0;
}

hipError_t launch_expert_plan(const ExpertPlan& p, hipStream_t stream) {
  return launch_plan<kPlanThreads, kMaxExperts>(p, stream);
}

hipError_t launch_expert_combine(int dtype, const ExpertCombine& p, hipStream_t stream) {
  const dim3 grid((unsigned)cdiv(p.tokens * p.N, 256));
  if (dtype == 1)
    hipLaunchKernelGGL((expert_combine_kernel<1>), grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((expert_combine_kernel<2>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace qgemm
