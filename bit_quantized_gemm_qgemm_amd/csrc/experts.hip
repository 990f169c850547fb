// Routing around the products grouped by expert: the order of a batch's rows,
// and the sum of each token's expert outputs.
#include "qgemm_common.h"
#include "wave_sums.h"

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
// is the pairs' own.  The counts of the waves, and of the workgroups before, then
// become places.
//
// Where several workgroups share the pairs, a launch ahead leaves each workgroup's counts in the workspace, expert by expert, where a wave
// of the second sums 64 workgroups' at once.
// A workgroup of THREADS takes ROUNDS pairs a thread, of up to EXPERTS experts.
template <int THREADS_, int ROUNDS_, int EXPERTS_>
struct PlanShape {
  static constexpr int THREADS = THREADS_, ROUNDS = ROUNDS_, EXPERTS = EXPERTS_;
  static constexpr int kWaves = THREADS / 64, kPairs = THREADS * ROUNDS;
};

template <class S>
struct PlanState {
  int e[S::ROUNDS];    // expert, or -1
  int at[S::ROUNDS];   // place among the wave's pairs of that expert
};

// counts [wave][experts] in LDS; pair (wave * ROUNDS + r) * 64 + lane of the share
template <class S>
__device__ __forceinline__ void count_pairs(PlanState<S>& s, const ExpertPlan& p, int64_t first,
                                            int* counts) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int r = 0; r < S::ROUNDS; ++r) {
    const int64_t i = first + (wave * S::ROUNDS + r) * 64 + lane;
    int64_t id = -1;
    if (i < p.pairs)
      id = p.wide ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
    s.e[r] = id >= 0 && id < p.experts ? (int)id : -1;
  }
  for (int i = threadIdx.x; i < S::kWaves * p.experts; i += S::THREADS) counts[i] = 0;
  const int bits = 32 - __builtin_clz(p.experts);   // of 0 .. experts
  __syncthreads();
  volatile int* mine = counts + wave * p.experts;
#pragma unroll
  for (int r = 0; r < S::ROUNDS; ++r) {
    const bool some = s.e[r] >= 0;
    uint64_t same = __ballot(some);
    s.at[r] = 0;
    if (same == 0) continue;   // of the whole wave: its share has ended
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

template <class S>
__global__ __launch_bounds__(S::THREADS) void expert_count_kernel(const ExpertPlan p) {
  __shared__ int counts[S::kWaves * S::EXPERTS];
  PlanState<S> s;
  count_pairs<S>(s, p, (int64_t)blockIdx.x * S::kPairs, counts);
  for (int e = threadIdx.x; e < p.experts; e += S::THREADS) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < S::kWaves; ++w) n += counts[w * p.experts + e];
    p.counts[(int64_t)e * gridDim.x + blockIdx.x] = n;
  }
}

template <class S>
__global__ __launch_bounds__(S::THREADS) void expert_place_kernel(const ExpertPlan p) {
  __shared__ int counts[S::kWaves * S::EXPERTS];
  __shared__ int earlier[S::EXPERTS], all[S::EXPERTS];   // pairs of the workgroups before, and of all
  __shared__ int wave_sum[S::kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t first = (int64_t)blockIdx.x * S::kPairs;
  const int groups = gridDim.x;
  if (groups > 1) {
    // experts wave, wave + kWaves, ...: the counts of all of them in flight at once
    constexpr int kEach = S::EXPERTS / S::kWaves;
    for (int b0 = 0; b0 < groups; b0 += 64) {
      const int mine = (int)blockIdx.x - b0;   // workgroups of these 64 before this one
      int n[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int e = wave + j * S::kWaves;
        n[j] = e < p.experts && b0 + lane < groups ? p.counts[(int64_t)e * groups + b0 + lane] : 0;
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int e = wave + j * S::kWaves;
        const int upto = int_sums_of_wave(n[j]);
        const int sum = __builtin_amdgcn_readlane(upto, 63);
        const int before = mine <= 0 ? 0 : mine < 64 ? __builtin_amdgcn_readlane(upto, mine - 1) : sum;
        if (lane == 0 && e < p.experts) {
          earlier[e] = (b0 > 0 ? earlier[e] : 0) + before;
          all[e] = (b0 > 0 ? all[e] : 0) + sum;
        }
      }
    }
  }
  PlanState<S> s;
  count_pairs<S>(s, p, first, counts);

  // sums over the experts, THREADS of them at a time
  int before = 0;   // pairs of the experts of the rounds before
  for (int e0 = 0; e0 < p.experts; e0 += S::THREADS) {
    const int e = e0 + tid;
    int n[S::kWaves], total = 0, at = 0;
#pragma unroll
    for (int w = 0; w < S::kWaves; ++w) n[w] = e < p.experts ? counts[w * p.experts + e] : 0;
    if (groups > 1) {
      if (e < p.experts) {
        at = earlier[e];
        total = all[e];
      }
    } else {
#pragma unroll
      for (int w = 0; w < S::kWaves; ++w) total += n[w];
    }
    const int upto = int_sums_of_wave(total);
    if (lane == 63) wave_sum[wave] = upto;
    __syncthreads();
    int base = before;
#pragma unroll
    for (int w = 0; w < S::kWaves; ++w) {
      if (w < wave) base += wave_sum[w];
      before += wave_sum[w];
    }
    if (e < p.experts) {
      base += upto - total;
      if (blockIdx.x == 0) p.offsets[e] = base;
      at += base;
#pragma unroll
      for (int w = 0; w < S::kWaves; ++w) {
        counts[w * p.experts + e] = at;
        at += n[w];
      }
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.experts] = before;
#pragma unroll
  for (int r = 0; r < S::ROUNDS; ++r) {
    const int64_t i = first + (wave * S::ROUNDS + r) * 64 + lane;
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
__device__ __forceinline__ uint16_t from_float(float v) {   // conversions of the hardware, to nearest even
  if constexpr (DT == 1) return __builtin_bit_cast(uint16_t, (_Float16)v);
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// out[t, n] = sum_j gates[t, j] * y[places[t, j], n] in fp32, in the order of j.  A
// thread forms eight neighbouring elements of a token and has the rows of eight
// choices in flight.  UNIFORM: a row is whole waves, so the places and gates are
// the wave's and come through the scalar cache.
constexpr int kChoices = 8;
typedef uintx4 __attribute__((aligned(2))) uintx4_any;   // 16 bytes at any element

template <int DT, bool UNIFORM>
__global__ __launch_bounds__(256) void expert_combine_kernel(const ExpertCombine p, uint32_t chunks) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  uint32_t t = i / chunks;
  const uint32_t n = 8 * (i - t * chunks);
  if (UNIFORM) t = __builtin_amdgcn_readfirstlane(t);
  if (t >= p.tokens) return;
  const int32_t* places = p.places + (int64_t)t * p.top;
  const float* gates = p.gates + (int64_t)t * p.top;
  const bool whole = n + 8 <= p.N;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  for (int j0 = 0; j0 < p.top; j0 += kChoices) {
    uintx4 v[kChoices];
    float gate[kChoices];
#pragma unroll
    for (int j = 0; j < kChoices; ++j) {
      const int place = j0 + j < p.top ? places[j0 + j] : -1;
      const bool some = (uint32_t)place < p.rows;
      gate[j] = some ? gates[j0 + j] : 0.f;   // and zeros for the row: left out whatever both hold
      v[j] = uintx4{0, 0, 0, 0};
      if (!some) continue;
      const uint16_t* row = p.y + (int64_t)place * p.N + n;
      if (whole) {
        v[j] = *reinterpret_cast<const uintx4_any*>(row);
      } else {
        uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 7; ++e)
          if (n + e < p.N) d[e >> 1] |= (uint32_t)row[e] << (16 * (e & 1));
        v[j] = uintx4{d[0], d[1], d[2], d[3]};
      }
    }
#pragma unroll
    for (int j = 0; j < kChoices; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        sum[e] = __builtin_fmaf(gate[j], to_float<DT>((uint16_t)(v[j][e >> 1] >> (16 * (e & 1)))), sum[e]);
  }
  uint32_t d[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    d[e] = (uint32_t)from_float<DT>(sum[2 * e]) | (uint32_t)from_float<DT>(sum[2 * e + 1]) << 16;
  uint16_t* out = p.out + (int64_t)t * p.N + n;
  if (whole) {
    *reinterpret_cast<uintx4_any*>(out) = uintx4{d[0], d[1], d[2], d[3]};
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (n + e < p.N) out[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
  }
}

template <class S>
hipError_t launch_plan(const ExpertPlan& p, hipStream_t stream) {
  const int64_t groups = cdiv(p.pairs, S::kPairs);
  const dim3 grid((unsigned)(groups > 0 ? groups : 1));
  if (groups > 1)
    hipLaunchKernelGGL((expert_count_kernel<S>), grid, dim3(S::THREADS), 0, stream, p);
  hipLaunchKernelGGL((expert_place_kernel<S>), grid, dim3(S::THREADS), 0, stream, p);
  return hipGetLastError();
}

// Pairs of a workgroup.  One does up to 4096 (512 tokens x 8 of 128 experts 7.3 us;
// two of 2048 with their second launch 11.0, 600 tokens 11.0, 14.2 with shares of
// 4096).  Shares of 2048 end sooner up to 2^18 pairs (16384 pairs 12.4 us, 15.6 with
// 4096 and 23.5 with 8192; 262144 pairs of 256 experts 18.0, 17.5, 25.1), above that
// the second launch's sums over all of them do not (2^22: 593, 176 and 73).
constexpr int64_t kPlanAlone = 4096, kPlanMany = (int64_t)1 << 18;
int64_t plan_share(int64_t pairs) { return pairs <= kPlanAlone ? kPlanAlone : pairs <= kPlanMany ? 2048 : 8192; }

template <int EXPERTS>
hipError_t launch_plan_of(const ExpertPlan& p, hipStream_t stream) {
  switch (plan_share(p.pairs)) {
    case 2048: return launch_plan<PlanShape<1024, 2, EXPERTS>>(p, stream);
    case 4096: return launch_plan<PlanShape<1024, 4, EXPERTS>>(p, stream);
    default: return launch_plan<PlanShape<1024, 8, EXPERTS>>(p, stream);
  }
}

}  // namespace

int64_t expert_plan_workspace(int64_t pairs, int64_t experts) {
  const int64_t groups = cdiv(pairs, plan_share(pairs));
  return groups > 1 ? groups * experts * (int64_t)sizeof(int) : 0;
}

// Few pairs take four waves (32 tokens x 8 of 128 experts: 5.1 -> 2.4 us, with one
// round instead of eight).
hipError_t launch_expert_plan(const ExpertPlan& p, hipStream_t stream) {
  if (p.experts > 256) return launch_plan_of<kMaxExperts>(p, stream);
  if (p.pairs <= 256) return launch_plan<PlanShape<256, 1, 256>>(p, stream);
  if (p.pairs <= 1024) return launch_plan<PlanShape<256, 4, 256>>(p, stream);
  return launch_plan_of<256>(p, stream);
}

hipError_t launch_expert_combine(int dtype, const ExpertCombine& p, hipStream_t stream) {
  const uint32_t chunks = (uint32_t)cdiv(p.N, 8);
  const bool uniform = chunks % 64 == 0;
  auto kernel = dtype == 1 ? (uniform ? expert_combine_kernel<1, true> : expert_combine_kernel<1, false>)
                           : (uniform ? expert_combine_kernel<2, true> : expert_combine_kernel<2, false>);
  hipLaunchKernelGGL(kernel, dim3((unsigned)cdiv((int64_t)p.tokens * chunks, 256)), dim3(256), 0, stream, p, chunks);
  return hipGetLastError();
}

}  // namespace qgemm
