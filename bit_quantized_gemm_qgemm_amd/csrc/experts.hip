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
// Where several workgroups share the pairs, a launch ahead leaves their counts in the
// workspace, and each workgroup of the second sums those it needs.
//
// The bytes are few (32768 tokens x 8: 4.2 MB, below a microsecond); what it takes are
// trips to memory and barriers one after the other: 2.4 us for 32 tokens x 8 of 128
// experts, and for 32768 x 8 of 256 experts 4.1 of counts and 9.7 of places.

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

// pair (wave * ROUNDS + r) * 64 + lane of the share
template <class S>
__device__ __forceinline__ void load_pairs(PlanState<S>& s, const ExpertPlan& p, int64_t first) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int r = 0; r < S::ROUNDS; ++r) {
    const int64_t i = first + (wave * S::ROUNDS + r) * 64 + lane;
    int64_t id = -1;
    if (i < p.pairs)
      id = p.wide ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
    s.e[r] = id >= 0 && id < p.experts ? (int)id : -1;
  }
}

// counts [wave][experts] in LDS
template <class S>
__device__ __forceinline__ void count_pairs(PlanState<S>& s, const ExpertPlan& p, int* counts) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
  load_pairs<S>(s, p, (int64_t)blockIdx.x * S::kPairs);
  count_pairs<S>(s, p, counts);
  for (int e = threadIdx.x; e < p.experts; e += S::THREADS) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < S::kWaves; ++w) n += counts[w * p.experts + e];
    p.counts[(int64_t)blockIdx.x * p.experts + e] = n;
  }
}

template <class S>
__global__ __launch_bounds__(S::THREADS) void expert_place_kernel(const ExpertPlan p) {
  __shared__ int counts[S::kWaves * S::EXPERTS];
  constexpr int kParts = S::THREADS / S::EXPERTS;   // threads that sum the workgroups' counts of an expert
  __shared__ int earlier[kParts][S::EXPERTS], all[kParts][S::EXPERTS];   // of the workgroups before, of all
  __shared__ int wave_sum[S::kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t first = (int64_t)blockIdx.x * S::kPairs;
  const int groups = gridDim.x;
  PlanState<S> s;
  load_pairs<S>(s, p, first);
  // Plain sums of a thread, eight loads in flight: sums of a wave over its lanes took
  // half of the kernel's time (32768 tokens x 8 of 256 experts: 17.5 -> 13.4 us).
  const int part = tid / S::EXPERTS, mine = tid % S::EXPERTS;
  if (groups > 1 && mine < p.experts) {
    int sum = 0, before = 0;   // of the workgroups from this one on, of those before it
    const int32_t* left = p.counts + mine;
    int b = part;
#pragma unroll 8
    for (; b < (int)blockIdx.x; b += kParts) before += left[(int64_t)b * p.experts];
#pragma unroll 8
    for (; b < groups; b += kParts) sum += left[(int64_t)b * p.experts];
    earlier[part][mine] = before;
    all[part][mine] = before + sum;
  }
  count_pairs<S>(s, p, counts);

  // sums over the experts, THREADS of them at a time
  int before = 0;   // pairs of the experts of the rounds before
  for (int e0 = 0; e0 < p.experts; e0 += S::THREADS) {
    const int e = e0 + tid;
    int n[S::kWaves], total = 0, at = 0;
#pragma unroll
    for (int w = 0; w < S::kWaves; ++w) n[w] = e < p.experts ? counts[w * p.experts + e] : 0;
    if (groups > 1) {
      if (e < p.experts)
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          at += earlier[i][e];
          total += all[i][e];
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
// the wave's and come through the scalar cache.  What bounds it is memory: each row
// is read once, past the caches, and each output written once past them (8192 tokens
// x 8 choices of 4096 elements: 100 us, 6.0 TB/s; through the caches 118.  4096 x 2:
// 18.4, 22.4.  16 x 8: 3.5, the launch and one trip to memory).
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
        v[j] = __builtin_nontemporal_load(reinterpret_cast<const uintx4_any*>(row));
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
    __builtin_nontemporal_store(uintx4_any{d[0], d[1], d[2], d[3]}, reinterpret_cast<uintx4_any*>(out));
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

// Pairs of a workgroup.  One does up to 4096 (512 tokens x 8 of 128 experts 7.2 us; two
// of 2048 with their second launch 8.3; 600 tokens: 8.4, with shares of 4096 11.7).
// Above it shares of 2048 end soonest (2^14 pairs of 256 experts 9.4 us, 12.9 with
// shares of 4096 and 20.2 with 8192; 2^18 13.5, 16.1, 23.4; 2^19 of 128 15.4, 17.1,
// 22.7) until the sums over all the workgroups, in each of them, weigh more (2^20: 29.6,
// 21.4, 25.7; 2^22 of 16: 187, 75, 50).
constexpr int64_t kPlanAlone = 4096, kPlanMany = (int64_t)1 << 19, kPlanMost = (int64_t)1 << 20;
int64_t plan_share(int64_t pairs) {
  return pairs <= kPlanAlone ? 4096 : pairs <= kPlanMany ? 2048 : pairs <= kPlanMost ? 4096 : 8192;
}

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
  if (pairs <= kPlanAlone) return 0;
  // no less than fewer pairs need, so that one sized for the most serves them all
  int64_t groups = cdiv(pairs, plan_share(pairs)), fewer = cdiv(pairs < kPlanMany ? pairs : kPlanMany, 2048);
  if (groups < fewer) groups = fewer;
  return groups * experts * (int64_t)sizeof(int);
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
