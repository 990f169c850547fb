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
// Where several workgroups share the pairs, a first launch leaves each workgroup's counts
// in the workspace and each pair's place among its workgroup's pairs of its expert in
// `places`; in the second each workgroup sums the counts that it needs.
//
// The bytes are few (32768 tokens x 8: 4.2 MB, below a microsecond); what it takes are
// trips to memory and barriers one after the other: 2.4 us for 32 tokens x 8 of 128
// experts, 5.5 for 512 x 8, and for 32768 x 8 of 256 3.8 of counts and 6.2 of places.
template <int THREADS_, int ROUNDS_, int EXPERTS_>
struct PlanShape {
  static constexpr int THREADS = THREADS_, ROUNDS = ROUNDS_, EXPERTS = EXPERTS_;
  static constexpr int kWaves = THREADS / 64;
  static constexpr int64_t kPairs = THREADS * ROUNDS;
  static_assert(THREADS >= EXPERTS, "a thread for each expert");
};

template <class S>
struct PlanState {
  int e[S::ROUNDS];    // expert, or -1
  int at[S::ROUNDS];   // place among the wave's pairs of that expert
};

// Expert of pair i, or -1.
__device__ __forceinline__ int expert_of(const ExpertPlan& p, int64_t i) {
  const int64_t id = p.wide ? static_cast<const int64_t*>(p.ids)[i] : static_cast<const int32_t*>(p.ids)[i];
  return id >= 0 && id < p.experts ? (int)id : -1;
}

// pair (wave * ROUNDS + r) * 64 + lane of the share
template <class S>
__device__ __forceinline__ void load_pairs(PlanState<S>& s, const ExpertPlan& p, int64_t first) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int r = 0; r < S::ROUNDS; ++r) {
    const int64_t i = first + (wave * S::ROUNDS + r) * 64 + lane;
    s.e[r] = i < p.pairs ? expert_of(p, i) : -1;
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

// Of the expert `threadIdx.x`, which has `total` pairs (0 past the last): the pairs of the
// experts before, and of all in `sum`.
template <class S>
__device__ __forceinline__ int pairs_before(int total, int& sum) {
  __shared__ int wave_sum[S::kWaves];
  const int wave = threadIdx.x >> 6, upto = int_sums_of_wave(total);
  if ((threadIdx.x & 63) == 63) wave_sum[wave] = upto;
  __syncthreads();
  int before = upto - total;
  sum = 0;
#pragma unroll
  for (int w = 0; w < S::EXPERTS / 64; ++w) {
    if (w < wave) before += wave_sum[w];
    sum += wave_sum[w];
  }
  return before;
}

// The waves' counts of one expert become the places where each begins.
template <class S>
struct WaveCounts {
  int n[S::kWaves], sum = 0;
  __device__ __forceinline__ WaveCounts(const int* counts, int experts, int e) {
#pragma unroll
    for (int w = 0; w < S::kWaves; ++w) n[w] = counts[w * experts + e];
#pragma unroll
    for (int w = 0; w < S::kWaves; ++w) sum += n[w];
  }
  __device__ __forceinline__ void begin(int* counts, int experts, int e, int at) const {
#pragma unroll
    for (int w = 0; w < S::kWaves; ++w) {
      counts[w * experts + e] = at;
      at += n[w];
    }
  }
};

// One pair's outputs, `total` pairs having rows.  (Calls that share a workspace at the
// same time spoil each other's places, but write nothing outside the arrays.)
__device__ __forceinline__ void place_pair(const ExpertPlan& p, int64_t i, int place, int total) {
  if ((uint32_t)place < (uint32_t)p.pairs) p.rows[place] = (int32_t)((uint32_t)i / (uint32_t)p.top);
  p.places[i] = place;
  if (i >= total) p.rows[i] = -1;   // past the last row
}

// All pairs in one workgroup.
template <class S>
__global__ __launch_bounds__(S::THREADS) void expert_plan_kernel(const ExpertPlan p) {
  __shared__ int counts[S::kWaves * S::EXPERTS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  PlanState<S> s;
  load_pairs<S>(s, p, 0);
  count_pairs<S>(s, p, counts);
  const bool some = tid < p.experts;
  const WaveCounts<S> n(counts, p.experts, some ? tid : 0);
  int sum;
  const int before = pairs_before<S>(some ? n.sum : 0, sum);
  if (some) {
    p.offsets[tid] = before;
    n.begin(counts, p.experts, tid, before);
  }
  if (tid == 0) p.offsets[p.experts] = sum;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < S::ROUNDS; ++r) {
    const int64_t i = (wave * S::ROUNDS + r) * 64 + lane;
    if (i >= p.pairs) break;
    place_pair(p, i, s.e[r] < 0 ? -1 : counts[wave * p.experts + s.e[r]] + s.at[r], sum);
  }
}

template <class S>
__global__ __launch_bounds__(S::THREADS) void expert_count_kernel(const ExpertPlan p) {
  __shared__ int counts[S::kWaves * S::EXPERTS];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t first = (int64_t)blockIdx.x * S::kPairs;
  PlanState<S> s;
  load_pairs<S>(s, p, first);
  count_pairs<S>(s, p, counts);
  if (tid < p.experts) {
    const WaveCounts<S> n(counts, p.experts, tid);
    n.begin(counts, p.experts, tid, 0);
    p.counts[(int64_t)blockIdx.x * p.experts + tid] = n.sum;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < S::ROUNDS; ++r) {
    const int64_t i = first + (wave * S::ROUNDS + r) * 64 + lane;
    if (i >= p.pairs) break;
    p.places[i] = s.e[r] < 0 ? -1 : counts[wave * p.experts + s.e[r]] + s.at[r];
  }
}

template <class S>
__global__ __launch_bounds__(S::THREADS) void expert_place_kernel(const ExpertPlan p) {
  constexpr int kParts = S::THREADS / S::EXPERTS;   // threads that sum the workgroups' counts of an expert
  __shared__ int earlier[kParts][S::EXPERTS], all[kParts][S::EXPERTS];   // of the workgroups before, of all
  __shared__ int start[S::EXPERTS];
  const int tid = threadIdx.x;
  const int64_t first = (int64_t)blockIdx.x * S::kPairs;
  int e[S::ROUNDS], at[S::ROUNDS];
#pragma unroll
  for (int r = 0; r < S::ROUNDS; ++r) {
    const int64_t i = first + r * S::THREADS + tid;
    e[r] = i < p.pairs ? expert_of(p, i) : -1;
    at[r] = i < p.pairs ? p.places[i] : 0;
  }
  // Plain sums of a thread, 16 loads in flight, then 4 (sums of a wave over its lanes
  // took half of the kernel's time).
  const int part = tid / S::EXPERTS, mine = tid % S::EXPERTS, groups = gridDim.x;
  if (mine < p.experts) {
    int sum = 0, before = 0, b = part;
    const int32_t* left = p.counts + mine;
    auto add = [&](int b) {
      const int n = left[(int64_t)b * p.experts];
      sum += n;
      before += b < (int)blockIdx.x ? n : 0;
    };
    for (; b + 15 * kParts < groups; b += 16 * kParts)
#pragma unroll
      for (int j = 0; j < 16; ++j) add(b + j * kParts);
    for (; b + 3 * kParts < groups; b += 4 * kParts)
#pragma unroll
      for (int j = 0; j < 4; ++j) add(b + j * kParts);
    for (; b < groups; b += kParts) add(b);
    earlier[part][mine] = before;
    all[part][mine] = sum;
  }
  __syncthreads();
  int total = 0, sum;
  if (tid < p.experts)
#pragma unroll
    for (int i = 0; i < kParts; ++i) total += all[i][tid];
  int before = pairs_before<S>(total, sum);
  if (tid < p.experts) {
    if (blockIdx.x == 0) p.offsets[tid] = before;
#pragma unroll
    for (int i = 0; i < kParts; ++i) before += earlier[i][tid];
    start[tid] = before;
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.experts] = sum;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < S::ROUNDS; ++r) {
    const int64_t i = first + r * S::THREADS + tid;
    if (i >= p.pairs) break;
    place_pair(p, i, e[r] < 0 ? -1 : start[e[r]] + at[r], sum);
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
  const dim3 grid((unsigned)cdiv(p.pairs, S::kPairs)), block(S::THREADS);
  if (grid.x <= 1) {
    hipLaunchKernelGGL((expert_plan_kernel<S>), dim3(1), block, 0, stream, p);
  } else {
    hipLaunchKernelGGL((expert_count_kernel<S>), grid, block, 0, stream, p);
    hipLaunchKernelGGL((expert_place_kernel<S>), grid, block, 0, stream, p);
  }
  return hipGetLastError();
}

// Pairs of a workgroup.  One does up to 2048 (256 tokens x 8 of 128 experts 4.6 us, in
// two of 1024 with their second launch 5.4).  Above it small shares end soonest until
// the sums over all the workgroups, in each of them, weigh more.  us with shares of
// 1024 / 2048 / 4096 / 8192: 2^14 pairs of 256 experts 6.4 / 7.9 / 10.5 / 16.1, 2^16 of
// 64 6.2 / 9.0 / 10.4 / 14.7, 2^18 of 256 11.5 / 11.2 / 13.5 / 21.0, 2^19 of 128 20.4 /
// 13.4 / 14.7 / 21.7, 2^20 of 128 48 / 25.1 / 18.8 / 26.1, 2^21 146 / 58 / 35.7 / 38.4,
// 2^22 of 256 665 / 205 / 88 / 68.
constexpr int64_t kPlanAlone = 2048, kPlanFew = (int64_t)1 << 17, kPlanMany = (int64_t)1 << 19,
                  kPlanMost = (int64_t)1 << 21;
int64_t plan_share(int64_t pairs) {
  return pairs <= kPlanAlone ? 2048 : pairs <= kPlanFew ? 1024 : pairs <= kPlanMany ? 2048
                                   : pairs <= kPlanMost ? 4096 : 8192;
}

template <int EXPERTS>
hipError_t launch_plan_of(const ExpertPlan& p, hipStream_t stream) {
  switch (plan_share(p.pairs)) {
    case 1024: return launch_plan<PlanShape<1024, 1, EXPERTS>>(p, stream);
    case 2048: return launch_plan<PlanShape<1024, 2, EXPERTS>>(p, stream);
    case 4096: return launch_plan<PlanShape<1024, 4, EXPERTS>>(p, stream);
    default: return launch_plan<PlanShape<1024, 8, EXPERTS>>(p, stream);
  }
}

}  // namespace

int64_t expert_plan_workspace(int64_t pairs, int64_t experts) {
  if (pairs <= kPlanAlone) return 0;
  // no less than fewer pairs need, so that one sized for the most serves them all
  int64_t groups = 0;
  for (const int64_t most : {kPlanFew, kPlanMany, kPlanMost, pairs}) {
    const int64_t n = most < pairs ? most : pairs, g = cdiv(n, plan_share(n));
    if (g > groups) groups = g;
  }
  return groups * experts * (int64_t)sizeof(int);
}

// Few pairs take four waves (32 tokens x 8 of 128 experts 2.4 us, with 16 waves 2.8), up
// to 1024 one round of 16 waves (128 x 8 of 256 experts 3.5, four rounds of four 4.8).
hipError_t launch_expert_plan(const ExpertPlan& p, hipStream_t stream) {
  if (p.experts > 256) return launch_plan_of<kMaxExperts>(p, stream);
  if (p.pairs <= 256) return launch_plan<PlanShape<256, 1, 256>>(p, stream);
  if (p.pairs <= 1024) return launch_plan<PlanShape<1024, 1, 256>>(p, stream);
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
