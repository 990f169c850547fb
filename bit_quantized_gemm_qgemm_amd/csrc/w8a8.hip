// Products of 8-bit integers with scales for each token and channel, for one
// weight or for rows grouped by expert, plain or gated.
//
//   Y[m, n] = (sum_k A[m, k] W[k, n]) * a_scale[m] * w_scale[n]
//   gated, N = 2F:  H[m, f] = silu(Y[m, f]) * Y[m, F + f],  silu(y) = y / (1 + exp(-y))
//
// The sum is exact in 32 bits (|A W| <= 2^14 and K < 2^17); it becomes fp32 with
// one rounding, the scales multiply it in fp32, and the result is rounded once to
// the output type.
#include <cmath>
#include <type_traits>

#include "qgemm_common.h"
#include "tile_common.h"
#include "wave_sums.h"

namespace qgemm {
namespace {

// Launch arguments of the kernels.
struct Args {
  const uint8_t* a;
  const float* a_scale;
  const uint8_t* w;
  const float* w_scale;
  const int32_t *offsets, *rows;
  uint16_t* out;
  uint32_t a_bytes;
  int a_rows, M, N, K;    // N: columns of the weight
  int out_n;              // columns of the output
  int experts, CG, KT;
  int64_t w_bytes;        // of one expert
  int col_blocks;         // of the kernel's own width
  bool gated, bf16;
};

int64_t col_blocks(const W8a8& p, int64_t cols) {
  return cdiv(w8a8_geom(p.K, p.N, p.gated).cg * kTileN, cols);
}

Args args_of(const W8a8& p, int64_t cols) {
  const W8a8Geom geom = w8a8_geom(p.K, p.N, p.gated);
  Args g;
  g.a = reinterpret_cast<const uint8_t*>(p.a);
  g.a_scale = p.a_scale;
  g.w = p.w;
  g.w_scale = p.w_scale;
  g.offsets = p.offsets;
  g.rows = p.rows;
  g.out = p.out;
  g.a_bytes = (uint32_t)(p.a_rows * p.K);
  g.a_rows = (int)p.a_rows;
  g.M = (int)p.M;
  g.N = (int)p.N;
  g.K = (int)p.K;
  g.out_n = (int)(p.gated ? p.N / 2 : p.N);
  g.experts = (int)p.experts;
  g.CG = (int)geom.cg;
  g.KT = (int)geom.kt;
  g.w_bytes = geom.bytes;
  g.col_blocks = (int)col_blocks(p, cols);
  g.gated = p.gated;
  g.bf16 = p.bf16;
  return g;
}

// Row blocks that a launch has at most: an expert's last block may be part full.
int64_t most_row_blocks(const W8a8& p, int64_t rows) {
  if (!p.offsets) return cdiv(p.M, rows);
  return (p.M < p.experts ? p.M : p.experts) + p.M / rows;
}

// Workgroups of a launch: the items, an eighth of them for each XCD.
int64_t workgroups(const W8a8& p, int64_t rows, int64_t cols) {
  return cdiv(most_row_blocks(p, rows) * col_blocks(p, cols), 8) * 8;
}

// What a workgroup computes: rows m0 .. m0 + BM - 1 (those below hi) and one
// block of columns of expert e.
struct Item {
  int e, m0, hi, cb;
  bool some;
};

// First and last row of expert e, whatever the offsets hold.
__device__ __forceinline__ int2 rows_of(const Args& g, int e) {
  const int lo = min(max(g.offsets[e], 0), g.M);
  return make_int2(lo, min(max(g.offsets[e + 1], lo), g.M));
}

// The workgroups' items lie in one row: expert after expert, of each groups of
// GROUP row blocks, of a group its column blocks in turn, and of a column block the
// row blocks.  Workgroups are handed to the 8 XCDs round-robin; each XCD takes an
// eighth of the row, so that the row blocks that share a weight tile meet in one L2.
// The experts' places in the row follow from their row counts: a wave counts the
// blocks of all experts, each lane those of `per` neighbours.  Offsets that do not
// fall leave at most as many blocks as the launch has; of any others there are no
// items.
template <int BM, int GROUP>
__device__ __forceinline__ Item item_of(const Args& g) {
  Item it{0, 0, g.M, 0, true};
  int blocks = (g.M + BM - 1) / BM, before = 0, total = blocks;
  const int lane = threadIdx.x & 63;
  const int per = (g.experts + 63) / 64;
  int2 r = make_int2(0, 0);
  int mine = 0, upto = 0;
  auto blocks_of = [](int2 r) { return (r.y - r.x + BM - 1) / BM; };
  if (g.offsets) {
    bool falls = false;
    for (int j = 0; j < per; ++j) {
      const int e = lane * per + j;
      if (e < g.experts) {
        r = rows_of(g, e);
        mine += blocks_of(r);
        falls |= g.offsets[e + 1] < g.offsets[e];
      }
    }
    upto = int_sums_of_wave(mine);
    total = __ballot(falls) == 0 ? __builtin_amdgcn_readlane(upto, 63) : 0;
  }
  const int items = total * g.col_blocks, share = (items + 7) / 8;
  const int slot = blockIdx.x >> 3, i = (int)(blockIdx.x & 7) * share + slot;
  if (slot >= share || i >= items) {
    it.some = false;
    return it;
  }
  if (g.offsets) {
    const int q = i / g.col_blocks;   // lies among the blocks of its expert
    int at = __builtin_ctzll(__ballot(upto > q));
    before = __builtin_amdgcn_readlane(upto - mine, at);
    it.e = at * per;
    if (per > 1) {   // the lanes take the neighbours one by one
      r = make_int2(0, 0);
      if (lane < per && it.e + lane < g.experts) r = rows_of(g, it.e + lane);
      mine = blocks_of(r);
      upto = int_sums_of_wave(mine);
      at = __builtin_ctzll(__ballot(before + upto > q));
      before += __builtin_amdgcn_readlane(upto - mine, at);
      it.e += at;
    }
    it.m0 = __builtin_amdgcn_readlane(r.x, at);
    it.hi = __builtin_amdgcn_readlane(r.y, at);
    blocks = (it.hi - it.m0 + BM - 1) / BM;
  }
  // GROUP row blocks at a time: they cross all columns before the next ones
  const int rem = __builtin_amdgcn_readfirstlane(i - before * g.col_blocks);
  const int group = rem / (GROUP * g.col_blocks), in_group = rem - group * (GROUP * g.col_blocks);
  const int rows = min(blocks - group * GROUP, GROUP);
  it.cb = in_group / rows;
  it.m0 += (group * GROUP + in_group - it.cb * rows) * BM;
  return it;
}

// Column of the output, and of the weight's scales, of packed column c.
__device__ __forceinline__ int scale_column(const Args& g, int c) {
  if (!g.gated) return c;
  const int f = (c >> 5) * 16 + (c & 15);
  return f < g.out_n ? ((c >> 4) & 1) * g.out_n + f : g.N;   // N: none
}

// silu(gate) * up.  The exponential and the reciprocal are the hardware's, each
// within one step of fp32; a gate below -87.3 gives 0.
__device__ __forceinline__ float gated_value(float gate, float up) {
  const float e = __builtin_amdgcn_exp2f(gate * -1.44269504089f);
  return gate * __builtin_amdgcn_rcpf(1.0f + e) * up;
}

__device__ __forceinline__ uint16_t rounded(float v, bool bf16) {
  return bf16 ? f32_to_bf16_rne(v) : f32_to_f16_bits(v);
}

// ---- up to 16 rows ----------------------------------------------------------
// A workgroup owns 16 rows and G column groups of 16; its NW waves share the K
// tiles.  Weight tiles go from memory straight into registers, two of a wave in
// flight, and meet the rows' codes in 16 x 16 x 64 matrix instructions; the waves'
// sums meet in LDS.  The weight's bytes bound it: 64 experts of 4096 x 2048, of which
// 16 tokens x 8 reach 53, take 67 us (446 MB: 6.7 TB/s, a plain read 7.07), one row by
// 4096 x 11008 9.1 to 9.6 (45 MB, of which 3 us are the launch and the way in and out).
template <int G>
struct SlabTile {
  uintx4 x[2], w[G][2];
};

template <int G, int NW>
__global__ __launch_bounds__(NW * kWave) void w8a8_slab_kernel(const Args g) {
  constexpr int D = 2;   // K tiles of a wave in flight
  __shared__ intx4 red[NW][G][kWave];
  __shared__ float a_scale[16], w_scale[16 * G];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Item it = item_of<16, 64>(g);
  if (!it.some) return;   // the whole workgroup
  const int cg0 = it.cb * G;

  const int64_t w0 = (int64_t)cg0 * g.KT * kTileBytes;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.a, g.a_bytes);
  const __amdgpu_buffer_rsrc_t wr =
      make_rsrc(g.w + it.e * g.w_bytes + w0, (uint32_t)(g.w_bytes - w0));
  const int last = g.CG - 1 - cg0;
  const uint32_t stride = (uint32_t)g.KT * kTileBytes;
  auto load_w = [&](SlabTile<G>& t, int kt) {
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        t.w[j][h] = __builtin_amdgcn_raw_buffer_load_b128(
            wr, 16u * lane + 1024u * h, (uint32_t)min(j, last) * stride + (uint32_t)kTileBytes * kt, 2);
  };
  // the weight does not wait for the row numbers
  // (without K tiles: tile 0 of a buffer of 0 bytes, so nothing is read.  Tile -1 would be
  // an offset of 4 GB - 2 KB in a scalar register, and the hardware compares a lane's offset
  // with the buffer's size less the scalar one.)
  const int last_kt = max(g.KT - 1, 0);
  SlabTile<G> ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load_w(ring[d], min(wave + d * NW, last_kt));

  uint32_t xoff = kOutOfRange;
  float as = 0.f, ws = 0.f;
  {
    const int m = it.m0 + (lane & 15);
    int row = -1;
    if (m < it.hi) row = g.rows ? g.rows[m] : m;
    if ((uint32_t)row < (uint32_t)g.a_rows) {
      xoff = (uint32_t)row * (uint32_t)g.K + 32u * (lane >> 4);
      as = g.a_scale[row];
    }
    const int c = scale_column(g, cg0 * 16 + lane);   // lanes below 16 G
    if (c < g.N) ws = g.w_scale[(int64_t)it.e * g.N + c];
  }
  // (codes past K in the last tile are the next row's: they meet zeros of W)
  auto load_x = [&](SlabTile<G>& t, int kt) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      t.x[h] = __builtin_amdgcn_raw_buffer_load_b128(xr, xoff + 128u * kt + 16u * h, 0, 0);
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load_x(ring[d], min(wave + d * NW, last_kt));
  auto load = [&](SlabTile<G>& t, int kt) {
    load_x(t, kt);
    load_w(t, kt);
  };

  intx4 acc[G];
#pragma unroll
  for (int j = 0; j < G; ++j) acc[j] = intx4{0, 0, 0, 0};
  auto multiply = [&](const SlabTile<G>& t) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < G; ++j)
        acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(intx4, t.x[h]),
                                                       __builtin_bit_cast(intx4, t.w[j][h]), acc[j],
                                                       0, 0, 0);
  };

  // no branch around a load while whole rounds last: where its paths merge, the
  // compiler waits for every load in flight
  int base = wave;
  for (; base + (2 * D - 1) * NW < g.KT; base += D * NW) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      multiply(ring[d]);
      load(ring[d], base + (d + D) * NW);
    }
  }
  for (; base < g.KT; base += D * NW) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int kt = base + d * NW;
      if (kt < g.KT) {
        multiply(ring[d]);
        if (kt + D * NW < g.KT) load(ring[d], kt + D * NW);
      }
    }
  }

  if (threadIdx.x < 16) a_scale[threadIdx.x] = as;
  if (threadIdx.x < 16 * G) w_scale[threadIdx.x] = ws;
#pragma unroll
  for (int j = 0; j < G; ++j) red[wave][j][lane] = acc[j];
  __syncthreads();
  // lane l of a group holds rows 4 (l >> 4) + [0, 4) of column l & 15
  const int* sums = reinterpret_cast<const int*>(red);
  auto value = [&](int m, int j, int c) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += sums[((w * G + j) * kWave + 16 * (m >> 2) + c) * 4 + (m & 3)];
    return (float)sum * a_scale[m] * w_scale[16 * j + c];
  };
  if (!g.gated) {
    for (int o = threadIdx.x; o < 256 * G; o += NW * kWave) {
      const int m = o / (16 * G), c = o - m * (16 * G);
      const int gm = it.m0 + m, gn = cg0 * 16 + c;
      if (gm < it.hi && gn < g.N)
        g.out[(int64_t)gm * g.out_n + gn] = rounded(value(m, c >> 4, c & 15), g.bf16);
    }
  } else if constexpr (G % 2 == 0) {
    for (int o = threadIdx.x; o < 128 * G; o += NW * kWave) {
      const int m = o / (8 * G), c = o - m * (8 * G), j = 2 * (c >> 4);
      const int gm = it.m0 + m, gn = cg0 * 8 + c;
      if (gm < it.hi && gn < g.out_n)
        g.out[(int64_t)gm * g.out_n + gn] = rounded(
            gated_value(value(m, j, c & 15), value(m, j + 1, c & 15)), g.bf16);
    }
  }
}

template <int G, int NW>
hipError_t launch_slab(const W8a8& p, hipStream_t stream) {
  const Args g = args_of(p, 16 * G);
  hipLaunchKernelGGL((w8a8_slab_kernel<G, NW>), dim3((unsigned)workgroups(p, 16, 16 * G)),
                     dim3(NW * kWave), 0, stream, g);
  return hipGetLastError();
}

// ---- more rows --------------------------------------------------------------
// A workgroup of WR x WC x KS waves owns BM = 32 FM WR rows and BN = 32 FN WC
// columns.  A wave owns FM x FN fragments of 32 x 32 and, where KS > 1, the K tiles
// kq, kq + KS, ...; the waves of kq = 0 add up the sums at the end.  A wave's
// weight fragments go from memory straight into registers (the packed tiles are in
// lane order), WB - 1 steps ahead; the rows' codes pass through a ring of four LDS
// stages, copied three steps ahead.  A step is one K tile of 128 for each of the
// KS: 4 slices of 32, each FM FN matrix instructions of 32 x 32 x 32 a wave.  The
// weight is the first operand, so the accumulators hold the output transposed: lane
// l has row l & 31 of a fragment and, for each e >> 2, four columns 8 (e >> 2) +
// 4 (l >> 5) + [0, 4).  Of a gated weight a fragment is 16 columns of the gate and
// the 16 of the up value that they meet, so elements e and e + 8 of one lane form
// an output.
//
// Per slice u, between the matrix instructions: the LDS reads of the next slice's
// codes, the weight fragments of slice u of step s + WB - 1, and a share of the
// copies of step s + 3; after slice 2 the wait for the copies of step s + 1.
//
// What bounds the largest tiles is power: 8192 x 8192 x 8192 takes 422 us (2.6 POP/s)
// with the matrix pipe busy 72 % of it at 1.65 GHz, where these instructions alone, on
// codes of all sizes, run at 3.3 POP/s and 1.54 GHz (on zeros at 4.7).  What bounds
// the middle ones is the way from the L2 to the CUs, 17 TB/s in all, and below some
// ten steps the way in and out: 300 rows by 4096 x 11008, gated, 19 us with the weight
// in the Infinity Cache, 28.7 from memory.  The weight does not pass through LDS:
// each fragment is read by one wave, or by two, that its CU's cache partly serves.
template <int FM_, int FN_, int WR_, int WC_, int KS_, int WB_>
struct Tile {
  static constexpr int FM = FM_, FN = FN_, WR = WR_, WC = WC_, KS = KS_, WB = WB_;
  static constexpr int NS = 4;   // stages of the ring
  static constexpr int kWaves = WR * WC * KS, kThreads = 64 * kWaves;
  static constexpr int kRows = 32 * FM * WR, kCols = 32 * FN * WC;
  static constexpr int kTileBytes = kRows * 128;          // the rows' codes of one K tile
  static constexpr int kStage = KS * kTileBytes;
  static constexpr int kCopies = 4 * FM / WC;             // of a wave and step, 8 rows each
  static_assert(4 * FM % WC == 0, "whole copies for each wave");
  static constexpr int kPartials = (KS - 1) * WR * WC * FM * FN * 4096;
  static constexpr int kOut = kRows * kCols * 2;
  static constexpr int kMost = kPartials > kOut ? kPartials : kOut;
  static constexpr int kLds = NS * kStage > kMost ? NS * kStage : kMost;
  static constexpr int kScales = (kCols + kRows + kThreads - 1) / kThreads;   // of a thread
  static constexpr int copies_before(int u) { return u * kCopies / 4; }
  // memory instructions issued after the copies of step s + 1 when the wait after
  // slice 2 of step s runs: all of step s - 1 and slices 0 .. 2 of step s
  static constexpr int kCopyWait = (NS - 3) * (4 * FN + kCopies) + 3 * FN + copies_before(3);
  // the same after the loop, where with WB > 2 no fragments are loaded
  static constexpr int kLastWait = WB == 2 ? kCopyWait : (NS - 3) * kCopies + copies_before(3);
  static constexpr int kUnroll = WB > NS ? WB : NS;
  static_assert(kUnroll % WB == 0 && kUnroll % NS == 0, "stages and fragments at fixed places");
  // row blocks that a walk over the columns keeps together
  static constexpr int kGroup = kRows < 1024 ? 1024 / kRows : 1;
};

struct TilePlan {
  const uint8_t *a, *w;
  uint32_t a_n, w_n;      // bytes from them on
  int rd;                 // LDS: chunk l >> 5 of the lane's row (slice u: XOR 32 u)
  uint32_t wo[4];         // fragment f of K tile 0 (tile kt: + 2048 kt; slice u: + 256 u)
  int kq, KT, lds_copy, lds_read;
};

__device__ __forceinline__ int row_swizzle(int r) { return (r >> 1) & 7; }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_at(const uint8_t* p, uint32_t n, uint32_t off) {
  return make_rsrc(p + off, __builtin_amdgcn_readfirstlane(n > off ? n - off : 0u));
}

typedef int intx16 __attribute__((ext_vector_type(16)));

template <int FM>
__device__ __forceinline__ void tile_read(uintx4 (&x)[FM], const uint8_t* st, const TilePlan& P, int u) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
    x[i] = *reinterpret_cast<const uintx4*>(st + (P.rd ^ (32 * u)) + i * 4096);
}

template <class T>
__device__ __forceinline__ void tile_load_w(uintx4 (&w)[4][T::FN], int s, int u, const TilePlan& P) {
  const int kt = T::KS * s + P.kq;
  const __amdgpu_buffer_rsrc_t r = rsrc_at(P.w, kt < P.KT ? P.w_n : 0u, (uint32_t)kt * 2048u);
#pragma unroll
  for (int f = 0; f < T::FN; ++f)
    w[u][f] = __builtin_amdgcn_raw_buffer_load_b128(r, P.wo[f] + 256u * u, 0, 0);
}

// Slice u's share of this wave's copies of step s.  (Codes past K are the next
// row's and meet zeros of the weight; of a K tile past the last nothing is read, of
// the weight neither.)
template <class T>
__device__ __forceinline__ void tile_copy(uint8_t* stage, int s, int u,
                                          const uint32_t (&from)[T::kCopies], const TilePlan& P) {
  const int kt = T::KS * s + P.kq;
  const __amdgpu_buffer_rsrc_t r = rsrc_at(P.a, kt < P.KT ? P.a_n : 0u, (uint32_t)kt * 128u);
#pragma unroll
  for (int i = T::copies_before(u); i < T::copies_before(u + 1); ++i)
    dma16(r, stage + P.lds_copy + i * 1024, from[i]);
}

template <class T>
__device__ __forceinline__ void tile_multiply(const uintx4 (&x)[T::FM], const uintx4 (&w)[T::FN],
                                              intx16 (&acc)[T::FM][T::FN]) {
#pragma unroll
  for (int f = 0; f < T::FN; ++f)
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
      acc[i][f] = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(intx4, w[f]),
                                                        __builtin_bit_cast(intx4, x[i]), acc[i][f], 0,
                                                        0, 0);
}

// The slice's matrix instructions, the first ones each followed by LDS reads and
// by one of the N memory instructions.
template <class T, int N>
__device__ __forceinline__ void tile_order() {
  constexpr int kMul = T::FM * T::FN;
  constexpr int kReads = (2 * T::FM + kMul - 1) / kMul;   // at each of the first half
#pragma unroll
  for (int i = 0; i < kMul; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (i * kReads < T::FM) __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
    if (i < N) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
  }
}

// Step s in stage S = s % 4; w[S % WB] holds its fragments, x[0] slice 0's codes.
// LAST: one of the steps after the loop.  With WB > 2 their fragments are all
// there and they load none (loads that nothing uses would be left out by the
// compiler, and the count of the wait would be wrong).
template <class T, int S, bool LAST>
__device__ __forceinline__ void tile_step(int s, uint8_t* lds, uintx4 (&w)[T::WB][4][T::FN],
                                          uintx4 (&x)[2][T::FM], const uint32_t (&from)[T::kCopies],
                                          const TilePlan& P, intx16 (&acc)[T::FM][T::FN]) {
  constexpr int B = S % T::WB, BN = (S + T::WB - 1) % T::WB;
  constexpr bool kLoads = !LAST || T::WB == 2;
  const uint8_t* st = lds + S % T::NS * T::kStage + P.lds_read;
  const uint8_t* next = lds + (S + 1) % T::NS * T::kStage + P.lds_read;
  uint8_t* to = lds + (S + T::NS - 1) % T::NS * T::kStage;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (u < 3)
      tile_read<T::FM>(x[(u + 1) & 1], st, P, u + 1);
    else
      tile_read<T::FM>(x[0], next, P, 0);
    tile_multiply<T>(x[u & 1], w[B][u], acc);
    if constexpr (kLoads) tile_load_w<T>(w[BN], s + T::WB - 1, u, P);
    tile_copy<T>(to, s + T::NS - 1, u, from, P);
    tile_order<T, (kLoads ? T::FN : 0) + (T::kCopies + 3) / 4>();
    if (u == 2) {
      QG_WAIT_VM_LGKM_BARRIER((LAST ? T::kLastWait : T::kCopyWait));
    } else {
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

template <class T, int S>
__device__ __forceinline__ void tile_steps(int s, uint8_t* lds, uintx4 (&w)[T::WB][4][T::FN],
                                           uintx4 (&x)[2][T::FM], const uint32_t (&from)[T::kCopies],
                                           const TilePlan& P, intx16 (&acc)[T::FM][T::FN]) {
  tile_step<T, S, false>(s + S, lds, w, x, from, P, acc);
  if constexpr (S + 1 < T::kUnroll) tile_steps<T, S + 1>(s, lds, w, x, from, P, acc);
}

template <class T, int S>
__device__ __forceinline__ void tile_last_steps(int s, int steps, uint8_t* lds,
                                                uintx4 (&w)[T::WB][4][T::FN], uintx4 (&x)[2][T::FM],
                                                const uint32_t (&from)[T::kCopies], const TilePlan& P,
                                                intx16 (&acc)[T::FM][T::FN]) {
  if (s + S >= steps) return;
  tile_step<T, S, true>(s + S, lds, w, x, from, P, acc);
  if constexpr (S + 2 < T::kUnroll) tile_last_steps<T, S + 1>(s, steps, lds, w, x, from, P, acc);
}

typedef uintx4 __attribute__((aligned(2))) uintx4_any;   // 16 bytes at any element

template <bool BF16>
__device__ __forceinline__ uint32_t rounded_pair(float lo, float hi) {
  typedef float float2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  if constexpr (BF16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t{lo, hi}), bf16x2_t));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t{lo, hi}), half2_t));
}

template <class T>
__global__ __launch_bounds__(T::kThreads, T::kThreads > 256 ? 1 : 2) void w8a8_tile_kernel(const Args g) {
  constexpr int FM = T::FM, FN = T::FN, WR = T::WR, WC = T::WC, KS = T::KS, WB = T::WB;
  // One array: with more than one the compiler tells them apart, takes the copies
  // into LDS for writes to any of them and waits for all memory before each read.
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::kLds + 4 * (T::kRows + T::kCols)];
  float* const w_scale = reinterpret_cast<float*>(smem + T::kLds);
  float* const a_scale = w_scale + T::kCols;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Item it = item_of<T::kRows, T::kGroup>(g);
  if (!it.some) return;   // the whole workgroup
  const int cg0 = it.cb * (T::kCols / 16);
  const int cw = wave % WC, wr = wave / WC % WR;   // which of the columns and rows

  TilePlan P;
  P.a = g.a;
  P.a_n = g.a_bytes;
  P.w = g.w + it.e * g.w_bytes;
  P.w_n = (uint32_t)g.w_bytes;
  P.kq = wave / (WR * WC);
  P.KT = g.KT;
  P.lds_copy = P.kq * T::kTileBytes + wave % (WR * WC) * T::kCopies * 1024;
  P.lds_read = P.kq * T::kTileBytes + wr * FM * 4096;
  P.rd = (lane & 31) * 128 + 16 * ((lane >> 5) ^ row_swizzle(lane & 31));
#pragma unroll
  for (int f = 0; f < FN; ++f)
    P.wo[f] = (uint32_t)(cg0 + 2 * (FN * cw + f) + ((lane >> 4) & 1)) * (uint32_t)g.KT * 2048u +
              1024u * (lane >> 5) + 16u * (lane & 15);

  // row that output row m reads, or -1
  auto source = [&](int m) {
    int row = -1;
    if (m < it.hi) row = g.rows ? g.rows[m] : m;
    return (uint32_t)row < (uint32_t)g.a_rows ? row : -1;
  };
  uint32_t from[T::kCopies];
#pragma unroll
  for (int i = 0; i < T::kCopies; ++i) {
    const int r = 8 * (wave % (WR * WC) * T::kCopies + i) + (lane >> 3);
    const int row = source(it.m0 + r);
    from[i] = row < 0 ? kOutOfRange
                      : (uint32_t)row * (uint32_t)g.K + 16u * ((lane & 7) ^ row_swizzle(r));
  }

  // scales of the tile's rows and columns, asked for ahead of everything else
  float scale[T::kScales];
#pragma unroll
  for (int j = 0; j < T::kScales; ++j) {
    const int c = threadIdx.x + j * T::kThreads;
    scale[j] = 0.f;
    if (c < T::kCols) {
      const int n = scale_column(g, cg0 * 16 + c);
      if (n < g.N) scale[j] = g.w_scale[(int64_t)it.e * g.N + n];
    } else if (c < T::kCols + T::kRows) {
      const int row = source(it.m0 + c - T::kCols);
      if (row >= 0) scale[j] = g.a_scale[row];
    }
  }

  intx16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][f][e] = 0;

  uintx4 w[WB][4][FN];
#pragma unroll
  for (int b = 0; b < WB - 1; ++b)
#pragma unroll
    for (int u = 0; u < 4; ++u) tile_load_w<T>(w[b], b, u, P);
#pragma unroll
  for (int s = 0; s < T::NS - 1; ++s)
#pragma unroll
    for (int u = 0; u < 4; ++u) tile_copy<T>(smem + s * T::kStage, s, u, from, P);
  // the fragments and the copies of steps 0 and 1 landed (fewer instructions follow
  // those of step 1 in step 0 than its wait counts on)
  QG_WAIT_VM_BARRIER(T::kCopies);
#pragma unroll
  for (int j = 0; j < T::kScales; ++j)
    if (threadIdx.x + j * T::kThreads < T::kCols + T::kRows) w_scale[threadIdx.x + j * T::kThreads] = scale[j];
  uintx4 x[2][FM];
  tile_read<FM>(x[0], smem + P.lds_read, P, 0);
  // nothing of the lgkm counter left pending on the way into the loop, so the
  // compiler's wait at the loop head is the loop's own
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)

  const int steps = (g.KT + KS - 1) / KS;
  int s = 0;
  for (; s + T::kUnroll <= steps; s += T::kUnroll) tile_steps<T, 0>(s, smem, w, x, from, P, acc);
  tile_last_steps<T, 0>(s, steps, smem, w, x, from, P, acc);

  // every copy and load has landed before the stage memory takes other data
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();

  if constexpr (KS > 1) {
    intx4* part = reinterpret_cast<intx4*>(smem) + lane;   // [wave of kq > 0][fragment][quad][lane]
    constexpr int kOf = FM * FN * 4 * 64;
    if (P.kq > 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            part[(wave - WR * WC) * kOf + ((i * FN + f) * 4 + q) * 64] =
                intx4{acc[i][f][4 * q], acc[i][f][4 * q + 1], acc[i][f][4 * q + 2], acc[i][f][4 * q + 3]};
    }
    __syncthreads();
    if (P.kq == 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < KS - 1; ++k) {
              const intx4 v = part[(k * WR * WC + wave) * kOf + ((i * FN + f) * 4 + q) * 64];
#pragma unroll
              for (int t = 0; t < 4; ++t) acc[i][f][4 * q + t] += v[t];
            }
    }
    __syncthreads();
  }

  // The output tile in LDS, row-major, 16-byte chunk k of row r at slot k ^ (r & mask),
  // then whole rows to memory.
  const int chunks = g.gated ? T::kCols / 16 : T::kCols / 8;
  const int mask = chunks < 16 ? chunks - 1 : 15;
  auto put = [&](auto bf16, auto gated) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = 32 * (FM * wr + i) + (lane & 31);
      const float sa = a_scale[row];
      uint8_t* base = smem + row * (16 * chunks);
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        const intx16& v = acc[i][f];
        const int c0 = 32 * (FN * cw + f) + 4 * (lane >> 5);
#pragma unroll
        for (int q = 0; q < (gated ? 2 : 4); ++q) {
          const floatx4 sw = *reinterpret_cast<const floatx4*>(&w_scale[c0 + 8 * q]);
          float y[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) y[t] = (float)v[4 * q + t] * sa * sw[t];
          int col = c0 + 8 * q;
          if constexpr (gated) {
            const floatx4 su = *reinterpret_cast<const floatx4*>(&w_scale[c0 + 8 * q + 16]);
#pragma unroll
            for (int t = 0; t < 4; ++t) y[t] = gated_value(y[t], (float)v[4 * q + 8 + t] * sa * su[t]);
            col = 16 * (FN * cw + f) + 8 * q + 4 * (lane >> 5);
          }
          const uintx2 d = {rounded_pair<bf16>(y[0], y[1]), rounded_pair<bf16>(y[2], y[3])};
          *reinterpret_cast<uintx2*>(base + 16 * ((col >> 3) ^ (row & mask)) + 2 * (col & 7)) = d;
        }
      }
    }
  };
  if (KS == 1 || P.kq == 0) {
    using Yes = std::true_type;
    using No = std::false_type;
    if (g.gated)
      g.bf16 ? put(Yes(), Yes()) : put(No(), Yes());
    else
      g.bf16 ? put(Yes(), No()) : put(No(), No());
  }
  __syncthreads();
  const int n0 = it.cb * 8 * chunks;
  const int shift = 31 - __builtin_clz(chunks);
  for (int i = threadIdx.x; i < T::kRows << shift; i += T::kThreads) {
    const int row = i >> shift, ch = i & (chunks - 1);
    const int m = it.m0 + row, n = n0 + 8 * ch;
    if (m >= it.hi) break;
    if (n >= g.out_n) continue;
    const uintx4 v = *reinterpret_cast<const uintx4*>(smem + row * (16 * chunks) +
                                                      16 * (ch ^ (row & mask)));
    uint16_t* dst = g.out + (int64_t)m * g.out_n + n;
    if (n + 8 <= g.out_n) {
      *reinterpret_cast<uintx4_any*>(dst) = v;
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (n + t < g.out_n) dst[t] = (uint16_t)(v[t >> 1] >> (16 * (t & 1)));
    }
  }
}

template <class T>
hipError_t launch_tile(const W8a8& p, hipStream_t stream) {
  const Args g = args_of(p, T::kCols);
  hipLaunchKernelGGL((w8a8_tile_kernel<T>), dim3((unsigned)workgroups(p, T::kRows, T::kCols)),
                     dim3(T::kThreads), 0, stream, g);
  return hipGetLastError();
}

// ---- which kernel -----------------------------------------------------------
// What a variant takes is estimated from the sizes, and the least is launched.  An
// item (a workgroup's tile) runs through K in steps of KS K tiles of 128; a step
// takes `step` us, or `shared` us for each item that a CU works on where that is
// more; the weight's bytes stream beside that at 6.9 TB/s and show with the factor
// `stream`; `fixed` us go before and after.  The figures are fitted to 236 sizes of
// plain products in bf16 (N 640 .. 28672, K 1024 .. 8192; 161 of 1 .. 4096 rows, 75 of
// 8 .. 128 experts with 1 .. 1024 rows on average), each timed with those 5 to 12 of the
// variants that come into question for so many rows.  Over these the choice is 0.8 %
// slower than the best timed (0.3 % with one weight, 2.1 % by expert), 17 % at worst.
// Gated products and sizes outside these ranges follow the same rule unmeasured, but for
// some (4096 x 11008 gated, 16 .. 512 rows: 0 to 6 % less than plain).  Single sizes, us:
//   K = N = 8192, 16 / 64 / 256 / 1024 / 4096 rows: 32 columns by 16 rows 12.9 /
//     26.9, 64 x 32 20.0 / 19.7 (32 and 64 rows), 128 x 64 30.7 (256), 256 x 128
//     64.3 (1024), 256 x 256 213 (4096; 256 x 128 219, 128 x 128 260)
//   64 experts, K = 4096, N = 2048, 4 / 16 / 64 / 1024 rows each: 32 x 16 77 / 101
//     / - / -, 128 x 32 99 (16), 128 x 64 115 (64), 256 x 128 497 (1024)
struct Variant {
  int rows, cols, ks, threads;
  float fixed, step, shared, stream;
  hipError_t (*launch)(const W8a8&, hipStream_t);
};

template <int G, int NW>
constexpr Variant slab(float fixed, float step, float shared, float stream) {
  return {16, 16 * G, NW, NW * kWave, fixed, step, shared, stream, launch_slab<G, NW>};
}
template <int FM, int FN, int WR, int WC, int KS, int WB>
constexpr Variant tile(float fixed, float step, float shared, float stream) {
  using T = Tile<FM, FN, WR, WC, KS, WB>;
  return {T::kRows, T::kCols, KS, T::kThreads, fixed, step, shared, stream, launch_tile<T>};
}

constexpr Variant kVariants[] = {
    slab<1, 8>(2.79f, 0.193f, 0.727f, 0.37f),               // 16 x 16; not gated: one of a pair
    slab<2, 4>(3.00f, 0.382f, 0.517f, 0.36f),               // 16 x 32
    slab<4, 4>(2.82f, 0.746f, 0.907f, 0.57f),               // 16 x 64
    tile<1, 1, 1, 1, 4, 4>(3.29f, 0.320f, 0.561f, 1.14f),   // 32 x 32
    tile<1, 1, 1, 2, 4, 2>(3.53f, 0.459f, 0.747f, 1.12f),   // 32 x 64
    tile<1, 1, 1, 4, 1, 4>(3.52f, 0.169f, 0.287f, 1.13f),   // 32 x 128
    tile<2, 1, 1, 2, 2, 4>(4.21f, 0.289f, 0.499f, 1.06f),   // 64 x 64
    tile<2, 1, 1, 4, 1, 4>(3.77f, 0.223f, 0.377f, 1.07f),   // 64 x 128
    tile<4, 1, 1, 4, 1, 4>(5.09f, 0.000f, 0.551f, 1.14f),   // 128 x 128
    tile<3, 2, 1, 4, 1, 2>(5.93f, 0.142f, 0.751f, 1.33f),   // 96 x 256
    tile<4, 2, 1, 4, 1, 2>(7.11f, 0.544f, 0.905f, 1.26f),   // 128 x 256
    tile<4, 2, 2, 4, 1, 2>(6.98f, 1.039f, 1.744f, 0.86f),   // 256 x 256
};

// Of rows that fall on the experts at random: how many experts have any.
double busy_experts(const W8a8& p) {
  return p.offsets ? (double)p.experts * (1 - std::exp(-(double)p.M / (double)p.experts)) : 1;
}

// A launch holds less than 2^32 threads in one dimension of its grid.  Of many columns and
// rows that many experts share a small tile has more; the one of 128 x 256 never has: with
// M N < 2^31 and up to M row blocks more than full ones, 2^23 workgroups of 256 threads.
bool fits_a_launch(const Variant& v, const W8a8& p) {
  return workgroups(p, v.rows, v.cols) * v.threads < (int64_t)1 << 32;
}

double estimate(const Variant& v, const W8a8& p, double busy) {
  // row blocks: of experts with fewer rows than a block one or two each, of others
  // half a block more than full ones
  const double M = (double)p.M, rows = v.rows;
  double blocks = (double)cdiv(p.M, v.rows);
  if (p.offsets) {
    const double each = M / (double)p.experts;
    blocks = M / rows + (each < rows ? busy * (1 - 0.5 * each / rows) : 0.5 * (double)p.experts);
  }
  double items = blocks * (double)cdiv(p.N, v.cols) / 256;   // of a CU
  if (items < 6) items = 0.4 * items + 0.6 * std::ceil(items);   // whole rounds, while there are few
  const double loop = (double)cdiv(cdiv(p.K, kTileK8), v.ks) * std::fmax(v.step, v.shared * items);
  const double stream = v.stream * busy * (double)p.N * (double)p.K / 6.9e6;
  return v.fixed + std::sqrt(loop * loop + stream * stream);
}

const Variant& variant_for(const W8a8& p) {
  const Variant* best = nullptr;
  double least = 0;
  // 16 rows at a time: timed up to 64 rows for each weight
  const bool few = p.M <= 64 * (p.offsets ? p.experts : 1);
  const double busy = busy_experts(p);
  for (const Variant& v : kVariants) {
    if ((v.rows == 16 && !few) || (v.cols == 16 && p.gated)) continue;
    const double t = estimate(v, p, busy);
    if ((!best || t < least) && fits_a_launch(v, p)) {
      best = &v;
      least = t;
    }
  }
  return *best;
}

// ---- prepack ----------------------------------------------------------------
// One thread per 32-bit word of the packed weight, grid y over experts.
__global__ __launch_bounds__(256) void prepack_w8a8_kernel(const int8_t* __restrict__ w,
                                                           uint32_t* __restrict__ out, int K, int N,
                                                           int KT, int64_t words, bool gated) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (d >= words) return;
  const int64_t e = blockIdx.y;
  const int64_t tile = d >> 9;
  const int off = (int)(d & 511) * 4, h = off >> 10, lane = (off & 1023) >> 4;
  const int cg = (int)(tile / KT), kt = (int)(tile - (int64_t)cg * KT);
  int n = cg * kTileN + (lane & 15);
  if (gated) {
    const int f = (cg >> 1) * kTileN + (lane & 15);
    n = f < N / 2 ? (cg & 1) * (N / 2) + f : N;
  }
  const int k0 = kt * kTileK8 + 32 * (lane >> 4) + 16 * h + (off & 15);
  uint32_t word = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (n < N && k0 + b < K)
      word |= (uint32_t)(uint8_t)w[(e * K + k0 + b) * N + n] << (8 * b);
  out[e * words + d] = word;
}

}  // namespace

hipError_t launch_prepack_w8a8(const int8_t* w, void* packed, int64_t experts, int64_t K, int64_t N,
                               bool gated, hipStream_t stream) {
  const W8a8Geom g = w8a8_geom(K, N, gated);
  const int64_t words = g.bytes / 4;
  hipLaunchKernelGGL(prepack_w8a8_kernel, dim3((unsigned)cdiv(words, 256), (unsigned)experts),
                     dim3(256), 0, stream, w, static_cast<uint32_t*>(packed), (int)K, (int)N,
                     (int)g.kt, words, gated);
  return hipGetLastError();
}

hipError_t launch_w8a8(const W8a8& p, hipStream_t stream) { return variant_for(p).launch(p, stream); }

W8a8Tile w8a8_tile(const W8a8& p) {
  const Variant& v = variant_for(p);
  return W8a8Tile{v.rows, v.cols, v.ks};
}

}  // namespace qgemm
