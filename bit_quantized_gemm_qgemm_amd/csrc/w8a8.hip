// Products of 8-bit integers with scales for each token and channel, for one
// weight or for rows grouped by expert, plain or gated.
//
//   Y[m, n] = (sum_k A[m, k] W[k, n]) * a_scale[m] * w_scale[n]
//   gated, N = 2F:  H[m, f] = silu(Y[m, f]) * Y[m, F + f],  silu(y) = y / (1 + exp(-y))
//
// The sum is exact in 32 bits (|A W| <= 2^14 and K < 2^17); it becomes fp32 with
// one rounding, the scales multiply it in fp32, and the result is rounded once to
// the output type.
#include "qgemm_common.h"

namespace qgemm {
namespace {

constexpr uint32_t kPastEnd = 0x80000000u;   // past every activation buffer

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

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
  g.col_blocks = (int)cdiv(geom.cg * kTileN, cols);
  g.gated = p.gated;
  g.bf16 = p.bf16;
  return g;
}

// Row blocks that a launch has at most: an expert's last block may be part full.
int64_t most_row_blocks(const W8a8& p, int64_t rows) {
  if (!p.offsets) return cdiv(p.M, rows);
  return (p.M < p.experts ? p.M : p.experts) + p.M / rows;
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

// The workgroups' items lie in one row: expert after expert, of each its column
// blocks in turn, and of a column block the row blocks.  Workgroups are handed
// to the 8 XCDs round-robin; each XCD takes an eighth of the row, so that the
// row blocks that share a weight tile meet in one L2.  The experts' places
// in the row follow from their row counts: a wave counts the blocks of all
// experts, each lane those of `per` neighbours.
template <int BM>
__device__ __forceinline__ Item item_of(const Args& g) {
  Item it{0, 0, g.M, 0, true};
  int blocks = (g.M + BM - 1) / BM, before = 0, q = 0;
  const int lane = threadIdx.x & 63;
  int total = blocks, mine = 0, upto = 0;
  const int per = (g.experts + 63) / 64;
  if (g.offsets) {
    for (int j = 0; j < per; ++j) {
      const int e = lane * per + j;
      if (e < g.experts) {
        const int2 r = rows_of(g, e);
        mine += (r.y - r.x + BM - 1) / BM;
      }
    }
    upto = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    total = __builtin_amdgcn_readlane(upto, 63);
  }
  const int items = total * g.col_blocks, share = (items + 7) / 8;
  const int slot = blockIdx.x >> 3, i = (int)(blockIdx.x & 7) * share + slot;
  if (slot >= share || i >= items) {
    it.some = false;
    return it;
  }
  if (g.offsets) {
    q = i / g.col_blocks;   // lies among the blocks of its expert
    const int at = __builtin_ctzll(__ballot(upto > q));
    before = __builtin_amdgcn_readlane(upto - mine, at);
    it.e = at * per;
    for (;; ++it.e) {
      const int2 r = rows_of(g, it.e);
      blocks = (r.y - r.x + BM - 1) / BM;
      if (q < before + blocks) {
        it.m0 = __builtin_amdgcn_readfirstlane(r.x);
        it.hi = __builtin_amdgcn_readfirstlane(r.y);
        break;
      }
      before += blocks;
    }
    blocks = __builtin_amdgcn_readfirstlane(blocks);
    it.e = __builtin_amdgcn_readfirstlane(it.e);
  }
  const int rem = __builtin_amdgcn_readfirstlane(i - before * g.col_blocks);
  it.cb = rem / blocks;
  it.m0 += (rem - it.cb * blocks) * BM;
  return it;
}

// Column of the output, and of the weight's scales, of packed column c.
__device__ __forceinline__ int scale_column(const Args& g, int c) {
  if (!g.gated) return c;
  const int f = (c >> 5) * 16 + (c & 15);
  return f < g.out_n ? ((c >> 4) & 1) * g.out_n + f : g.N;   // N: none
}

// silu(gate) * up
__device__ __forceinline__ float gated_value(float gate, float up) {
  return gate / (1.0f + __expf(-gate)) * up;
}

__device__ __forceinline__ uint16_t rounded(float v, bool bf16) {
  return bf16 ? f32_to_bf16_rne(v) : f32_to_f16_bits(v);
}

// ---- up to 16 rows ----------------------------------------------------------
// A workgroup owns 16 rows and G column groups of 16; its NW waves share the K
// tiles.  Weight tiles go from memory straight into registers, D tiles ahead,
// and meet the rows' codes in 16 x 16 x 64 matrix instructions; the waves' sums
// meet in LDS.
template <int G>
struct SlabTile {
  uintx4 x[2], w[G][2];
};

template <int G, int NW, int D>
__global__ __launch_bounds__(NW * kWave) void w8a8_slab_kernel(const Args g) {
  __shared__ intx4 red[NW][G][kWave];
  __shared__ float a_scale[16], w_scale[16 * G];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Item it = item_of<16>(g);
  if (!it.some) return;   // the whole workgroup
  const int cg0 = it.cb * G;

  uint32_t xoff = kPastEnd;
  {
    const int m = it.m0 + (lane & 15);
    int row = -1;
    if (m < it.hi) row = g.rows ? g.rows[m] : m;
    const bool some = (uint32_t)row < (uint32_t)g.a_rows;
    if (some) xoff = (uint32_t)row * (uint32_t)g.K + 32u * (lane >> 4);
    if (threadIdx.x < 16) a_scale[threadIdx.x] = some ? g.a_scale[row] : 0.f;
    if (threadIdx.x < 16 * G) {
      const int c = scale_column(g, cg0 * 16 + (int)threadIdx.x);
      w_scale[threadIdx.x] = c < g.N ? g.w_scale[(int64_t)it.e * g.N + c] : 0.f;
    }
  }
  const int64_t w0 = (int64_t)cg0 * g.KT * kTileBytes;
  const __amdgpu_buffer_rsrc_t xr = buffer_of(g.a, g.a_bytes);
  const __amdgpu_buffer_rsrc_t wr =
      buffer_of(g.w + it.e * g.w_bytes + w0, (uint32_t)(g.w_bytes - w0));
  const int last = g.CG - 1 - cg0;
  const uint32_t stride = (uint32_t)g.KT * kTileBytes;

  // (codes past K in the last tile are the next row's: they meet zeros of W)
  auto load = [&](SlabTile<G>& t, int kt) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      t.x[h] = __builtin_amdgcn_raw_buffer_load_b128(xr, xoff + 128u * kt + 16u * h, 0, 0);
#pragma unroll
    for (int j = 0; j < G; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        t.w[j][h] = __builtin_amdgcn_raw_buffer_load_b128(
            wr, 16u * lane + 1024u * h, (uint32_t)min(j, last) * stride + (uint32_t)kTileBytes * kt, 2);
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

  SlabTile<G> ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load(ring[d], min(wave + d * NW, g.KT - 1));
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

template <int G, int NW, int D>
hipError_t launch_slab(const W8a8& p, hipStream_t stream) {
  const Args g = args_of(p, 16 * G);
  const int64_t items = most_row_blocks(p, 16) * g.col_blocks;
  hipLaunchKernelGGL((w8a8_slab_kernel<G, NW, D>), dim3((unsigned)(cdiv(items, 8) * 8)),
                     dim3(NW * kWave), 0, stream, g);
  return hipGetLastError();
}

// ---- prepack ----------------------------------------------------------------
// One thread per 32-bit word of the packed weight, grid z over experts.
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

hipError_t launch_w8a8(const W8a8& p, hipStream_t stream) {
  return launch_slab<2, 8, 2>(p, stream);
}

}  // namespace qgemm
