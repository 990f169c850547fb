// Attention of one new token per request over the paged key-value cache.
//
// For one request and one kv head, the heads that share it (up to 16 of them)
// are the columns of two matrix products over a tile of 32 tokens:
//   S^T [32 tokens x 16 heads] = K [32 x D] Q^T [D x 16]
//   O^T [D x 16 heads]        += V^T [D x 32] P^T [32 x 16],  P = exp2(S - m)
// with the running maximum m and sum l of each head kept per lane column.
// The K index of a matrix instruction may be permuted freely as long as both
// operands agree, and both uses of that keep what is loaded and what is computed
// from it in its lane, K, V and P without LDS or shuffles (Q^T waits in LDS; row
// numbers go round by shuffles, maxima by moves between lanes):
//   - the 4 tokens that a lane holds of each S^T tile are the ones that it
//     feeds as P^T: the token order of O^T's product is chosen as the order
//     that S^T's accumulators come in;
//   - V is read by rows (a lane takes W elements of 8 tokens, in pieces of up
//     to 16 bytes that lie side by side in the 16 lanes of a token) and
//     transposed inside the lane by byte permutes, so that instruction j of
//     the W makes the outputs d = PW m + j of its piece.
// The work is 4 D (K and V bytes) against 4 D group flops per token: bound by
// the cache's bytes for every group.  What matters is bytes in flight: each
// wave keeps one 32-token tile of K and V loading while it works on the last.
// 128K tokens of 8 x 128, bf16, take 85.3 us (6.3 TB/s; a plain read reaches
// 7.1), of which 1.4 go by before the first load; neither a fourth workgroup a
// CU, nor smaller shares, nor waves kept in step by priorities change that.
// The join's launch adds 6 us and the gap before it.  A short call is latency:
// 204 tokens take 6.0 us, 32 tokens 4.5.
#include "qgemm_common.h"

namespace qgemm {
namespace {

typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kAttnWaves = 4;
constexpr int kTileTokens = 32;
constexpr int kMaxGroup = 16;           // heads of one item: the columns of a matrix tile
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
  PagedAttention a;
  uint32_t page_magic, page_shift;   // token / page_size = umulhi(2 token, magic) >> shift
  int group;                         // heads of an item (its last chunk may hold fewer)
  int chunks;                        // items per kv head
  int groups;                        // workgroups that share the tiles; 0: one item each
  int slot_floats;                   // of a partial result
  // in the workspace, where workgroups share items
  uint32_t* parts;                   // [batch * items]: first workgroup << 16 | further ones
  float* partial;                    // two slots for each workgroup
};

// What a partial result holds: m[16], l[16], then o[heads][dim].
constexpr int kSlotHead = 2 * kMaxGroup;

template <int DT, bool E4M3, int KS, bool FULL>
struct Attn {
  static constexpr int W = KS <= 2 ? 4 : KS <= 4 ? 8 : 16;   // elements of V per lane and token
  // K: a lane takes 16 bytes of a row at a time, 4 lanes 64 bytes of it: the
  // elements of one step of 32, or of two steps for e4m3
  static constexpr int KE = E4M3 ? 16 : 8;
  static constexpr int KL = KS * 8 / KE;                     // loads per row
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int VD = W * ES / 4;                      // dwords of W elements of V
  static constexpr int PW = W * ES > 16 ? 16 / ES : W;       // elements of a piece of V
  static constexpr int PD = PW * ES / 4, NP = W / PW;        // its dwords; pieces
  // Rows of 32 KS elements that one item reads are loaded non-temporally: kept out
  // of the caches they leave them to what is read again (270 MB of bf16, 128
  // elements: 60.8 us through the caches, 54.7 past them).  Otherwise the caches
  // serve a second read: lanes past a shorter row's end take its last elements
  // again (80 elements: 57.8 us, and 62.3 past them; 160, though whole sectors,
  // 62.0 and 65.6; 224 73.3 and 78.0), or further items all of it (32 heads a kv
  // head: 90 and 103).
  static constexpr bool kOnce = FULL;
  // probabilities and V enter the matrix cores as fp16 for e4m3 (its values
  // are exact there, and P takes two parts of fp16), else in the cache's type
  static constexpr bool kHalfPV = E4M3 || DT == 1;
  // 16-bit parts whose sum is a probability: bf16's three hold all 24 bits of
  // fp32; fp16's two, each rounded to nearest, 23 (what is left is 2^-23, or
  // 2^-39 of the largest where that is more: see bias).  Two parts of
  // bf16 left up to 2^-15, always towards 0, while l held all of it.  The third
  // costs nothing where bytes bound the call; where waves wait for one tile after
  // the other, 13 requests of up to 935 tokens of 8 x 80 take 10.1 us, 9.6 with two.
  static constexpr int kParts = kHalfPV ? 2 : 3;
  // workgroups of a CU, by the registers that a tile's K, V and sums take
  // (98 to 115 up to 64 elements, 126 to 167 up to 128, 179 to 256 past them,
  // where 16-bit rows of 208 elements on spill 8 to 15 if they are not whole or
  // several items read them).  e4m3 of 128
  // elements has room for a fourth and gains nothing by it (67.9 and 68.3 us).
  static constexpr int kResident = KS > 4 ? 2 : KS > 2 ? 3 : 4;
  // A factor 2^bias on the probabilities, and so on l, the same for all parts
  // of an item.  fp16's smallest stay normal.  bf16's add up to 1 at most over
  // the item's n tokens: sums stay finite for values up to the type's largest,
  // and products are no smaller than an evenly weighted mean's have to be (one
  // token of the smallest normal value keeps it; a factor for the longest
  // request, 2^-30, made 0 of it).
  static __device__ __forceinline__ float bias(int n) {
    return kHalfPV ? 15.0f : -(float)(32 - __clz(n - 1));
  }
};

// x of this lane and of the lane 16 (or 32) lanes away, as the two results of
// exchanging rows between two copies of x.
template <int DIST>
__device__ __forceinline__ floatx2 both(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto y = DIST == 16 ? __builtin_amdgcn_permlane16_swap(u, u, false, false)
                            : __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t y0 = y[0], y1 = y[1];
  return floatx2{__builtin_bit_cast(float, y0), __builtin_bit_cast(float, y1)};
}

// over the four lanes 16 apart
__device__ __forceinline__ float max_over_groups(float x) {
  floatx2 y = both<16>(x);
  y = both<32>(fmaxf(y[0], y[1]));
  return fmaxf(y[0], y[1]);
}

__device__ __forceinline__ float sum_over_groups(float x) {
  floatx2 y = both<16>(x);
  y = both<32>(y[0] + y[1]);
  return y[0] + y[1];
}

// x of lane I of this lane's 16
template <int I>
__device__ __forceinline__ uint64_t in_group(uint64_t x) {
  const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)x, 0x150 + I, 0xf, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(x >> 32), 0x150 + I, 0xf, 0xf, false);
  return (uint64_t)hi << 32 | lo;
}

// Four e4m3 codes -> two dwords of 16-bit pairs (exact in fp16 and in bf16).
template <bool HALF>
__device__ __forceinline__ void expand_e4m3(uint32_t c, uint32_t* out) {
  if constexpr (HALF) {
    out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false));
    out[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true));
  } else {
    out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
    out[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
  }
}

template <bool HALF>
__device__ __forceinline__ floatx4 mma(uintx4 a, uintx4 b, floatx4 c) {
  if constexpr (HALF)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                                  __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

template <bool ONCE, class T>
__device__ __forceinline__ T load(const uint8_t* p) {
  const T* x = reinterpret_cast<const T*>(p);
  if constexpr (ONCE) return __builtin_nontemporal_load(x);
  return *x;
}

// N dwords from p: 1, 2 or 4.
template <bool ONCE, int N>
__device__ __forceinline__ void load_dwords(uint32_t* r, const uint8_t* p) {
  if constexpr (N == 4) {
    const uintx4 v = load<ONCE, uintx4>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = v[j];
  } else if constexpr (N == 2) {
    const uintx2 v = load<ONCE, uintx2>(p);
    r[0] = v[0];
    r[1] = v[1];
  } else {
    static_assert(N == 1, "4, 8 or 16 bytes");
    r[0] = load<ONCE, uint32_t>(p);
  }
}

template <int DT>
__device__ __forceinline__ uint16_t to_bits(float y) {
  return DT == 1 ? f32_to_f16_bits(y) : f32_to_bf16_rne(y);
}

// x without what bf16 does not hold of it: x less that is exact.
__device__ __forceinline__ float truncated(float x) {
  return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0xffff0000u);
}

// The tokens of request b that count: [first, n).
__device__ __forceinline__ void token_range(const PagedAttention& a, int b, int* first, int* n) {
  int len = a.lens[b];
  len = len < 0 ? 0 : (len < a.limit ? len : (int)a.limit);
  *n = len;
  *first = a.window > 0 && len > a.window ? len - (int)a.window : 0;
}

__device__ __forceinline__ int tiles_of(const PagedAttention& a, int b) {
  int first, n;
  token_range(a, b, &first, &n);
  return (n - first + kTileTokens - 1) / kTileTokens;
}

// The tiles of all items stand in one row, request by request, item by item,
// each item followed by kItemCost empty places: what it costs a workgroup to
// take up one more (its first loads, the join of its waves), in tiles.
// Workgroup w gets the w-th of `used` equal stretches of that row.  With 8
// places against none: 64 requests of 256 to 8192 tokens, e4m3, 77 -> 68 us.
constexpr int kItemCost = 8;
constexpr int kMinShare = 2 * kAttnWaves;   // places: two tiles a wave (four measured the same)

__device__ __forceinline__ int places_of(int tiles) { return tiles > 0 ? tiles + kItemCost : 0; }

struct Stretches {
  uint64_t size, longer;   // the first `longer` of them hold one place more
  __device__ __forceinline__ Stretches(uint64_t total, uint64_t used) {
    size = total / used;
    longer = total - size * used;
  }
  __device__ __forceinline__ uint64_t start(uint64_t w) const {
    return w * size + (w < longer ? w : longer);
  }
  __device__ __forceinline__ uint32_t holder(uint64_t place) const {
    const uint64_t split = longer * (size + 1);
    return (uint32_t)(place < split ? place / (size + 1) : longer + (place - split) / size);
  }
};

struct AttnShared {
  float m[kAttnWaves][kMaxGroup], l[kAttnWaves][kMaxGroup];
  uint32_t scan[kAttnWaves];
  uint32_t before;
  int request;
};

// Element d of one head's sum over tokens [t0, t1) where it came out infinite or
// NaN and the sum of the weights did not.  The matrix cores multiply an infinite
// value by parts of its weight that may be 0, and a weight itself may be below
// fp32's range; but every weight of a finite score is above 0, so the sum is that
// infinity, NaN for two of both signs, for a NaN among the values and for a
// score of -infinity at an infinite value.  One lane reads the values again, one
// after the other, and the key of an infinite one: slow, and only for such sums
// (128K tokens of 8 x 128: 97 us, 17 ms if every value is infinite).
template <int DT>
__device__ __forceinline__ float sum_of_infinities(int b, int kvh, int head, int d, int t0, int t1,
                                                   float sum) {
  // the kernel's argument read anew: what only this uses takes no registers earlier
  auto fresh = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(fresh));
  const AttnArgs& args = *reinterpret_cast<const AttnArgs*>(fresh);
  const PagedAttention& a = args.a;
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)b * a.q_batch_stride +
                      (int64_t)head * a.q_head_stride;
  const int head_row = kvh * a.pool.head_rows;
  auto value = [](uint16_t bits) {
    return DT == 1 ? (float)__builtin_bit_cast(_Float16, bits)
                   : __builtin_bit_cast(float, (uint32_t)bits << 16);
  };
  bool up = false, down = false;
#pragma unroll 1
  for (int t = t0; t < t1; ++t) {
    const int page = (int)(__umulhi(2u * (uint32_t)t, args.page_magic) >> args.page_shift);
    const int e = table[page];
    if (e < 0 || e >= a.pool.pages) continue;
    const int row = e * a.pool.page_rows + head_row + (t - page * a.pool.page_size) * a.pool.token_rows;
    const int64_t at = (int64_t)row * a.dim;
    const float v = value(static_cast<const uint16_t*>(a.v_cache)[at + d]);
    if (fabsf(v) < INFINITY) continue;
    if (v != v) return v;
    const uint16_t* k = static_cast<const uint16_t*>(a.k_cache) + at;
    float s = 0.f;
    for (int x = 0; x < a.dim; x += 8) {
      const uintx4 qx = *reinterpret_cast<const uintx4*>(q + x), kx = *reinterpret_cast<const uintx4*>(k + x);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        s = __builtin_fmaf(value((uint16_t)(qx[j >> 1] >> (16 * (j & 1)))),
                           value((uint16_t)(kx[j >> 1] >> (16 * (j & 1)))), s);
    }
    if (s * (a.scale * kLog2e) == -INFINITY) return __builtin_nanf("");
    if (v > 0.f) up = true; else down = true;
  }
  if (up && down) return __builtin_nanf("");
  return up ? INFINITY : down ? -INFINITY : sum;
}

// Tokens [t0, t1) of one item (request b, heads h0 .. h0 + hn - 1, which share
// kv head kvh, out of `span` tokens) through the waves of the workgroup; the
// joined result goes to `out` (divided and scaled) or, unscaled, to `slot`.
template <int DT, bool E4M3, int KS, bool FULL>
__device__ __forceinline__ void attend(const AttnArgs& args, AttnShared& sh, uintx4* sq, float* so, int b,
                                       int kvh, int h0, int hn, int t0, int t1, int span, float* slot) {
  using A = Attn<DT, E4M3, KS, FULL>;
  constexpr int W = A::W, KE = A::KE, KL = A::KL, VD = A::VD, PW = A::PW;
  constexpr bool kHalfPV = A::kHalfPV;
  const PagedAttention& a = args.a;
  const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int D = a.dim;

  const float bias = A::bias(__builtin_amdgcn_readfirstlane(span));
  const float kscale = (E4M3 ? a.k_scale[kvh] : 1.0f) * a.scale * kLog2e;
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  const int head_row = kvh * a.pool.head_rows;
  const uint8_t* kc = static_cast<const uint8_t*>(a.k_cache);
  // lanes past the row's end read its last elements (never stored)
  const uint8_t* vc[A::NP];
#pragma unroll
  for (int i = 0; i < A::NP; ++i) {
    const int d = PW * (16 * i + r);
    vc[i] = static_cast<const uint8_t*>(a.v_cache) + (d < D ? d : D - PW) * A::ES;
  }
  const uint32_t row_bytes = (uint32_t)D * A::ES;

  floatx4 acc[W];
#pragma unroll
  for (int j = 0; j < W; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  constexpr int kStep = kTileTokens * kAttnWaves;
  // A lane looks up one token of a tile (lanes r >= 8 repeat): the one whose V
  // row the whole group g takes as its r-th, so that row goes round the group
  // by a broadcast within its 16 lanes.
  const int my_token = 16 * ((r >> 2) & 1) + 4 * g + (r & 3);
  // Table entry of that token; past the end, of the last one.
  auto entry = [&](int t) {
    t += my_token;
    t = t < t1 ? t : t1 - 1;
    return table[__umulhi(2u * (uint32_t)t, args.page_magic) >> args.page_shift];
  };
  // Its row, or -1 where the token does not count.
  auto row = [&](int t, int32_t e) {
    t += my_token;
    const int page = (int)(__umulhi(2u * (uint32_t)t, args.page_magic) >> args.page_shift);
    const int off = t - page * a.pool.page_size;
    const bool ok = t < t1 && e >= 0 && e < a.pool.pages;
    return ok ? e * a.pool.page_rows + head_row + off * a.pool.token_rows : -1;
  };
  // lanes that looked up tokens r and 16 + r
  const int k_lane = 16 * (r >> 2) + (r & 3);
  uintx4 kr[2][KL];
  uint32_t vr[8][VD];
  // Tokens that do not count read row 0 of the pool (there is one: a pool
  // without pages has no tokens); what they read is dropped.
  auto load_k = [&](const int (&x)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* p = kc + (uint64_t)(uint32_t)x[u] * row_bytes;
#pragma unroll
      for (int s = 0; s < KL; ++s) {
        const int d = KE * (4 * s + g);
        kr[u][s] = load<A::kOnce, uintx4>(p + (FULL || d < D ? d : D - KE) * A::ES);
      }
    }
  };
  auto load_v = [&](int rows) {
    const uint64_t at = (uint64_t)(uint32_t)(rows < 0 ? 0 : rows) * row_bytes;
    auto token = [&](uint32_t* v, uint64_t at) {
#pragma unroll
      for (int i = 0; i < A::NP; ++i) load_dwords<A::kOnce, A::PD>(v + A::PD * i, vc[i] + at);
    };
    token(vr[0], in_group<0>(at));
    token(vr[1], in_group<1>(at));
    token(vr[2], in_group<2>(at));
    token(vr[3], in_group<3>(at));
    token(vr[4], in_group<4>(at));
    token(vr[5], in_group<5>(at));
    token(vr[6], in_group<6>(at));
    token(vr[7], in_group<7>(at));
  };
  auto k_rows = [&](int rows, int (&x)[2]) {
    rows = rows < 0 ? 0 : rows;
    x[0] = __shfl(rows, k_lane, 64);
    x[1] = __shfl(rows, k_lane + 4, 64);
  };

  // Q^T goes to LDS as the lanes of a wave read it: lane (head r, group g) takes the
  // elements of each step that it takes of K.  Read again for every tile: 4 KS
  // registers less.  Wave w brings steps w, w + 4, ...; loaded first, stored
  // once the wave's first tile is on its way.
  constexpr int kQSteps = (KS + kAttnWaves - 1) / kAttnWaves;
  uintx4 qx[kQSteps];
  {
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)b * a.q_batch_stride +
                        (int64_t)(h0 + (r < hn ? r : 0)) * a.q_head_stride;
#pragma unroll
    for (int x = 0; x < kQSteps; ++x) {
      const int s = wave + kAttnWaves * x;
      const int d = E4M3 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
      qx[x] = uintx4{0, 0, 0, 0};
      if (r < hn && s < KS && (FULL || d < D)) qx[x] = *reinterpret_cast<const uintx4*>(q + d);
    }
  }
  int t = t0 + kTileTokens * wave;
  int32_t next_entry = 0;
  int rows = -1, kx_rows[2];
  if (t < t1) {
    next_entry = entry(t + kStep);
    rows = row(t, entry(t));
    k_rows(rows, kx_rows);
    load_k(kx_rows);
    // K before V here as in the loop: the loop's wait for K then leaves V in flight
    asm volatile("" ::: "memory");
    load_v(rows);
  }
#pragma unroll
  for (int x = 0; x < kQSteps; ++x)
    if (wave + kAttnWaves * x < KS) sq[64 * (wave + kAttnWaves * x) + lane] = qx[x];
  __syncthreads();
  for (; t < t1; t += kStep) {
    asm volatile("" ::: "memory");   // Q stays in LDS: not hoisted out of the loop
    const int32_t far_entry = entry(t + 2 * kStep);
    const int next_rows = row(t + kStep, next_entry);
    k_rows(next_rows, kx_rows);
    const uint64_t counts = __ballot(rows >= 0);

    // S^T
    floatx4 sc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const uintx4 qf = sq[64 * s + lane];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uintx4 kx = kr[u][s * 8 / KE];
        // the row's end falls into the last two steps
        if (!FULL && s >= KS - 2 && KE * (4 * (s * 8 / KE) + g) >= D) kx = uintx4{0, 0, 0, 0};
        if constexpr (E4M3) {
          uint32_t x[4];
          expand_e4m3<DT == 1>(kx[2 * (s & 1)], x);
          expand_e4m3<DT == 1>(kx[2 * (s & 1) + 1], x + 2);
          kx = uintx4{x[0], x[1], x[2], x[3]};
        }
        sc[u] = mma<DT == 1>(kx, qf, sc[u]);
      }
    }
    load_k(kx_rows);

    // softmax over the tile: lane (head r, group g) has tokens 4 g + i of both halves
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = sc[i >> 2][i & 3] * kscale;
    if (counts != ~0ull) {
      // of the lanes that looked them up; formed here (and V waited for here
      // only: a branch, not selects), eight masks kept for it took 16 registers
      uint32_t mine = (uint32_t)(counts >> (16 * g));
      asm volatile("" : "+v"(mine));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool ok = (mine >> i) & 1;
        p[i] = ok ? p[i] : -INFINITY;
#pragma unroll
        for (int j = 0; j < VD; ++j) vr[i][j] = ok ? vr[i][j] : 0u;
      }
    }
    float top = p[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, p[i]);
    // m is the maximum rounded up to a whole number: the factor 2^bias, the
    // difference of two m and the shrinking by it are exact, and m moves less
    top = fmaxf(m, __builtin_ceilf(max_over_groups(top)));
    const float base = (top == -INFINITY ? 0.f : top) - bias;
    if (__any(top != m)) {
      const float shrink = __builtin_amdgcn_exp2f(m - (top == -INFINITY ? 0.f : top));
      l *= shrink;
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] *= shrink;
      m = top;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(p[i] - base);
      l += p[i];
    }
    // P^T in 16-bit parts that add up to it
    uintx4 part[A::kParts];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = p[2 * i], y = p[2 * i + 1];
      if constexpr (kHalfPV) {
        const half2_t h = __builtin_convertvector((floatx2{x, y}), half2_t);
        const floatx2 rest = {x - (float)h[0], y - (float)h[1]};
        part[0][i] = __builtin_bit_cast(uint32_t, h);
        part[1][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, half2_t));
      } else {
#pragma unroll
        for (int n = 0; n < A::kParts; ++n) {
          part[n][i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, y),
                                             __builtin_bit_cast(uint32_t, x), 0x07060302u);
          x -= truncated(x);
          y -= truncated(y);
        }
      }
    }
    // O^T: two elements (one dword of V's 16-bit values) of 8 tokens at a time
#pragma unroll
    for (int j4 = 0; j4 < W / 4; ++j4) {
      uint32_t vx[8][2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (E4M3) {
          expand_e4m3<true>(vr[i][j4], vx[i]);
        } else {
          vx[i][0] = vr[i][2 * j4];
          vx[i][1] = vr[i][2 * j4 + 1];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        uintx4 vf[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vf[0][i] = __builtin_amdgcn_perm(vx[2 * i + 1][j >> 1], vx[2 * i][j >> 1], 0x05040100u);
          vf[1][i] = __builtin_amdgcn_perm(vx[2 * i + 1][j >> 1], vx[2 * i][j >> 1], 0x07060302u);
        }
#pragma unroll
        for (int n = 0; n < A::kParts; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            acc[4 * j4 + j + y] = mma<kHalfPV>(vf[y], part[n], acc[4 * j4 + j + y]);
      }
    }
    load_v(next_rows);
    rows = next_rows;
    next_entry = far_entry;
  }
  l = sum_over_groups(l);

  // Join the waves: sh.m, sh.l and so [wave][head][dim]
  const int pitch = D + 4;
  if (g == 0) {
    sh.m[wave][r] = m;
    sh.l[wave][r] = l;
  }
  if (r < hn) {
    float* o = so + (wave * args.group + r) * pitch;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < A::NP; ++x) {
        const int d = PW * (16 * x + 4 * g + i);
        if (d < D) {
#pragma unroll
          for (int j = 0; j < PW; ++j) o[d + j] = acc[PW * x + j][i];
        }
      }
  }
  __syncthreads();
  auto join = [&](auto&& fix) {
    for (int x = (int)threadIdx.x; x < hn * D; x += 64 * kAttnWaves) {
      const int h = x / D, d = x - h * D;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) top = fmaxf(top, sh.m[w][h]);
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(sh.m[w][h] - base);
        sum += f * sh.l[w][h];
        o += f * so[(w * args.group + h) * pitch + d];
      }
      fix(h, d, sum, o);
      if (slot) {
        if (d == 0) {
          slot[h] = top;
          slot[kMaxGroup + h] = sum;
        }
        slot[kSlotHead + h * D + d] = o;
      } else {
        const float y = sum == 0.f ? 0.f : o / sum * (E4M3 ? a.v_scale[kvh] : 1.0f);
        static_cast<uint16_t*>(a.out)[((int64_t)b * a.heads + h0 + h) * D + d] = to_bits<DT>(y);
      }
    }
  };
  auto odd = [](float sum, float o) { return !(fabsf(o) < INFINITY) && fabsf(sum) < INFINITY; };
  // Joined once more, seldom, where infinite values met (they are only noted here: in
  // this loop their code made short calls 0.2 us longer).
  bool again = false;
  join([&](int, int, float sum, float o) { again |= odd(sum, o); });
  if constexpr (!E4M3)   // whose values are finite or NaN
    if (__builtin_expect(again, 0))
      join([&](int h, int d, float sum, float& o) {
        if (odd(sum, o))
          o = sum_of_infinities<DT>(b, kvh, h0 + h, d, t0, t1, o);
      });
  __syncthreads();
}

// Item i of a request: kv head i / chunks, heads from chunk i % chunks on.
__device__ __forceinline__ void item_heads(const AttnArgs& args, int i, int* kvh, int* h0,
                                           int* hn) {
  const int per = args.a.heads / args.a.kv_heads;
  *kvh = i / args.chunks;
  const int c = (i - *kvh * args.chunks) * args.group;
  *h0 = *kvh * per + c;
  *hn = per - c < args.group ? per - c : args.group;
}

template <int DT, bool E4M3, int KS, bool FULL>
__global__ __launch_bounds__(64 * kAttnWaves, (Attn<DT, E4M3, KS, FULL>::kResident))
void paged_attention_kernel(const AttnArgs args) {
  __shared__ uintx4 sq[64 * KS];
  __shared__ float so[kAttnWaves * kMaxGroup * (32 * KS + 4)];
  __shared__ AttnShared sh;
  const PagedAttention& a = args.a;
  const int items = a.kv_heads * args.chunks;
  int kvh, h0, hn;
  if (args.groups == 0) {   // one item per workgroup
    const int b = (int)blockIdx.x / items;
    item_heads(args, (int)blockIdx.x - b * items, &kvh, &h0, &hn);
    int first, n;
    token_range(a, b, &first, &n);
    attend<DT, E4M3, KS, FULL>(args, sh, sq, so, b, kvh, h0, hn, first, n, n - first, nullptr);
    return;
  }
  // The places of all items (see Stretches), whatever the lengths are.
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int kThreads = 64 * kAttnWaves;
  // the requests without tokens among blockIdx.x, + gridDim.x, ... are this workgroup's
  const bool empty = (int)blockIdx.x < a.batch && tiles_of(a, (int)blockIdx.x) == 0;
  uint64_t start = 0, end = 0;
  uint32_t sum = 0, inc = 0, mine = 0;   // places over one item: below 2^32 by the host's checks
  auto scan = [&](int b0) {   // the sum up to request b0 + tid, this one's included, in inc
    const int x = b0 + tid;
    mine = x < a.batch ? places_of(tiles_of(a, x)) : 0;
    inc = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t y = __shfl_up(inc, off, 64);
      if (lane >= off) inc += y;
    }
    if (lane == 63) sh.scan[wave] = inc;
    __syncthreads();
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      const uint32_t y = sh.scan[w];
      if (w < wave) inc += y;
      all += y;
    }
    inc += sum;
    sum += all;
  };
  auto find = [&](int b0) {   // the request that holds the start
    if (start < end && (uint64_t)items * (inc - mine) <= start && start < (uint64_t)items * inc) {
      sh.request = b0 + tid;
      sh.before = inc - mine;
    }
    __syncthreads();   // also before sh.scan is written again
  };
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    if (b0 > 0) __syncthreads();
    scan(b0);
  }
  const uint64_t total = (uint64_t)items * (uint32_t)__builtin_amdgcn_readfirstlane(sum);
  uint64_t used = total / kMinShare;
  used = used < 1 ? 1 : used < (uint64_t)args.groups ? used : args.groups;
  const Stretches shares(total, used);
  if (blockIdx.x < used) {
    start = shares.start(blockIdx.x);
    end = shares.start(blockIdx.x + 1);
  }
  if (a.batch <= kThreads) {   // the sums are still at hand
    find(0);
  } else {
    sum = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      __syncthreads();
      scan(b0);
      find(b0);
    }
  }
  int b = 0;
  uint64_t before = 0;   // places of the requests before b
  // what follows is the same in all lanes: in scalar registers it leaves the loop's alone
  if (start < end) {
    b = __builtin_amdgcn_readfirstlane(sh.request);
    before = (uint64_t)items * (uint32_t)__builtin_amdgcn_readfirstlane(sh.before);
  }
  for (uint64_t pos = start; pos < end;) {
    const int tiles = tiles_of(a, b), places = places_of(tiles);
    const uint64_t at = pos - before;   // within the request
    if (at >= (uint64_t)places * items) {
      before += (uint64_t)places * items;
      ++b;
      continue;
    }
    const int i = (int)(at / (uint32_t)places), tile0 = (int)(at - (uint64_t)i * places);
    const uint64_t left = end - pos;
    const int stop = (uint64_t)(places - tile0) < left ? places : tile0 + (int)left;
    const int tile1 = stop < tiles ? stop : tiles;
    if (tile0 < tile1) {
      item_heads(args, i, &kvh, &h0, &hn);
      int first, n;
      token_range(a, b, &first, &n);
      const int t1 = first + tile1 * kTileTokens;
      // a part of an item goes to this workgroup's slot: 1 where it begins the
      // item, else 0 (a stretch holds at most one of each)
      float* slot = tile0 == 0 && tile1 == tiles
                        ? nullptr
                        : args.partial + (2 * (int64_t)blockIdx.x + (tile0 == 0)) * args.slot_floats;
      if (tile0 == 0 && tid == 0) {
        const uint32_t last = tile1 == tiles ? blockIdx.x : shares.holder(pos + tiles - 1);
        args.parts[(int64_t)b * items + i] = blockIdx.x << 16 | (last - blockIdx.x);
      }
      attend<DT, E4M3, KS, FULL>(args, sh, sq, so, b, kvh, h0, hn, first + tile0 * kTileTokens,
                                 t1 < n ? t1 : n, n - first, slot);
    }
    pos += stop - tile0;
  }
  for (int x = (int)blockIdx.x; x < a.batch; x += (int)gridDim.x) {
    if (x == (int)blockIdx.x ? !empty : tiles_of(a, x) != 0) continue;
    uint32_t* out = static_cast<uint32_t*>(a.out) + (int64_t)x * a.heads * (a.dim / 2);
    for (int j = tid; j < a.heads * (a.dim / 2); j += kThreads) out[j] = 0;
    for (int j = tid; j < items; j += kThreads) args.parts[(int64_t)x * items + j] = 0;
  }
}

// Joins the parts of the items that several workgroups shared.  One workgroup
// per (head, request): dim / 4 lanes take a part, four elements each, so that
// all parts load at once, and each lane set keeps a running maximum and sum.
// 8 x 96 parts take 6 us (16 when every wave walked the parts in turn), and 4096
// items of one to three 5 us.  Latency: two dependent loads and a launch; finding
// the maximum first measured no better.
template <int DT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void paged_attention_join_kernel(const AttnArgs args,
                                                                          const float* v_scale) {
  // of each set of lanes, of which there are 16 * WAVES at most (dim 16)
  __shared__ floatx4 sums[64 * WAVES];
  __shared__ float top_of[16 * WAVES], weight_of[16 * WAVES];
  const PagedAttention& a = args.a;
  const int b = (int)(blockIdx.x / a.heads), head = (int)blockIdx.x - b * a.heads, D = a.dim;
  const int items = a.kv_heads * args.chunks;
  const int per = a.heads / a.kv_heads, kvh = head / per, in_kv = head - kvh * per;
  const int i = kvh * args.chunks + in_kv / args.group, h = in_kv % args.group;
  const uint32_t info = args.parts[(int64_t)b * items + i];
  const int count = (int)(info & 0xffff) + 1, w0 = (int)(info >> 16);
  if (count == 1) return;   // one workgroup had all of it, or there was nothing
  const int lanes = D / 4, sets = 64 * WAVES / lanes;
  const int set = (int)threadIdx.x / lanes, e = (int)threadIdx.x - set * lanes;
  float top = -INFINITY, sum = 0.f;
  floatx4 o = {0.f, 0.f, 0.f, 0.f};
  constexpr int kAtOnce = 4;
  for (int p = set; p < count && set < sets; p += kAtOnce * sets) {
    float pm[kAtOnce], pl[kAtOnce];
    floatx4 po[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int q = p + j * sets < count ? p + j * sets : p;
      const float* x = args.partial + (2 * (int64_t)(w0 + q) + (q == 0)) * args.slot_floats;
      pm[j] = x[h];
      pl[j] = x[kMaxGroup + h];
      po[j] = *reinterpret_cast<const floatx4*>(x + kSlotHead + h * D + 4 * e);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (p + j * sets >= count) break;
      const float y = fmaxf(top, pm[j]), base = y == -INFINITY ? 0.f : y;
      const float f = __builtin_amdgcn_exp2f(top - base), g = __builtin_amdgcn_exp2f(pm[j] - base);
      sum = sum * f + pl[j] * g;
      o = o * f + po[j] * g;
      top = y;
    }
  }
  if (set < sets) {
    sums[threadIdx.x] = o;
    if (e == 0) {
      top_of[set] = top;
      weight_of[set] = sum;
    }
  }
  __syncthreads();
  if (set > 0) return;
  const int filled = count < sets ? count : sets;
  for (int x = 1; x < filled; ++x) {
    const float m = top_of[x], y = fmaxf(top, m), base = y == -INFINITY ? 0.f : y;
    const float f = __builtin_amdgcn_exp2f(top - base), g = __builtin_amdgcn_exp2f(m - base);
    sum = sum * f + weight_of[x] * g;
    o = o * f + sums[x * lanes + e] * g;
    top = y;
  }
  // A part that is infinite weighs more than 0, whatever its factor came to.
  if (__builtin_expect(!(fabsf(o[0]) < INFINITY && fabsf(o[1]) < INFINITY && fabsf(o[2]) < INFINITY &&
                         fabsf(o[3]) < INFINITY), 0)) {
    floatx4 odd = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int p = 0; p < count; ++p) {
      const float* x = args.partial + (2 * (int64_t)(w0 + p) + (p == 0)) * args.slot_floats + kSlotHead +
                       h * D + 4 * e;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!(fabsf(x[j]) < INFINITY)) odd[j] += x[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (odd[j] != 0.f) o[j] = odd[j];
  }
  const float vs = v_scale ? v_scale[kvh] : 1.0f;
  uint16_t* out = static_cast<uint16_t*>(a.out) + ((int64_t)b * a.heads + head) * D + 4 * e;
#pragma unroll
  for (int j = 0; j < 4; ++j) out[j] = to_bits<DT>(sum == 0.f ? 0.f : o[j] / sum * vs);
}

// ---- host side ---------------------------------------------------------------

constexpr int kCus = 256;
constexpr int kMaxGroups = 4 * kCus;
// One item per workgroup, and no second launch, up to that many elements of a
// kv head's keys.  One CU reads 40 to 60 GB/s however many waves ask (four and
// eight take the same time), which makes 768 tokens of 128 elements 10.8 us
// (bf16) or 9.7 us (e4m3); shared out they take 12.0 and 11.6 us, the join's
// launch included.  At 2048 tokens it is 24.6 against 12.9 us.  Other sizes, one
// request of 8 kv heads each: 1024 tokens of 64 elements 9.1 and 10.8, 256 of 256
// elements 10.4 and 14.9; 16 requests of 768 x 128 16.2 and 19.5.  The rule goes
// by max_len, so a caller that passes the most it serves shares short requests
// out too: 204 tokens 11.0 us with a max_len of 8192, 6.3 with their own.
constexpr int64_t kOneItemElements = 768 * 128;

struct Shares {
  int group, chunks, groups;
  int64_t slot_floats;
};

Shares shares(int64_t heads, int64_t kv_heads, int64_t dim, int64_t max_len, int64_t window) {
  Shares s{};
  const int64_t per = heads / kv_heads;
  s.chunks = (int)cdiv(per, kMaxGroup);
  s.group = s.chunks > 0 ? (int)cdiv(per, s.chunks) : 1;
  s.slot_floats = kSlotHead + s.group * dim;
  const int64_t span = window > 0 && window < max_len ? window : max_len;
  if (span * dim > kOneItemElements) s.groups = kMaxGroups;
  return s;
}

int64_t parts_bytes(int64_t batch, int64_t kv_heads, const Shares& s) {
  return cdiv(4 * batch * kv_heads * s.chunks, 16) * 16;
}

template <int DT, int WAVES>
void launch_join(const AttnArgs& args, const float* v_scale, hipStream_t stream) {
  hipLaunchKernelGGL((paged_attention_join_kernel<DT, WAVES>),
                     dim3((unsigned)((int64_t)args.a.batch * args.a.heads)), dim3(64 * WAVES), 0,
                     stream, args, v_scale);
}

// As many waves as let all workgroups run at once (32 waves a CU), 8 at most
// (16 measured no better): few items may have a hundred parts each, many have
// few.  4096 items: 68.5 us with four waves, 66.5 with two, attention included;
// 1280 with up to 60 parts 27.7 with four, 28.9 with two.
template <int DT>
void launch_join(const AttnArgs& args, const float* v_scale, hipStream_t stream) {
  const int64_t pairs = (int64_t)args.a.batch * args.a.heads;
  if (pairs <= 4 * kCus)
    launch_join<DT, 8>(args, v_scale, stream);
  else if (pairs <= 8 * kCus)
    launch_join<DT, 4>(args, v_scale, stream);
  else
    launch_join<DT, 2>(args, v_scale, stream);
}

template <int DT, bool E4M3, int KS, bool FULL>
hipError_t launch_main(AttnArgs* args, hipStream_t stream) {
  if (args->groups > 0) args->groups = kCus * Attn<DT, E4M3, KS, FULL>::kResident;
  const PagedAttention& a = args->a;
  const dim3 grid(args->groups > 0 ? (unsigned)args->groups
                                   : (unsigned)((int64_t)a.batch * a.kv_heads * args->chunks));
  hipLaunchKernelGGL((paged_attention_kernel<DT, E4M3, KS, FULL>), grid, dim3(64 * kAttnWaves), 0, stream,
                     *args);
  return hipGetLastError();
}

template <int DT, bool E4M3, int KS>
hipError_t launch_full(AttnArgs* args, hipStream_t stream) {
  // whole rows, each read by one item (see kOnce)
  return args->a.dim == 32 * KS && args->chunks == 1
             ? launch_main<DT, E4M3, KS, true>(args, stream)
             : launch_main<DT, E4M3, KS, false>(args, stream);
}

template <int DT, bool E4M3>
hipError_t launch_ks(AttnArgs* args, hipStream_t stream) {
  const int steps = (int)cdiv(args->a.dim, 32);
  if (steps <= 2) return launch_full<DT, E4M3, 2>(args, stream);
  if constexpr (!E4M3)   // e4m3 takes its steps in twos
    if (steps <= 3) return launch_full<DT, E4M3, 3>(args, stream);
  if (steps <= 4) return launch_full<DT, E4M3, 4>(args, stream);
  if (steps <= 6) return launch_full<DT, E4M3, 6>(args, stream);
  return launch_full<DT, E4M3, 8>(args, stream);
}

}  // namespace

int64_t paged_attention_workspace(int64_t batch, int64_t heads, int64_t kv_heads, int64_t dim,
                                  int64_t max_len, int64_t window) {
  if (batch == 0 || heads == 0) return 0;
  const Shares s = shares(heads, kv_heads, dim, max_len, window);
  if (s.groups == 0) return 0;
  return parts_bytes(batch, kv_heads, s) + 2 * s.groups * s.slot_floats * 4;
}

hipError_t launch_paged_attention(int dtype, int cache_dtype, const PagedAttention& a,
                                  hipStream_t stream) {
  AttnArgs args{};
  args.a = a;
  const Shares s = shares(a.heads, a.kv_heads, a.dim, a.max_len, a.window);
  args.group = s.group;
  args.chunks = s.chunks;
  args.groups = s.groups;
  args.slot_floats = (int)s.slot_floats;
  args.parts = static_cast<uint32_t*>(a.workspace);
  args.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) +
                                          parts_bytes(a.batch, a.kv_heads, s));
  // 2^(s-1) < P <= 2^s: ceil(2^(31+s) / P) fits 32 bits, and n * it >> (31 + s) is n / P for
  // every n < 2^31 (the excess over n / P stays below 1 / P)
  uint32_t shift = 0;
  while (((uint64_t)1 << shift) < (uint64_t)a.pool.page_size) ++shift;
  args.page_shift = shift;
  args.page_magic = (uint32_t)((((uint64_t)1 << (31 + shift)) + a.pool.page_size - 1) /
                               a.pool.page_size);
  const bool e4m3 = cache_dtype == 3;
  const hipError_t e = dtype == 1 ? (e4m3 ? launch_ks<1, true>(&args, stream)
                                          : launch_ks<1, false>(&args, stream))
                                  : (e4m3 ? launch_ks<2, true>(&args, stream)
                                          : launch_ks<2, false>(&args, stream));
  if (e != hipSuccess || s.groups == 0) return e;
  const float* v_scale = e4m3 ? a.v_scale : nullptr;
  dtype == 1 ? launch_join<1>(args, v_scale, stream) : launch_join<2>(args, v_scale, stream);
  return hipGetLastError();
}

}  // namespace qgemm
