// 4-bit weights with group scales: the product of a few bf16 rows with them,
// and their way into that form and back.
//
//   d[m][n] = bf16( sum over groups g of K of
//                   s[n][g] * (sum_{k in g} c[n][k] * a[m][k] - z[n][g] * sum_{k in g} a[m][k]) )
//
// c is the e2m1 value of a code (z = 0) or the code 0..15 itself with an
// integer zero point z per row and group.  Codes are packed two per byte along
// K (element 2i in the low nibble), scales are bf16, groups are 32, 64 or 128
// wide.
//
// Weights are half a byte each and serve few rows of a, so the kernels are laid
// out around their loads.  K is walked in units of 128.  A wave takes 16 weight
// rows of a unit with one load of 16 bytes (32 codes) a lane, four lanes to a
// row; the codes change lanes in LDS, and are the B operand of
// v_mfma_f32_16x16x32_bf16 once their nibbles are widened.  Two kernels, both one
// launch with the same bits on every call:
//
//   w4_rows_kernel: 16 weight rows by up to 16 rows of a.  The waves of a
//     workgroup split K and add their fp32 sums in LDS in wave order, without
//     scratch memory.  More rows of a read the weights again for every 16.
//   w4_tile_kernel: 128 weight rows by 32 or 64 rows of a, K in splits that are
//     added in split order by way of the stream's workspace.
//
// Widening is exact.  e2m1 codes go through the hardware conversion to bf16;
// integer codes become bf16 128 + c by setting bits under the exponent of 128
// (bf16 has 7 fraction bits), and the 128 is taken out again with the zero
// point: sum (128 + c) a - (128 + z) sum a, both sums in fp32 from the matrix
// cores.  They hold terms of up to 143 |a|, where (c - z) a has up to 15 |a|: an
// fp32 rounding is then up to 2^-17 of the group's sum |a| (times the scale), and
// the output is bf16.  The scale multiplies the fp32 sum of its group, so no weight is
// rounded to bf16 after scaling.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_kernel.h"
#include "quant_kernel.h"

namespace dg {

enum W4Format { kW4E2m1 = 0, kW4U4 = 1 };

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_to_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }

// fp32 -> bf16, nearest even (v_cvt_pk_bf16_f32); NaN stays NaN.
__device__ __forceinline__ uint32_t pack2_bf16(float a, float b) {
  v2bf r;
  r[0] = (__bf16)a;
  r[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint16_t f32_to_bf16(float a) { return (uint16_t)(pack2_bf16(a, a) & 0xFFFFu); }

// Eight codes of one dword as the eight bf16 of a B fragment.  e2m1: in their
// order; u4: 128 + c in the order 0 4 1 5 2 6 3 7 (w4_order_a puts a's values
// in the same order; a dot product does not mind).
template <int FMT>
__device__ __forceinline__ v8bf w4_widen(uint32_t w) {
  v4u r;
  if constexpr (FMT == kW4E2m1) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3));
  } else {
    // in registers, so that mask and bias are one v_and_or_b32
    uint32_t mask = 0x000F000Fu, bias = 0x43004300u;
    asm("" : "+s"(mask));
    asm("" : "+v"(bias));
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = ((w >> (4 * i)) & mask) | bias;
  }
  return __builtin_bit_cast(v8bf, r);
}

template <int FMT>
__device__ __forceinline__ v8bf w4_order_a(v4u x) {
  if constexpr (FMT == kW4U4) {
    v4u r;
    r[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);
    r[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);
    r[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);
    r[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);
    return __builtin_bit_cast(v8bf, r);
  } else {
    return __builtin_bit_cast(v8bf, x);
  }
}

// Transposes a 4 x 4 matrix of dwords held as w[j] in the four 16-lane groups
// of a wave: afterwards lane group i holds in w[j] what group j held in w[i].
// A unit's 32-wide quarters then follow each other from w[0] to w[3], each
// spread over all lanes, and one MFMA covers K of one quarter only.
__device__ __forceinline__ void w4_transpose(v4u& w) {
  v2u a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  v2u b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  v2u c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  v2u d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w[0] = c[0];
  w[1] = c[1];
  w[2] = d[0];
  w[3] = d[1];
}

struct W4Params {
  const uint16_t* a;       // [m][k] bf16
  const uint8_t* codes;    // [n][k/2]
  const uint16_t* scales;  // [n][k/group] bf16
  const uint8_t* zeros;    // [n][k/group], u4 only
  uint16_t* d;             // [m][n] bf16
  int m, n, k;
  float* partial;  // w4_tile_kernel with splits: [tiles][splits] partial tiles
  int* count;      // and their arrival counters, zero between calls
  int per, more;   // units of a split; the first `more` splits have one more (a division less in the kernel)
};

// Quarters (32 of K) of unit u that lie inside K; K is a multiple of 32, and
// WHOLE says of 128.
template <bool WHOLE>
__device__ __forceinline__ int w4_quarters(int k, int u) {
  return WHOLE ? 4 : max(0, min(4, (k - u * 128) / 32));
}

constexpr uint32_t kW4Nowhere = 0x80000000u;  // a byte offset past every buffer here (k is at most 2^23)

// 16 weight rows of a wave, and the way of their codes and scales from memory
// to the lanes that use them.
//
// The matrix instruction wants row l % 16 in lane l.  Loaded that way, no two
// neighbouring lanes read the same cache line, and the vector memory pipe is
// what bounds the kernel (25 us for 1 x 7168 x 16384, 14.0 as it is here,
// 4.3 TB/s).  So lane l loads
// piece l % 4 of row l / 4, four lanes a line, and the codes change lanes in
// LDS of the wave's own (no barrier: a wave's LDS instructions are in order).
// Scales come 64 at a time: four a row, which is 4 / (128 / GROUP) units.
//
// Loads are never under a branch, where the compiler could not count them and
// would wait for all that are in flight: past the last unit, or outside the
// matrix, they go to an offset past the buffer's end, which gives zeros and no
// memory traffic.
template <int FMT, int GROUP, bool WHOLE>
struct W4Rows {
  static constexpr int kG = 128 / GROUP;  // groups of a unit
  static constexpr int kSU = 4 / kG;      // units of a load of scales
  static constexpr int kLds = 64 * 16 + 2 * 64 * 4;

  __amdgpu_buffer_rsrc_t codes, scales, zeros;
  uint32_t at_codes, at_group;  // of this lane's row, in bytes and in groups
  int groups, k;

  __device__ __forceinline__ W4Rows(const W4Params& p, int n0) {
    k = p.k;
    groups = p.k / GROUP;
    const int base = min(n0, p.n - 1), rows = n0 < p.n ? min(p.n - n0, 16) : 0, r = (threadIdx.x & 63) >> 2;
    codes = __builtin_amdgcn_make_buffer_rsrc((void*)(p.codes + (size_t)base * (k / 2)), 0, rows * (k / 2), kBufferRsrcWord3);
    scales = __builtin_amdgcn_make_buffer_rsrc((void*)(p.scales + (size_t)base * groups), 0, rows * groups * 2, kBufferRsrcWord3);
    zeros = scales;
    if constexpr (FMT == kW4U4)
      zeros = __builtin_amdgcn_make_buffer_rsrc((void*)(p.zeros + (size_t)base * groups), 0, rows * groups, kBufferRsrcWord3);
    at_codes = (uint32_t)r * (uint32_t)(k / 2) + (threadIdx.x & 3) * 16;
    at_group = (uint32_t)r * (uint32_t)groups;
  }

  // This lane's piece of unit u of `units`.
  __device__ __forceinline__ v4u load(int u, int units) const {
    const bool in = u < units && (WHOLE || (int)(threadIdx.x & 3) < w4_quarters<WHOLE>(k, u));
    const auto w = __builtin_amdgcn_raw_buffer_load_b128(codes, in ? at_codes + u * 64 : kW4Nowhere, 0, 0);
    return __builtin_bit_cast(v4u, w);
  }
  // This lane's scale and zero of units u, u + step, ..
  __device__ __forceinline__ void load_scales(int u, int step, uint32_t& s, uint32_t& z) const {
    const int part = threadIdx.x & 3, g = (u + part / kG * step) * kG + part % kG;
    const uint32_t at = g < groups ? at_group + g : kW4Nowhere / 2;
    s = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(scales, at * 2, 0, 0);
    if constexpr (FMT == kW4U4) z = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(zeros, at, 0, 0);
  }
  // Into the wave's LDS, and out of it for row l % 16: quarter l / 16 of the
  // codes; the scales (and what zero points subtract: 128 + z).
  static __device__ __forceinline__ void put(uint8_t* lds, v4u w) {
    const int r = (threadIdx.x & 63) >> 2, part = threadIdx.x & 3;
    ((v4u*)lds)[r * 4 + (part ^ ((r >> 2) & 3))] = w;
  }
  static __device__ __forceinline__ v4u get(const uint8_t* lds) {
    const int r = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
    return ((const v4u*)lds)[r * 4 + (q ^ ((r >> 2) & 3))];
  }
  static __device__ __forceinline__ void put_scales(uint8_t* lds, uint32_t s, uint32_t z) {
    ((uint32_t*)(lds + 1024))[threadIdx.x & 63] = s << 16;
    if constexpr (FMT == kW4U4) ((float*)(lds + 1280))[threadIdx.x & 63] = (float)(z + 128u);
  }
  static __device__ __forceinline__ void get_scales(const uint8_t* lds, v4f& s, v4f& z) {
    s = ((const v4f*)(lds + 1024))[threadIdx.x & 15];
    if constexpr (FMT == kW4U4) z = ((const v4f*)(lds + 1280))[threadIdx.x & 15];
  }
};

// Adds a unit's products with MT tiles of 16 rows of A to acc (lane l: weight
// row l % 16, row 4 (l / 16) + e of A for e < E).  w, s and z are the unit's
// codes, scales and zeros as W4Rows gives them, `first` the unit's first scale
// among the four.  load_a(t, j) gives tile t's fragment for quarter-wide
// product j, in the order that w4_widen leaves K in.
template <int FMT, int GROUP, int MT, int NT, int E, bool WHOLE, class LoadA>
__device__ __forceinline__ void w4_accumulate(int k, int u, v4u (&w)[NT], const v4f (&s)[NT], const v4f (&z)[NT],
                                              int first, float (&acc)[MT][NT][E], LoadA load_a) {
  constexpr int kG = 128 / GROUP;
  constexpr int kPer = 4 / kG;  // products of a group
  const int groups = w4_quarters<WHOLE>(k, u) / kPer;
  if constexpr (GROUP < 128) {
#pragma unroll
    for (int i = 0; i < NT; ++i) w4_transpose(w[i]);
  }
  const v4u one4 = v4u{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const v8bf ones = __builtin_bit_cast(v8bf, one4);
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    if (!WHOLE && g >= groups) break;
    v8bf b[NT][kPer];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t eight = w[i][g * kPer + j];
        b[i][j] = w4_widen<FMT>(eight);
      }
    // all tiles side by side, and two chains of products where there is but
    // one: a product waits some 30 cycles for the one before it in its chain
    constexpr int kChains = MT * NT == 1 && kPer > 1 ? 2 : 1;
    v4f part[kChains][MT][NT], sum[kChains][MT];
#pragma unroll
    for (int c = 0; c < kChains; ++c)
#pragma unroll
      for (int mi = 0; mi < MT; ++mi) {
        sum[c][mi] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NT; ++i) part[c][mi][i] = v4f{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
#pragma unroll
      for (int mi = 0; mi < MT; ++mi) {
        const int c = j % kChains;
        const v8bf a = load_a(mi, g * kPer + j);
        if constexpr (FMT == kW4U4) sum[c][mi] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, ones, sum[c][mi], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          part[c][mi][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[i][j], part[c][mi][i], 0, 0, 0);
      }
#pragma unroll
    for (int mi = 0; mi < MT; ++mi)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float x = part[0][mi][i][e], y = sum[0][mi][e];
          if constexpr (kChains == 2) {
            x += part[1][mi][i][e];
            y += sum[1][mi][e];
          }
          if constexpr (FMT == kW4U4) x -= z[i][first + g] * y;
          acc[mi][i][e] += s[i][first + g] * x;
        }
  }
}

// Where 16-byte piece `part` of a unit of row `row` of a lies in LDS: pieces in
// the order in which products take them (product j takes piece 4 q + j in lane
// group q where a group is the whole unit, else 4 j + q), and rows apart by an
// exclusive or, so that the 16 rows that are read together, and the lane
// groups, fall on different banks.
template <int GROUP>
__device__ __forceinline__ int w4_slot_a(int row, int part) {
  return (GROUP == 128 ? (part & 3) * 4 + (part >> 2) : part) ^ (row & 15);
}

// Few rows of a: a workgroup takes up to 16 of them and 16 weight rows, and its
// 4 or 8 waves every so many-th unit of K each.  A wave keeps kW4Depth units of weights in
// flight and refills a unit's registers as soon as it is used.
//
// a is the same for all workgroups and comes from L2, but a fragment of it is
// 16 rows wide whatever m is.  So each wave loads U units of ROWS rows
// densely, a chunk ahead, and turns them into fragments through its LDS.
// Row i of a becomes row 4 (i % 4) + i / 4 of A: of the four sums that a lane
// has of every product, only the first E are then of rows below m, and only
// these are scaled.
//
// One copy of the four units' code, for every number of units: most waves pass
// through once or twice, and what they do not find in the instruction cache
// costs them more than a branch a unit (with separate code for the last units
// 7.4 us for 5 x 1001 x 1056, without 4.2).
constexpr int kW4Depth = 4;
template <int FMT, int GROUP, int U, int ROWS, bool WHOLE>
__global__ __launch_bounds__(512, 4) void w4_rows_kernel(W4Params p) {
  using Rows = W4Rows<FMT, GROUP, WHOLE>;
  constexpr int E = ROWS / 4, kLoads = U * ROWS / 4, kChunk = U * ROWS * 256;
  extern __shared__ __align__(16) uint8_t lds[];  // of each wave: a chunk of a, then Rows::kLds; later the waves' sums
  const int waves = blockDim.x >> 6, waves_log2 = waves == 8 ? 3 : 2;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * ROWS, m = min(p.m - m0, ROWS);
  const int units = (p.k + 127) / 128;
  const int count = (units - wave + waves - 1) >> waves_log2;  // this wave's units: wave, wave + waves, ..
  v4u* mine = (v4u*)(lds + wave * (kChunk + Rows::kLds));
  uint8_t* mine_w = (uint8_t*)mine + kChunk;
  const Rows rows(p, n0);
  const __amdgpu_buffer_rsrc_t src_a =
      __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + (size_t)m0 * p.k), 0, m * p.k * 2, kBufferRsrcWord3);

  // chunk of a from the wave's unit number u on: load i brings piece `part` of
  // unit number u + v of row row_of(i), and zeros for rows past m
  v4u held[kLoads];
  const int v = (lane >> 4) & (U - 1), part = lane & 15;
  auto row_of = [&](int i) { return i * (4 / U) + lane / (16 * U); };
  auto fetch = [&](int u, int i) {
    const int unit = wave + (u + v) * waves;
    const bool in = row_of(i) < m && unit < units && (WHOLE || part < 4 * w4_quarters<WHOLE>(p.k, unit));
    const uint32_t at = (uint32_t)row_of(i) * (uint32_t)p.k + unit * 128 + part * 8;
    const auto x = __builtin_amdgcn_raw_buffer_load_b128(src_a, in ? at * 2 : kW4Nowhere, 0, 0);
    held[i] = __builtin_bit_cast(v4u, x);
  };
  auto put = [&](int i) {
    mine[(row_of(i) * U + v) * 16 + w4_slot_a<GROUP>(row_of(i), part)] = __builtin_bit_cast(v4u, w4_order_a<FMT>(held[i]));
  };
  const int row = (r >> 2) + 4 * (r & 3) & (ROWS - 1);
  float acc[1][1][E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[0][0][e] = 0.f;

  v4u t[kW4Depth];
  uint32_t s[kW4Depth / Rows::kSU], z[kW4Depth / Rows::kSU];
#pragma unroll
  for (int i = 0; i < kW4Depth; ++i) {
    t[i] = rows.load(wave + i * waves, units);
    if (i % Rows::kSU == 0) rows.load_scales(wave + i * waves, waves, s[i / Rows::kSU], z[i / Rows::kSU]);
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) fetch(0, i);
  v4f s4[1], z4[1];
#pragma unroll 1
  for (int u = 0; u < count; u += kW4Depth) {
#pragma unroll
    for (int i = 0; i < kW4Depth; ++i) {
      const int next = wave + (u + i + kW4Depth) * waves;
      Rows::put(mine_w, t[i]);
      t[i] = rows.load(next, units);
      if (i % Rows::kSU == 0) {
        Rows::put_scales(mine_w, s[i / Rows::kSU], z[i / Rows::kSU]);
        rows.load_scales(next, waves, s[i / Rows::kSU], z[i / Rows::kSU]);
        Rows::get_scales(mine_w, s4[0], z4[0]);
      }
      if (i % U == 0) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          put(j);
          fetch(u + i + U, j);
        }
      }
      v4u w[1] = {Rows::get(mine_w)};
      w4_accumulate<FMT, GROUP, 1, 1, E, WHOLE>(p.k, wave + (u + i) * waves, w, s4, z4, i % Rows::kSU * Rows::kG, acc,
                                                [&](int, int j) {
        return __builtin_bit_cast(v8bf, mine[(row * U + i % U) * 16 + ((j * 4 + q) ^ row)]);
      });
      __builtin_amdgcn_sched_barrier(0);  // a unit at a time: mixing units only takes registers
      if (u + i + 1 >= count) goto done;
    }
  }
done:
  __syncthreads();
  float* red = (float*)lds;  // [waves][E][64]
#pragma unroll
  for (int e = 0; e < E; ++e) red[(wave * E + e) * 64 + lane] = acc[0][0][e];
  __syncthreads();
  const int e = threadIdx.x >> 6;  // a wave for each of the E rows of a lane group
  if (e >= E) return;
  float sum = red[e * 64 + lane];
#pragma unroll 1
  for (int w = 1; w < waves; ++w) sum += red[(w * E + e) * 64 + lane];
  const int out = q + 4 * e, col = n0 + r;
  if (out < m && col < p.n) p.d[(size_t)(m0 + out) * p.n + col] = f32_to_bf16(sum);
}
// LDS of a workgroup
template <int FMT, int GROUP, int U, int ROWS, bool WHOLE>
constexpr int w4_rows_smem(int waves) {
  return waves * (U * ROWS * 256 + W4Rows<FMT, GROUP, WHOLE>::kLds);
}

// Many rows of a: a workgroup of four waves takes 16 MT rows and 128
// weight rows, 32 a wave, over one split of K.  The unit of a that all four
// waves multiply with goes through LDS, in two buffers, fetched two units
// ahead; each wave brings its own weights, kAhead units ahead.  Splits meet in
// the stream's workspace: partial tiles are stored and loaded at agent scope
// (SC1), each thread waits for its stores, a barrier and a relaxed counter
// follow, and the last of a tile's workgroups adds all of them in split order.
template <int FMT, int GROUP, int MT, bool WHOLE>
__global__ __launch_bounds__(256, 2) void w4_tile_kernel(W4Params p) {
  using Rows = W4Rows<FMT, GROUP, WHOLE>;
  constexpr int NT = 2, kAhead = 4, kTile = MT * NT * 4 * 64 * 4;  // floats of a workgroup's tile
  __shared__ v4u s_a[2][16 * MT * 16];
  __shared__ __align__(16) uint8_t s_w[4][NT][Rows::kLds];
  __shared__ int s_last;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, q = lane >> 4;
  const int n0 = blockIdx.x * 128 + wave * 32, m0 = blockIdx.z * 16 * MT;
  const int split = blockIdx.y, splits = gridDim.y;
  const int u0 = split * p.per + min(split, p.more), u1 = u0 + p.per + (split < p.more);
  const Rows rows[NT] = {Rows(p, n0), Rows(p, n0 + 16)};

  v4u held[2][MT];
  auto fetch_a = [&](int u, int set) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int c = tid + 256 * i, row = min(m0 + c / 16, p.m - 1), part = c % 16;
      const int inside = WHOLE ? part : min(part, 4 * w4_quarters<WHOLE>(p.k, u) - 1);
      held[set][i] = *(const v4u*)(p.a + (size_t)row * p.k + (size_t)u * 128 + inside * 8);
    }
  };
  auto put_a = [&](int buf, int set) {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int c = tid + 256 * i, row = c / 16, part = c % 16;
      s_a[buf][row * 16 + w4_slot_a<GROUP>(row, part)] = __builtin_bit_cast(v4u, w4_order_a<FMT>(held[set][i]));
    }
  };
  v4u t[kAhead][NT];
  uint32_t s[kAhead / Rows::kSU][NT], z[kAhead / Rows::kSU][NT];
  float acc[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
  // past the split's end its last unit of a is loaded again, and not used
  fetch_a(u0, 0);
  fetch_a(min(u0 + 1, u1 - 1), 1);
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      t[i][j] = rows[j].load(u0 + i, u1);
      if (i % Rows::kSU == 0) rows[j].load_scales(u0 + i, 1, s[i / Rows::kSU][j], z[i / Rows::kSU][j]);
    }
  put_a(0, 0);
  fetch_a(min(u0 + 2, u1 - 1), 0);
  __syncthreads();
  v4f s4[NT], z4[NT];
#pragma unroll 1
  for (int u = u0; u < u1; u += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int buf = i & 1, next = u + i + kAhead;  // kAhead is even
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        Rows::put(s_w[wave][j], t[i][j]);
        t[i][j] = rows[j].load(next, u1);
        if (i % Rows::kSU == 0) {
          Rows::put_scales(s_w[wave][j], s[i / Rows::kSU][j], z[i / Rows::kSU][j]);
          rows[j].load_scales(next, 1, s[i / Rows::kSU][j], z[i / Rows::kSU][j]);
          Rows::get_scales(s_w[wave][j], s4[j], z4[j]);
        }
      }
      put_a(buf ^ 1, buf ^ 1);
      fetch_a(min(u + i + 3, u1 - 1), buf ^ 1);
      v4u w[NT] = {Rows::get(s_w[wave][0]), Rows::get(s_w[wave][1])};
      w4_accumulate<FMT, GROUP, MT, NT, 4, WHOLE>(p.k, u + i, w, s4, z4, i % Rows::kSU * Rows::kG, acc, [&](int mi, int j) {
        return __builtin_bit_cast(v8bf, s_a[buf][(mi * 16 + (lane & 15)) * 16 + ((j * 4 + q) ^ (lane & 15))]);
      });
      __builtin_amdgcn_sched_barrier(0);
      __syncthreads();
      if (u + i + 1 >= u1) goto done;
    }
  }
done:

  if (splits > 1) {
    const int tile = blockIdx.z * gridDim.x + blockIdx.x;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        p.partial + (size_t)tile * splits * kTile, 0, splits * kTile * 4, kBufferRsrcWord3);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v4f{acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]}), rs,
                                               (blockIdx.y * kTile + ((i * NT + j) * 256 + tid) * 4) * 4, 0, kCpolSc1);
    wait_vmem_all();
    __syncthreads();
    if (tid == 0)
      s_last = __hip_atomic_fetch_add(p.count + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == splits - 1;
    __syncthreads();
    if (!s_last) return;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
    // four splits' parts in flight: the loads come from beyond L2, and every
    // round of them costs its latency
    constexpr int kRound = 4;
    for (int s0 = 0; s0 < splits; s0 += kRound) {
      v4f part[kRound][MT][NT];
#pragma unroll
      for (int s = 0; s < kRound; ++s)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            // past the last split the buffer's bounds give zero
            const auto v = __builtin_amdgcn_raw_buffer_load_b128(
                rs, ((s0 + s) * kTile + ((i * NT + j) * 256 + tid) * 4) * 4, 0, kCpolSc1);
            part[s][i][j] = __builtin_bit_cast(v4f, v);
          }
#pragma unroll
      for (int s = 0; s < kRound; ++s)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] += part[s][i][j][e];
    }
    if (tid == 0) __hip_atomic_store(p.count + tile, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next call
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int col = n0 + j * 16 + (lane & 15);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = m0 + i * 16 + q * 4 + e;
        if (row < p.m && col < p.n) p.d[(size_t)row * p.n + col] = f32_to_bf16(acc[i][j][e]);
      }
    }
}

// ---- quantiser and its inverse: streaming passes, bound by HBM

// Eight consecutive values of x (bf16 or fp32) as fp32.
template <bool BF16>
__device__ __forceinline__ void w4_read8(const void* x, size_t at, float (&v)[8]) {
  if constexpr (BF16) {
    const v4u r = *(const v4u*)((const uint16_t*)x + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r[i] << 16);
      v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  } else {
    const float4 lo = *(const float4*)((const float*)x + at), hi = *(const float4*)((const float*)x + at + 4);
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  }
}

// x / s for one s and many x, correctly rounded as one division each would be,
// in three instructions instead of ten: with r = 1 / s correctly rounded, q = x
// r and the exact remainder x - q s, q + r (x - q s) rounds to the quotient
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990; s has 8 significant bits, so it is none of the theorem's
// exceptions).  Remainders that underflow belong to quotients that round to
// the code of zero.
__device__ __forceinline__ float w4_quotient(float x, float s, float r) {
  const float q = x * r;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, x), r, q), x);  // -0 stays -0
}

// A thread holds 8 values of a group, GROUP / 8 neighbouring lanes a group.
//   e2m1: s = bf16(max(amax, 1e-4) / 6), c = e2m1(x / s)
//   u4:   lo = min(x, 0), hi = max(x, 0) over the group, s = bf16(max(hi - lo, 1e-4) / 15),
//         z = min(rint(-lo / s), 15), c = clamp(rint(x / s) + z, 0, 15)
// Codes are taken against the rounded scale, so its rounding costs no accuracy.
template <int FMT, int GROUP, bool BF16>
__global__ __launch_bounds__(256) void w4_quant_kernel(const void* __restrict__ x, uint8_t* __restrict__ codes,
                                                       uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros,
                                                       long long total8) {
  constexpr int kLanes = GROUP / 8;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const bool live = i < total8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live) w4_read8<BF16>(x, (size_t)i * 8, v);
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (FMT == kW4E2m1) {
      hi = fmaxf(hi, fabsf(v[e]));
    } else {
      lo = fminf(lo, v[e]);
      hi = fmaxf(hi, v[e]);
    }
  }
#pragma unroll
  for (int s = kLanes / 2; s >= 1; s >>= 1) {
    hi = fmaxf(hi, __shfl_xor(hi, s, 64));
    if constexpr (FMT == kW4U4) lo = fminf(lo, __shfl_xor(lo, s, 64));
  }
  if (!live) return;
  const uint16_t sb = f32_to_bf16(fmaxf(hi - lo, kAmaxFloor) / (FMT == kW4E2m1 ? kE2m1Max : 15.f));
  const float sc = bf16_to_f32(sb), r = 1.f / sc;
  uint32_t c = 0;
  float z = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = w4_quotient(v[e], sc, r);
  if constexpr (FMT == kW4E2m1) {
    // v_cvt_scalef32_pk_fp4_f32: nearest, ties to even, saturating at 6
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], 1.0f, 3);
  } else {
    z = fminf(rintf(-lo / sc), 15.f);
#pragma unroll
    for (int e = 0; e < 8; ++e) c |= (uint32_t)(int)fminf(fmaxf(rintf(v[e]) + z, 0.f), 15.f) << (4 * e);
  }
  *(uint32_t*)(codes + i * 4) = c;
  if ((threadIdx.x & (kLanes - 1)) == 0) {
    scales[i / kLanes] = sb;
    if constexpr (FMT == kW4U4) zeros[i / kLanes] = (uint8_t)z;
  }
}

// w[n][k] = bf16(s * (c - z)): 8 codes a thread.
template <int FMT, int GROUP>
__global__ __launch_bounds__(256) void w4_dequant_kernel(const uint8_t* __restrict__ codes,
                                                         const uint16_t* __restrict__ scales,
                                                         const uint8_t* __restrict__ zeros, uint16_t* __restrict__ w,
                                                         long long total8) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= total8) return;
  const uint32_t c = *(const uint32_t*)(codes + i * 4);
  const float s = bf16_to_f32(scales[i / (GROUP / 8)]);
  const v8bf wide = w4_widen<FMT>(c);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)wide[e];
  v4u r;
  if constexpr (FMT == kW4E2m1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = pack2_bf16(s * v[2 * e], s * v[2 * e + 1]);
  } else {  // widened as 128 + c in the order 0 4 1 5 2 6 3 7
    const float z = 128.f + (float)zeros[i / (GROUP / 8)];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int a = (2 * e) & 3, hi = (2 * e) >> 2;  // element 2e is wide[2 a + hi]
      r[e] = pack2_bf16(s * (v[2 * a + hi] - z), s * (v[2 * (a + 1) + hi] - z));
    }
  }
  *(v4u*)(w + i * 8) = r;
}

}  // namespace dg
