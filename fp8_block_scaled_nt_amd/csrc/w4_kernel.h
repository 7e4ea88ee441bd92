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
// The weights are read once, half a byte each, and serve at most 64 rows of a:
// the product is bound by HBM on all but the smallest sizes, so the kernel is
// laid out around its loads.  A wave owns 16 NT weight rows and a run of K in
// units of 128; lane l loads 16 bytes (32 codes) of row l % 16 at K offset
// 32 (l / 16), so one instruction takes 64 contiguous bytes of 16 rows, and
// the same registers are the B operand of v_mfma_f32_16x16x32_bf16 once their
// nibbles are widened.  The waves of a workgroup split K and add their fp32
// sums in LDS in wave order: one launch, no scratch memory, and the same bits
// on every call.
//
// Widening is exact.  e2m1 codes go through the hardware conversion to bf16;
// integer codes become bf16 128 + c by setting bits under the exponent of 128
// (bf16 has 7 fraction bits), and the 128 is taken out again with the zero
// point: sum (128 + c) a - (128 + z) sum a, both sums in fp32 from the matrix
// cores.  The scale multiplies the fp32 sum of its group, so no weight is
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
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
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
};

// One unit (128 of K) of a wave's operands, as loaded.
template <int GROUP, int MT, int NT>
struct W4Unit {
  static constexpr int kGroups = 128 / GROUP;
  v4u w[NT];
  v4u a[MT][4];
  uint16_t s[NT][kGroups];
  uint8_t z[NT][kGroups];
};

template <int FMT, int GROUP, int MT, int NT>
__device__ __forceinline__ void w4_load(const W4Params& p, int n0, int m0, int u, W4Unit<GROUP, MT, NT>& t) {
  constexpr int kG = W4Unit<GROUP, MT, NT>::kGroups;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int k0 = u * 128;
  // quarters of the unit inside K (always four when groups are 128 wide)
  const int quarters = GROUP == 128 ? 4 : min(4, (p.k - k0) / 32);
  const int groups = quarters * 32 / GROUP;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const size_t row = (size_t)min(n0 + i * 16 + r, p.n - 1);
    t.w[i] = v4u{0, 0, 0, 0};
    if (q < quarters) t.w[i] = *(const v4u*)(p.codes + row * (size_t)(p.k / 2) + k0 / 2 + q * 16);
    const size_t g0 = row * (size_t)(p.k / GROUP) + (size_t)u * kG;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const int gg = min(g, groups - 1);
      t.s[i][g] = p.scales[g0 + gg];
      if constexpr (FMT == kW4U4) t.z[i][g] = p.zeros[g0 + gg];
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const uint16_t* row = p.a + (size_t)min(m0 + i * 16 + r, p.m - 1) * p.k + k0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int jj = min(j, quarters - 1);
      t.a[i][j] = *(const v4u*)(row + (GROUP == 128 ? q * 32 + j * 8 : jj * 32 + q * 8));
    }
  }
}

template <int FMT, int GROUP, int MT, int NT>
__device__ __forceinline__ void w4_accumulate(const W4Params& p, int u, W4Unit<GROUP, MT, NT>& t,
                                              v4f (&acc)[MT][NT]) {
  constexpr int kG = W4Unit<GROUP, MT, NT>::kGroups;
  constexpr int kPer = 4 / kG;  // quarters of a group
  const int groups = GROUP == 128 ? 1 : min(4, (p.k - u * 128) / 32) / kPer;
  if constexpr (GROUP < 128) {
#pragma unroll
    for (int i = 0; i < NT; ++i) w4_transpose(t.w[i]);
  }
  const v4u one4 = v4u{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const v8bf ones = __builtin_bit_cast(v8bf, one4);
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    if (GROUP < 128 && g >= groups) break;
    v8bf b[NT][kPer];
    float s[NT], z[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) b[i][j] = w4_widen<FMT>(t.w[i][g * kPer + j]);
      s[i] = bf16_to_f32(t.s[i][g]);
      z[i] = FMT == kW4U4 ? 128.f + (float)t.z[i][g] : 0.f;
    }
#pragma unroll
    for (int mi = 0; mi < MT; ++mi) {
      v8bf a[kPer];
      v4f sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        a[j] = w4_order_a<FMT>(t.a[mi][g * kPer + j]);
        if constexpr (FMT == kW4U4) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], ones, sum, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        v4f part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kPer; ++j) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], b[i][j], part, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (FMT == kW4U4) part[e] -= z[i] * sum[e];
          acc[mi][i][e] += s[i] * part[e];
        }
      }
    }
  }
}

template <int FMT, int GROUP, int MT, int NT, int WAVES, int DEPTH>
__global__ __launch_bounds__(WAVES * 64) void w4_gemm_kernel(W4Params p) {
  __shared__ v4f red[WAVES][MT * NT][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int n0 = blockIdx.x * 16 * NT, m0 = blockIdx.y * 16 * MT;
  const int units = (p.k + 127) / 128;
  const int u1 = (int)((long long)units * (wave + 1) / WAVES);
  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  int u = (int)((long long)units * wave / WAVES);
  for (; u + DEPTH <= u1; u += DEPTH) {
    W4Unit<GROUP, MT, NT> t[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) w4_load<FMT>(p, n0, m0, u + i, t[i]);
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) w4_accumulate<FMT>(p, u + i, t[i], acc);
  }
  for (; u < u1; ++u) {
    W4Unit<GROUP, MT, NT> t;
    w4_load<FMT>(p, n0, m0, u, t);
    w4_accumulate<FMT>(p, u, t, acc);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  for (int e = threadIdx.x; e < MT * NT * 64; e += WAVES * 64) {
    const int tile = e >> 6, l = e & 63;
    v4f v = red[0][tile][l];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += red[w][tile][l];
    const int row = m0 + (tile / NT) * 16 + (l >> 4) * 4;
    const int col = n0 + (tile % NT) * 16 + (l & 15);
    if (col >= p.n) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row + i < p.m) p.d[(size_t)(row + i) * p.n + col] = f32_to_bf16(v[i]);
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
  const float sc = bf16_to_f32(sb);
  uint32_t c = 0;
  float z = 0.f;
  if constexpr (FMT == kW4E2m1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c |= e2m1_code(v[e] / sc) << (4 * e);
  } else {
    z = fminf(rintf(-lo / sc), 15.f);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      c |= (uint32_t)(int)fminf(fmaxf(rintf(v[e] / sc) + z, 0.f), 15.f) << (4 * e);
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
