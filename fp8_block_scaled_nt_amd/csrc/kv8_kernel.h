// A paged key/value cache in 8 bits and the attention that reads it.
//
// The cache holds e4m3 codes in blocks of `block` tokens (16, 32, 64 or 128),
// one fp32 scale for each block and head, keys and values apart:
//
//   k_codes [num_blocks][h_kv][block][d]     v_codes [num_blocks][h_kv][d][block]
//   k_scales, v_scales [num_blocks][h_kv]
//
// A block's tokens of one head lie together.  Keys lie token by token, values
// dimension by dimension: both then are what a matrix instruction takes as its
// A operand in whole 8- and 16-byte pieces, and the attention kernels read
// them from memory straight into registers, without a transpose.
// block_table[i][j] names the block that holds tokens j * block .. of
// sequence i.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_kernel.h"
#include "quant_kernel.h"
#include "w4_kernel.h"

namespace dg {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));

struct Kv8Cache {
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scales;
  float* v_scales;
  const int32_t* table;  // [batch][max_blocks]
  int h_kv, block, block_log2, num_blocks, max_blocks;
};

// The block of sequence `seq` that holds token `token`, or -1 where the table
// has none (past its width, or an entry outside the pool): such tokens are
// neither read nor written.
__device__ __forceinline__ int kv8_page(const Kv8Cache& c, int seq, int token) {
  const int j = token >> c.block_log2;
  if (j < 0 || j >= c.max_blocks) return -1;
  const int page = c.table[(size_t)seq * c.max_blocks + j];
  return page >= 0 && page < c.num_blocks ? page : -1;
}

// New rows of sequence `seq`: [first, first + count) of the packed tokens.
// cu holds batch + 1 running sums; whatever it holds, the range stays inside
// the `total` packed tokens, and count is at most `most`.
__device__ __forceinline__ void kv8_rows(const int32_t* cu, int seq, int total, int most, int* first, int* count) {
  const int lo = min(max(cu[seq], 0), total), hi = min(max(cu[seq + 1], 0), total);
  *first = lo;
  *count = min(max(hi - lo, 0), most);
}

// ---- append

// Smallest power of two s with x <= 448 s, for x >= 1e-4: 448 = 1.75 * 2^8,
// so the exponent of x less 8, one more if the fraction of x passes 1.75.
__device__ __forceinline__ float kv8_scale(float amax) {
  const uint32_t b = __float_as_uint(fmaxf(amax, kAmaxFloor));
  const uint32_t e = (b >> 23) + ((b & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
  return __uint_as_float((e - 8u) << 23);
}

// Four values as e4m3 codes: nearest even, saturated at 448; NaN stays NaN.
__device__ __forceinline__ uint32_t kv8_pack4(float a, float b, float c, float d) {
  auto clip = [](float x) {
    x = x > kE4m3Max ? kE4m3Max : x;
    return x < -kE4m3Max ? -kE4m3Max : x;
  };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(clip(a), clip(b), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(clip(c), clip(d), w, true);
  return (uint32_t)w;
}

// Four codes times `by` (a power of two below one), rounded onto the grid anew.
__device__ __forceinline__ uint32_t kv8_rescale4(uint32_t w, float by) {
  const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return kv8_pack4(lo[0] * by, lo[1] * by, hi[0] * by, hi[1] * by);
}

struct Kv8AppendParams {
  const uint16_t* k;  // bf16 [total][h_kv][d], k_stride elements from token to token
  const uint16_t* v;
  long long k_stride, v_stride;
  Kv8Cache c;
  const int32_t* ctx;  // tokens in the cache before the call, per sequence
  const int32_t* cu;   // running sums of the new tokens, batch + 1 entries
  int total, most;
};

// One workgroup takes one block of one head that gets new tokens, its keys
// (even blockIdx.y) or its values (odd).  It is the only one that touches that
// tile and its scale.
//
//   s' = max(s, smallest power of two with amax(new) <= 448 s), s = 0 for a
//   block without older tokens; new codes e4m3(x / s'); where s' > s the older
//   codes become e4m3(c * s / s').
//
// The scales are powers of two, so dividing by one is exact and growing it
// moves exponents only: codes change beyond their scale only where they fall
// below 2^-6 in the new one, and a cache filled token by token equals one
// filled at once up to those.  amax counts finite values only; infinities
// saturate at 448 s' and NaN is stored as NaN.
//
// The new values are read twice (amax, then codes; the second read comes from
// the caches) rather than kept in registers, which bounds no tile size.
// Values are turned on their way in an LDS tile of codes [d][block].
template <int D>
__global__ __launch_bounds__(256) void kv8_append_kernel(Kv8AppendParams p) {
  constexpr int kPer = D / 8;  // 16-byte pieces of a token's head
  __shared__ float s_max[4];
  __shared__ __align__(16) uint8_t turn[D * (128 + 16)];
  const int seq = blockIdx.z, head = blockIdx.y >> 1;
  const int block = p.c.block, tid = threadIdx.x;
  int first, count;
  kv8_rows(p.cu, seq, p.total, p.most, &first, &count);
  const int ctx = max(p.ctx[seq], 0);
  const int base = ((ctx >> p.c.block_log2) + (int)blockIdx.x) << p.c.block_log2;  // first token of this block
  const long long end = (long long)ctx + count;
  if (base >= end || count == 0) return;
  const int page = kv8_page(p.c, seq, base);
  if (page < 0) return;
  const int old = max(ctx - base, 0);                                  // older tokens of the block
  const int stop = (int)(end - base < block ? end - base : block);     // tokens after the call
  const bool values = (blockIdx.y & 1) != 0;
  const uint16_t* x = values ? p.v : p.k;
  const long long stride = values ? p.v_stride : p.k_stride;
  const uint16_t* src = x + (long long)(first + base + old - ctx) * stride + (long long)head * D;
  const size_t tile = (size_t)page * p.c.h_kv + head;
  float* scale = (values ? p.c.v_scales : p.c.k_scales) + tile;
  uint8_t* codes = (values ? p.c.v_codes : p.c.k_codes) + tile * (size_t)block * D;
  const float was = old > 0 ? *scale : 0.f;

  const int pieces = (stop - old) * kPer;
  float amax = 0.f;
  for (int e = tid; e < pieces; e += 256) {
    float f[8];
    w4_read8<true>(src + (long long)(e / kPer) * stride, (size_t)(e % kPer) * 8, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(f[i]);
      amax = fmaxf(amax, a < __builtin_huge_valf() ? a : 0.f);
    }
  }
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) amax = fmaxf(amax, __shfl_xor(amax, s, 64));
  if ((tid & 63) == 0) s_max[tid >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
  const float now = fmaxf(was, kv8_scale(amax));
  const float inv = 1.f / now;  // a power of two: exact
  const bool grow = old > 0 && now > was;
  const float by = was * inv;
  if (tid == 0) *scale = now;

  const int pitch = block + 16;
  for (int e = tid; e < pieces; e += 256) {
    const int t = e / kPer, c = e % kPer;
    float f[8];
    w4_read8<true>(src + (long long)t * stride, (size_t)c * 8, f);
    const uint32_t lo = kv8_pack4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    const uint32_t hi = kv8_pack4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
    if (!values) {
      *(uint2*)(codes + (size_t)(old + t) * D + c * 8) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        turn[(c * 8 + i) * pitch + old + t] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
  }
  if (!values) {
    if (grow)
      for (int e = tid; e < old * kPer; e += 256) {
        uint2* at = (uint2*)(codes + (size_t)e * 8);
        const uint2 w = *at;
        *at = make_uint2(kv8_rescale4(w.x, by), kv8_rescale4(w.y, by));
      }
    return;
  }
  __syncthreads();
  // 16 tokens of one dimension at a time: new codes from LDS, older ones
  // rounded anew, bytes past the new tokens as they were
  const int lo16 = grow ? 0 : old >> 4, hi16 = (stop + 15) >> 4;
  const int per_row = hi16 - lo16;
  for (int e = tid; e < D * per_row; e += 256) {
    const int row = e / per_row, t0 = (lo16 + e % per_row) * 16;
    v4u* at = (v4u*)(codes + (size_t)row * block + t0);
    const v4u fresh = *(const v4u*)(turn + row * pitch + t0);
    if (t0 >= old && t0 + 16 <= stop) {
      *at = fresh;
      continue;
    }
    const v4u held = *at;
    v4u w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t kept = grow ? kv8_rescale4(held[i], by) : held[i];
      uint32_t r = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int t = t0 + i * 4 + b;
        const uint32_t from = t < old ? kept : (t < stop ? fresh[i] : held[i]);
        r |= from & (0xFFu << (8 * b));
      }
      w[i] = r;
    }
    *at = w;
  }
}

// ---- attention
//
//   x[j] = scale * ks[j] * (q . kc[j])      over the tokens j that the row sees
//   o    = sum_j e^(x[j] - lse) * vs[j] * vc[j],  lse = log sum_j e^x[j]
//
// kc, vc are the cached codes, ks, vs the scales of their blocks.  Rows are
// the queries of one key/value head: row r of a sequence is query r / g, head
// r % g of the group of g = h_q / h_kv heads that share the keys.
//
// Per row the kernels carry the running maximum m of t[j] = log2(e) x[j] +
// log2(vs[j]), u = sum_j 2^(t[j] - m) vc[j] and l = sum_j 2^(t[j] - m) / vs[j],
// all in fp32.  With the values' scale inside the exponent, p = 2^(t - m) is
// what multiplies the codes, whichever block they are in: one accumulator
// serves blocks of any scale, o = u / l, and lse = (m + log2 l) ln 2.
//
// Both products run on the matrix cores with the 16 (or 32) rows as columns:
// x^T = K q^T in bf16 (e4m3 codes are exact in bf16, q is bf16 anyway) and
// u^T = V^T p^T in fp16.  fp16 holds e4m3 codes exactly too and rounds p to
// 11 bits where bf16 keeps 8; p is at most 2^kSlack and what falls below
// 2^-24 of that adds nothing that bf16 output could show.
// The keys of a 64-key step are dealt to the rows of the A operand so that
// lane group g (lanes 16 g ..) ends up with p for keys 16 g .. 16 g + 15,
// which is how a lane of the second product's B operand wants them against
// 16 contiguous bytes of V^T: no value moves between lanes or through LDS
// from load to result.

struct Kv8AttnParams {
  const uint16_t* q;  // bf16 [total][h_q][d], q_stride elements from token to token
  long long q_stride;
  Kv8Cache c;
  const int32_t* kv_lens;  // tokens in the cache, per sequence
  const int32_t* cu;       // running sums of the queries, batch + 1 entries
  uint16_t* out;           // bf16 [total][h_q][d]
  float* lse;              // [total][h_q] or null
  float scale_log2;        // scale * log2(e)
  int causal, window, batch, total, most, h_q, group;
  // split work: workgroup w computes its share of the units below
  float* part_u;   // [workers][2][16][d]
  float* part_ml;  // [workers][2][16][2]
  int workers;
};

constexpr int kKv8Step = 64;    // keys of one step of one wave
constexpr float kKv8MinVs = 5.421010862427522e-20f;  // 2^-64: scales below are taken as this

// What a sequence asks for.
struct Kv8Seq {
  int first, count;   // its rows of q
  int kv;             // its tokens in the cache
  int step0, steps;   // steps of keys that any of its queries sees: step0 .. step0 + steps - 1
  int tiles;          // 16-row tiles of one key/value head
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8AttnParams& p, int seq) {
  Kv8Seq s;
  kv8_rows(p.cu, seq, p.total, p.most, &s.first, &s.count);
  const long long room = (long long)p.c.max_blocks << p.c.block_log2;
  const int kv = max(p.kv_lens[seq], 0);
  s.kv = kv < room ? kv : (int)room;
  const int lo = p.window > 0 ? max(s.kv - s.count - p.window + 1, 0) : 0;
  s.step0 = min(lo, s.kv) / kKv8Step;
  s.steps = (s.kv + kKv8Step - 1) / kKv8Step - s.step0;
  s.tiles = (s.count * p.group + 15) / 16;
  return s;
}

__device__ __forceinline__ long long kv8_units(const Kv8AttnParams& p, const Kv8Seq& s) {
  return (long long)p.c.h_kv * s.tiles * s.steps;
}

// Keys [lo, hi) that query `i` of the sequence sees.
__device__ __forceinline__ void kv8_sees(const Kv8AttnParams& p, const Kv8Seq& s, int i, int* lo, int* hi) {
  const int pos = s.kv - s.count + i;  // where the query stands (negative: before the cache, it sees nothing)
  *hi = p.causal ? min(max(pos + 1, 0), s.kv) : s.kv;
  *lo = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
}

// Sum over a workgroup of 256 threads; every thread gets it.  `box` is 4 longs of LDS.
__device__ __forceinline__ long long kv8_sum256(long long v, long long* box) {
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) box[threadIdx.x >> 6] = v;
  __syncthreads();
  return box[0] + box[1] + box[2] + box[3];
}

// Units of all sequences, and of the sequences before `upto`.
__device__ __forceinline__ void kv8_total(const Kv8AttnParams& p, int upto, long long* total, long long* before,
                                          long long* box) {
  long long all = 0, some = 0;
  for (int i = threadIdx.x; i < p.batch; i += 256) {
    const long long u = kv8_units(p, kv8_seq(p, i));
    all += u;
    some += i < upto ? u : 0;
  }
  *total = kv8_sum256(all, box);
  *before = kv8_sum256(some, box);
}

// The sequence that unit `at` (below the total) is of, and its first unit.
__device__ __forceinline__ void kv8_find(const Kv8AttnParams& p, long long at, int* seq, long long* seq0,
                                         long long* box) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  long long carry = 0;
  for (int c = 0; c < p.batch; c += 256) {
    const int i = c + tid;
    const long long u = i < p.batch ? kv8_units(p, kv8_seq(p, i)) : 0;
    long long sum = u;  // of the wave's lanes up to this one
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const long long o = __shfl_up(sum, s, 64);
      if (lane >= s) sum += o;
    }
    __syncthreads();
    if (lane == 63) box[wave] = sum;
    __syncthreads();
    long long before = carry + sum - u;
    for (int w = 0; w < wave; ++w) before += box[w];
    carry += box[0] + box[1] + box[2] + box[3];
    if (u > 0 && at >= before && at < before + u) {
      box[4] = i;
      box[5] = before;
    }
    if (at < carry) break;
  }
  __syncthreads();
  *seq = (int)box[4];
  *seq0 = box[5];
}

// How many workgroups share the units: all that run, but no more than would
// leave each of a workgroup's waves a step.
__device__ __forceinline__ int kv8_workers(const Kv8AttnParams& p, long long total) {
  return (int)min((long long)p.workers, (total + 3) / 4);
}

// Workgroup w of `workers` takes units [total w / workers, total (w + 1) / workers).
__device__ __forceinline__ long long kv8_share(long long total, int w, int workers) { return total * w / workers; }

// The workgroup that has unit x.
__device__ __forceinline__ int kv8_owner(long long total, long long x, int workers) {
  return (int)(((x + 1) * workers - 1) / total);
}

// Eight e4m3 codes (two dwords) as bf16, and as fp16.
__device__ __forceinline__ v8bf e4m3_to_bf16(uint32_t lo, uint32_t hi) {
  v4u r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  return __builtin_bit_cast(v8bf, r);
}
__device__ __forceinline__ v8h e4m3_to_f16(uint32_t lo, uint32_t hi) {
  v4u r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true));
  return __builtin_bit_cast(v8h, r);
}

__device__ __forceinline__ uint32_t pack2_f16(float a, float b) {
  v2h r;
  r[0] = (_Float16)a;
  r[1] = (_Float16)b;
  return __builtin_bit_cast(uint32_t, r);
}

// Bytes of `w` whose code is NaN (0x7F, 0xFF), as 0x01 in each such byte.
__device__ __forceinline__ uint32_t kv8_nan_bytes(uint32_t w) {
  // 0x7F + 1 carries into bit 7 of the byte, any smaller magnitude does not
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) >> 7 & 0x01010101u;
}

// A wave's running state for its 16 rows: lane l holds row l % 16, dimensions
// 16 i + 4 (l / 16) + e of u in u[i][e], and its own lane group's part of l.
template <int D>
struct Kv8State {
  v4f u[D / 16];
  float m, l;
};

// One step: 64 keys from token `base` on.
template <int D>
__device__ __forceinline__ void kv8_step(const Kv8AttnParams& p, int seq, int head, const Kv8Seq& sq, int base,
                                         int row_lo, int row_hi, bool masked, const v8bf (&qf)[D / 32],
                                         Kv8State<D>& st) {
  const int lane = threadIdx.x & 63, a = lane & 15, g = lane >> 4;
  const Kv8Cache& c = p.c;
  // this lane's 16-key run: as a row of K in the first product, and as the
  // keys of its lane group in p and V^T
  const int run_k = base + (a >> 2) * 16, run_v = base + g * 16;
  const int page_k = run_k < sq.kv ? kv8_page(c, seq, run_k) : -1;
  const int page_v = run_v < sq.kv ? kv8_page(c, seq, run_v) : -1;
  const int inside = c.block - 1;
  v4u kw[4][D / 64];
  {
    const uint8_t* src = c.k_codes + ((size_t)max(page_k, 0) * c.h_kv + head) * (size_t)c.block * D +
                         (size_t)((run_k & inside) + (a & 3)) * D + g * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        kw[j][h] = v4u{0, 0, 0, 0};
        if (page_k >= 0) kw[j][h] = *(const v4u*)(src + j * 4 * D + h * 64);
      }
  }
  v4u vw[D / 16];
  {
    const uint8_t* src = c.v_codes + ((size_t)max(page_v, 0) * c.h_kv + head) * (size_t)c.block * D +
                         (size_t)a * c.block + (run_v & inside);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      vw[i] = v4u{0, 0, 0, 0};
      if (page_v >= 0) vw[i] = *(const v4u*)(src + (size_t)i * 16 * c.block);
    }
  }
  float ks = 0.f, vs = 1.f;
  if (page_v >= 0) {
    ks = c.k_scales[(size_t)page_v * c.h_kv + head];
    vs = c.v_scales[(size_t)page_v * c.h_kv + head];
  }
  ks *= p.scale_log2;
  vs = fmaxf(vs, kKv8MinVs);
  const float lv = __builtin_amdgcn_logf(vs), inv_vs = __builtin_amdgcn_rcpf(vs);

  // t[4 j + e]: key run_v + 4 j + e of row a
  float t[16];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v4f s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_to_bf16(kw[j][h][0], kw[j][h][1]), qf[2 * h], s, 0, 0, 0);
      s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_to_bf16(kw[j][h][2], kw[j][h][3]), qf[2 * h + 1], s, 0, 0, 0);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) t[4 * j + e] = s[e] * ks + lv;
  }
  uint32_t seen = 0xFFFFu;  // bit i: this row sees key run_v + i
  if (masked) {
    seen = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool in = page_v >= 0 && run_v + i >= row_lo && run_v + i < row_hi;
      seen |= (in ? 1u : 0u) << i;
      t[i] = in ? t[i] : -__builtin_huge_valf();
    }
  }
  float m = t[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) m = fmaxf(m, t[i]);
  m = fmaxf(m, __shfl_xor(m, 16, 64));
  m = fmaxf(m, __shfl_xor(m, 32, 64));
  m = fmaxf(m, st.m);
  const float ref = m == -__builtin_huge_valf() ? 0.f : m;  // nothing seen yet: any finite reference
  if (__any(m > st.m)) {
    const float shrink = __builtin_amdgcn_exp2f(st.m - ref);
    st.l *= shrink;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.u[i] *= shrink;
    st.m = m;
  }
  float sum = 0.f;
  v4u pw[2], rest[2];
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float p0 = __builtin_amdgcn_exp2f(t[i] - ref), p1 = __builtin_amdgcn_exp2f(t[i + 1] - ref);
    sum += p0 + p1;
    pw[i / 8][(i / 2) & 3] = pack2_f16(p0, p1);
  }
  st.l += sum * inv_vs;
  if (masked) {
    // Bytes past the sequence's end hold anything: zero them.  A NaN code of
    // a token that some rows see and others do not must reach the former
    // only, and 0 * NaN would reach both: such codes are zeroed, and a second
    // product counts, per row and dimension, the NaN that the row sees.
    v4u keep;
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = min(max(sq.kv - (run_v + 4 * i), 0), 4);
      keep[i] = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      vw[i] &= keep;
#pragma unroll
      for (int e = 0; e < 4; ++e) bad |= kv8_nan_bytes(vw[i][e]);
    }
    if (__any(bad != 0)) {
      v4u sw[2];
#pragma unroll
      for (int i = 0; i < 16; i += 2)
        sw[i / 8][(i / 2) & 3] = (seen >> i & 1 ? 0x3C00u : 0u) | (seen >> i & 2 ? 0x3C000000u : 0u);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        v4f cnt = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v4u ind;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t b = kv8_nan_bytes(vw[i][2 * h + e]);
            vw[i][2 * h + e] &= ~(b * 255u);
            ind[2 * e] = (b & 1u) * 0x3C00u | (b >> 8 & 1u) * 0x3C000000u;
            ind[2 * e + 1] = (b >> 16 & 1u) * 0x3C00u | (b >> 24 & 1u) * 0x3C000000u;
          }
          cnt = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, ind), __builtin_bit_cast(v8h, sw[h]),
                                                       cnt, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (cnt[e] > 0.f) st.u[i][e] = __builtin_nanf("");
      }
    }
    // What fp16 left of p, as a second fp16: rows that see few keys (all of
    // them in a masked step) have large outputs that no averaging of the
    // rounding errors helps; with one piece 5 of 493568 outputs of prompts of
    // up to 150 tokens were off by more than 70% of 8e-3 |r| + 1e-3 rms, the
    // worst by 129%, with two in these steps none, the worst 49% (bf16's own
    // rounding).
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const uint32_t both = pw[i / 8][(i / 2) & 3];
      const v2h hi = __builtin_bit_cast(v2h, both);
      rest[i / 8][(i / 2) & 3] = pack2_f16(__builtin_amdgcn_exp2f(t[i] - ref) - (float)hi[0],
                                           __builtin_amdgcn_exp2f(t[i + 1] - ref) - (float)hi[1]);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        st.u[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(e4m3_to_f16(vw[i][2 * h], vw[i][2 * h + 1]),
                                                         __builtin_bit_cast(v8h, rest[h]), st.u[i], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      st.u[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(e4m3_to_f16(vw[i][2 * h], vw[i][2 * h + 1]),
                                                       __builtin_bit_cast(v8h, pw[h]), st.u[i], 0, 0, 0);
  }
}

// Rows are written by 16 threads each: thread part of a row holds D / 16 of
// its dimensions.
template <int D>
__device__ __forceinline__ void kv8_write(const Kv8AttnParams& p, const Kv8Seq& sq, int head, int row, int part,
                                          const float (&u)[D / 16], float m, float l) {
  if (row >= sq.count * p.group) return;
  const int token = sq.first + row / p.group, hq = head * p.group + row % p.group;
  const size_t at = (size_t)token * p.h_q + hq;
  // l == 0: the row sees no key
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < D / 16; i += 2)
    *(uint32_t*)(p.out + at * D + part * (D / 16) + i) = pack2_bf16(u[i] * inv, u[i + 1] * inv);
  if (p.lse && part == 0) p.lse[at] = (m + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
}

// A workgroup of four waves takes an equal share of all (sequence, head, row
// tile, 64-key step) units, in that order; within a run of steps of one tile
// its waves take every fourth step each and merge in LDS.  Runs that cover a
// tile's steps wholly are written out, others leave their (u, m, l) to
// kv8_join_kernel.  The shares come from the lengths on the device: nothing
// of the launch depends on them, and the longest sequence spreads over as
// many workgroups as its part of the batch's keys is worth.
template <int D>
__global__ __launch_bounds__(256) void kv8_attn_kernel(Kv8AttnParams p) {
  constexpr int kPitch = D + 4;
  __shared__ float s_u[4][16][kPitch];
  __shared__ float s_m[4][16], s_l[4][16];
  __shared__ long long box[6];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, a = lane & 15, g = lane >> 4;
  long long total, unused;
  kv8_total(p, 0, &total, &unused, box);
  const int workers = kv8_workers(p, total);
  if ((int)blockIdx.x >= workers) return;
  const long long begin = kv8_share(total, blockIdx.x, workers), end = kv8_share(total, blockIdx.x + 1, workers);
  long long at = begin;
  int seq;
  long long seq0;  // first unit of seq
  kv8_find(p, at, &seq, &seq0, box);
  Kv8Seq sq = kv8_seq(p, seq);
  long long units = kv8_units(p, sq);
  while (at < end) {
    while (at >= seq0 + units) {
      seq0 += units;
      ++seq;
      sq = kv8_seq(p, seq);
      units = kv8_units(p, sq);
    }
    const long long rel = at - seq0;
    const int tile_no = (int)(rel / sq.steps);
    const int head = tile_no / sq.tiles, tile = tile_no % sq.tiles;
    const int t0 = (int)(rel - (long long)tile_no * sq.steps);
    const int t1 = (int)min((long long)sq.steps, t0 + (end - at));

    // this lane's row: its query as B fragments, and the keys it sees
    const int row = tile * 16 + a, rows = sq.count * p.group;
    const int safe = min(row, rows - 1);
    const int qi = safe / p.group;
    const uint16_t* src = p.q + (long long)(sq.first + qi) * p.q_stride + (long long)(head * p.group + safe % p.group) * D;
    v8bf qf[D / 32];
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      qf[2 * h] = __builtin_bit_cast(v8bf, *(const v4u*)(src + h * 64 + g * 16));
      qf[2 * h + 1] = __builtin_bit_cast(v8bf, *(const v4u*)(src + h * 64 + g * 16 + 8));
    }
    int row_lo, row_hi;
    kv8_sees(p, sq, qi, &row_lo, &row_hi);
    // keys that every row of the tile sees, and that any row sees
    int all_lo, all_hi, any_lo, any_hi;
    kv8_sees(p, sq, min(tile * 16 + 15, rows - 1) / p.group, &all_lo, &any_hi);
    kv8_sees(p, sq, tile * 16 / p.group, &any_lo, &all_hi);
    Kv8State<D> st;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.u[i] = v4f{0.f, 0.f, 0.f, 0.f};
    st.m = -__builtin_huge_valf();
    st.l = 0.f;
    for (int t = t0 + wave; t < t1; t += 4) {
      const int base = (sq.step0 + t) * kKv8Step;
      if (base >= any_hi || base + kKv8Step <= any_lo) continue;  // no row sees any of it
      // a step needs masks unless every row sees all of it and the table has all of it
      bool masked = base < all_lo || base + kKv8Step > all_hi;
      if (!masked) masked = __any(kv8_page(p.c, seq, base + g * 16) < 0);
      kv8_step<D>(p, seq, head, sq, base, row_lo, row_hi, masked, qf, st);
    }
    // the waves' states, merged in LDS
    st.l += __shfl_xor(st.l, 16, 64);
    st.l += __shfl_xor(st.l, 32, 64);
    __syncthreads();
    if (g == 0) {
      s_m[wave][a] = st.m;
      s_l[wave][a] = st.l;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) *(v4f*)&s_u[wave][a][i * 16 + g * 4] = st.u[i];
    __syncthreads();
    {
      const int r = tid >> 4, part = tid & 15;
      float m = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
      const float ref = m == -__builtin_huge_valf() ? 0.f : m;
      float l = 0.f, u[D / 16];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) u[i] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_m[w][r] - ref);
        l += s_l[w][r] * f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) u[i] += s_u[w][r][part * (D / 16) + i] * f;
      }
      if (t0 == 0 && t1 == sq.steps) {
        kv8_write<D>(p, sq, head, tile * 16 + r, part, u, m, l);
      } else {
        const size_t slot = ((size_t)blockIdx.x * 2 + (at == begin ? 0 : 1)) * 16 + r;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) p.part_u[slot * D + part * (D / 16) + i] = u[i];
        if (part == 0) {
          p.part_ml[slot * 2] = m;
          p.part_ml[slot * 2 + 1] = l;
        }
      }
    }
    at += t1 - t0;
  }
}

// Joins the parts of every tile that more than one workgroup had, in their
// order, and writes the rows of sequences without keys.  One workgroup a
// (tile, head, sequence).
template <int D>
__global__ __launch_bounds__(256) void kv8_join_kernel(Kv8AttnParams p) {
  __shared__ long long box[4];
  const int tile = blockIdx.x, head = blockIdx.y, seq = blockIdx.z;
  const Kv8Seq sq = kv8_seq(p, seq);
  if (tile >= sq.tiles) return;
  const int r = threadIdx.x >> 4, part = threadIdx.x & 15;
  float u[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) u[i] = 0.f;
  float m = -__builtin_huge_valf(), l = 0.f;
  if (sq.steps > 0) {
    long long total, seq0;
    kv8_total(p, seq, &total, &seq0, box);
    const long long s0 = seq0 + ((long long)head * sq.tiles + tile) * sq.steps;
    const int workers = kv8_workers(p, total);
    const int w0 = kv8_owner(total, s0, workers), w1 = kv8_owner(total, s0 + sq.steps - 1, workers);
    if (w0 == w1) return;  // one workgroup had all of it and wrote it
    for (int w = w0; w <= w1; ++w) {
      const size_t slot = ((size_t)w * 2 + (s0 > kv8_share(total, w, workers) ? 1 : 0)) * 16 + r;
      const float mw = p.part_ml[slot * 2], lw = p.part_ml[slot * 2 + 1];
      const float to = fmaxf(m, mw), ref = to == -__builtin_huge_valf() ? 0.f : to;
      const float f = __builtin_amdgcn_exp2f(m - ref), fw = __builtin_amdgcn_exp2f(mw - ref);
      l = l * f + lw * fw;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) u[i] = u[i] * f + p.part_u[slot * D + part * (D / 16) + i] * fw;
      m = to;
    }
  }
  kv8_write<D>(p, sq, head, tile * 16 + r, part, u, m, l);
}

}  // namespace dg
