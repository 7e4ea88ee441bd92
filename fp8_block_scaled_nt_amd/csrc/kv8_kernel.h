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
typedef int16_t v2s __attribute__((ext_vector_type(2)));

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
// neither read nor written.  max_blocks is at least 1.
__device__ __forceinline__ int kv8_page(const Kv8Cache& c, int seq, int token) {
  const int j = token >> c.block_log2;
  const int page = c.table[(size_t)seq * c.max_blocks + min(max(j, 0), c.max_blocks - 1)];
  // one select, no branches around the load: it is to be in flight early
  return ((unsigned)j < (unsigned)c.max_blocks) & ((unsigned)page < (unsigned)c.num_blocks) ? page : -1;
}

// New rows of sequence `seq`: [first, first + count) of the packed tokens.
// cu holds batch + 1 running sums; whatever it holds, the range stays inside
// the `total` packed tokens, and count is at most `most`.  Returns the
// sequence's rows without that limit.
__device__ __forceinline__ int kv8_rows(const int32_t* cu, int seq, int total, int most, int* first, int* count) {
  const int lo = min(max(cu[seq], 0), total), hi = min(max(cu[seq + 1], 0), total), all = max(hi - lo, 0);
  *first = lo;
  *count = min(all, most);
  return all;
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
// The new values stay in registers between their maximum and their codes.  A
// thread takes items of 8 dimensions by 4 positions of the block (those with a
// new token in them), so that values, which lie dimension by dimension, turn
// in LDS by whole words of 4 tokens: D rows of `block` codes.
template <int D, int ITEMS, int THREADS>
__global__ __launch_bounds__(THREADS) void kv8_append_kernel(Kv8AppendParams p) {
  constexpr int kPer = D / 8;  // 16-byte pieces of a token's head
  __shared__ float s_max[THREADS / 64];
  extern __shared__ __align__(16) uint8_t turn[];  // values: [D][block + 16]
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
  const uint16_t* src = x + (long long)(first + base - ctx) * stride + (long long)head * D;  // position 0's row
  const size_t tile = (size_t)page * p.c.h_kv + head;
  float* scale = (values ? p.c.v_scales : p.c.k_scales) + tile;
  uint8_t* codes = (values ? p.c.v_codes : p.c.k_codes) + tile * (size_t)block * D;
  const float was = old > 0 ? *scale : 0.f;

  const int group0 = old >> 2, items = (((stop + 3) >> 2) - group0) * kPer;
  v4u held[ITEMS][4];
  float amax = 0.f;
#pragma unroll
  for (int n = 0; n < ITEMS; ++n) {
    const int e = tid + n * THREADS, pos = (group0 + e / kPer) * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      held[n][j] = v4u{0, 0, 0, 0};
      if (e < items && pos + j >= old && pos + j < stop)
        held[n][j] = *(const v4u*)(src + (long long)(pos + j) * stride + e % kPer * 8);
    }
  }
#pragma unroll
  for (int n = 0; n < ITEMS; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = fabsf(__uint_as_float(held[n][j][i] << 16)), hi = fabsf(__uint_as_float(held[n][j][i] & 0xFFFF0000u));
        amax = fmaxf(amax, lo < __builtin_huge_valf() ? lo : 0.f);
        amax = fmaxf(amax, hi < __builtin_huge_valf() ? hi : 0.f);
      }
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) amax = fmaxf(amax, __shfl_xor(amax, s, 64));
  if constexpr (THREADS > 64) {
    if ((tid & 63) == 0) s_max[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) amax = fmaxf(amax, s_max[w]);
  }
  const float now = fmaxf(was, kv8_scale(amax));
  const float inv = 1.f / now;  // a power of two: exact
  const bool grow = old > 0 && now > was;
  const float by = was * inv;
  if (tid == 0) *scale = now;

  const int pitch = block + 16;
#pragma unroll
  for (int n = 0; n < ITEMS; ++n) {
    const int e = tid + n * THREADS, pos = (group0 + e / kPer) * 4, c = e % kPer;
    if (e >= items) continue;
    uint32_t code[4][2];  // of each token, 4 dimensions a word
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t a = held[n][j][2 * i], b = held[n][j][2 * i + 1];
        code[j][i] = kv8_pack4(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xFFFF0000u) * inv,
                               __uint_as_float(b << 16) * inv, __uint_as_float(b & 0xFFFF0000u) * inv);
      }
    if (!values) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (pos + j >= old && pos + j < stop)
          *(uint2*)(codes + (size_t)(pos + j) * D + c * 8) = make_uint2(code[j][0], code[j][1]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // a 4 x 4 transpose of bytes: words of one dimension, 4 tokens each
        const uint32_t lo01 = __builtin_amdgcn_perm(code[1][i], code[0][i], 0x05010400u);
        const uint32_t lo23 = __builtin_amdgcn_perm(code[3][i], code[2][i], 0x05010400u);
        const uint32_t hi01 = __builtin_amdgcn_perm(code[1][i], code[0][i], 0x07030602u);
        const uint32_t hi23 = __builtin_amdgcn_perm(code[3][i], code[2][i], 0x07030602u);
        uint8_t* to = turn + (c * 8 + i * 4) * pitch + pos;
        *(uint32_t*)(to) = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
        *(uint32_t*)(to + pitch) = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
        *(uint32_t*)(to + 2 * pitch) = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
        *(uint32_t*)(to + 3 * pitch) = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
      }
    }
  }
  if (!values) {
    if (grow)
      for (int e = tid; e < old * kPer; e += THREADS) {
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
  for (int e = tid; e < D * per_row; e += THREADS) {
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
      const uint32_t was4 = held[i], fresh4 = fresh[i];
      const uint32_t kept = grow ? kv8_rescale4(was4, by) : was4;
      const int o = min(max(old - (t0 + i * 4), 0), 4), s = min(max(stop - (t0 + i * 4), 0), 4);
      const uint32_t is_old = o == 4 ? ~0u : (1u << (8 * o)) - 1u, is_in = s == 4 ? ~0u : (1u << (8 * s)) - 1u;
      w[i] = (kept & is_old) | (fresh4 & is_in & ~is_old) | (was4 & ~is_in);
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
// Per row the kernels carry a reference m, 7 to 11 below the running maximum of
// t[j] = log2(e) x[j] + log2(vs[j]), u = sum_j 2^(t[j] - m) vc[j] and l = sum_j
// 2^(t[j] - m) / vs[j], all in fp32.  With the values' scale inside the
// exponent, p = 2^(t - m) is what multiplies the codes, whichever block they are
// in: one accumulator serves blocks of any scale, o = u / l, and lse = (m + log2
// l) ln 2.
//
// Both products run on the matrix cores with the 16 (or 32) rows as columns:
// x^T = K q^T in bf16 (e4m3 codes are exact in bf16, q is bf16 anyway) and
// u^T = V^T p^T with p in one of two forms.  A small p may be all that an element
// has, as the codes beside a large one may be zeros in its dimension:
//
//   narrow: fp16, which holds e4m3 codes exactly too and rounds p to 11 bits.  p
//     goes up to 2^11, its normal range ends 2^-21 or less below the row's
//     largest p, and what lies below is off by at most 2^-32 of that largest.
//     Only where value scales are within 2^kKv8Near of the largest one met: an
//     element is then off by no more than 2^(kKv8Near - 32) of the largest weight
//     times value scale, per key, whatever the codes are.
//   wide: two bf16 pieces, 16 bits with the range of fp32, against codes in
//     bf16: where value scales lie further apart, and in steps that need masks
//     (rows that see few keys, all of them in such a step, have large outputs
//     that no averaging of rounding errors helps: 11 bits left 5 of 493568
//     outputs of prompts of up to 150 tokens off by more than 70% of 8e-3 |r| +
//     1e-3 rms, the worst by 129%).
//
// (With fp16 alone prompts of 2048 took 296 us against 300 and 4 x 256 of 256
// 20.2 against 21.2; with value scales 2^12 apart elements then missed their
// bound, at 2^60 they were zero.)
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
  int rows_lo, rows_hi;    // only sequences of rows_lo .. rows_hi - 1 rows (queries x group) are this launch's
  // split work: workgroup w computes its share of the units below
  float* part_u;   // [workers][2][16][d]
  float* part_ml;  // [workers][2][16][2]
  int* arrived;    // [workers] counters, zero between calls
  int workers;
};

constexpr int kKv8Step = 64;       // keys of one step of one wave
constexpr float kKv8Lead = 7.f;    // log2 of a row's largest p when its reference has moved
constexpr float kKv8Slack = 11.f;  // and of how large p may get before it moves again
constexpr float kKv8WideLog2 = 112.f;  // log2 of what p is multiplied with in the wide form: 16 keys' sum stays below 2^128
constexpr float kKv8WideInv = 1.925929944387236e-34f;  // 2^-112
constexpr float kKv8Near = 4.f;        // log2 of how far value scales may lie apart in narrow steps
constexpr float kKv8NearRatio = 16.f;  // 2^kKv8Near
constexpr float kKv8MinVs = 5.421010862427522e-20f;  // 2^-64: scales below are taken as this

// What a sequence asks for.
struct Kv8Seq {
  int first, count;   // its rows of q
  int kv;             // its tokens in the cache that the table has room for
  int pos;            // where its first query stands (negative: before the cache), by its length whatever the table's
  int step0, steps;   // steps of keys that any of its queries sees: step0 .. step0 + steps - 1
  int tiles;          // 16-row tiles of one key/value head
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8AttnParams& p, int seq) {
  Kv8Seq s;
  const int all = kv8_rows(p.cu, seq, p.total, p.most, &s.first, &s.count);
  if (s.count * p.group < p.rows_lo || s.count * p.group >= p.rows_hi) s.count = 0;
  const long long room = (long long)p.c.max_blocks << p.c.block_log2;
  const int kv = max(p.kv_lens[seq], 0);
  s.kv = kv < room ? kv : (int)room;
  s.pos = kv - all;
  const int lo = p.window > 0 ? max(max(s.pos, -1) - p.window + 1, 0) : 0;
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
  const int pos = max(s.pos + i, -1);  // -1: before the cache, it sees nothing if causal
  *hi = p.causal ? min(pos + 1, s.kv) : s.kv;
  *lo = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
}

// Inclusive running sum over a workgroup of 256 threads, and its total.
__device__ __forceinline__ long long kv8_scan256(long long v, long long* total, long long* box) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const long long o = __shfl_up(v, s, 64);
    if (lane >= s) v += o;
  }
  __syncthreads();
  if (lane == 63) box[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v += box[w];
  *total = box[0] + box[1] + box[2] + box[3];
  return v;
}

// Units of 256 sequences from `first` on: this thread's, the units before
// them among the 256, and the total.
struct Kv8Chunk {
  long long units, before, total;
};

__device__ __forceinline__ Kv8Chunk kv8_chunk(const Kv8AttnParams& p, int first, long long* box) {
  const int i = first + threadIdx.x;
  Kv8Chunk c;
  c.units = i < p.batch ? kv8_units(p, kv8_seq(p, i)) : 0;
  c.before = kv8_scan256(c.units, &c.total, box) - c.units;
  return c;
}

// The sequence that unit `at` is of, and its first unit; `c` is the chunk of
// the first 256 sequences, the only one of most batches.
__device__ __forceinline__ void kv8_find(const Kv8AttnParams& p, Kv8Chunk c, long long at, int* seq, long long* seq0,
                                         long long* box) {
  long long carry = 0;
  int first = 0;
  while (at >= carry + c.total) {
    carry += c.total;
    first += 256;
    c = kv8_chunk(p, first, box);
  }
  const long long from = carry + c.before;
  if (at >= from && at < from + c.units) {
    box[4] = first + threadIdx.x;
    box[5] = from;
  }
  __syncthreads();
  *seq = (int)box[4];
  *seq0 = box[5];
}

// a / b for a >= 0, b > 0; in 32 bits where they fit, which takes a tenth of
// the instructions (a 64-bit quotient in every place took the smallest calls 1
// us and more).
__device__ __attribute__((noinline)) long long kv8_div64(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long kv8_div(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : kv8_div64(a, b);
}

// Units of a workgroup's share: workgroup w takes units [w s, (w + 1) s).  At
// least one for each of its waves.
__device__ __forceinline__ long long kv8_share(const Kv8AttnParams& p, long long total) {
  return max(kv8_div(total + p.workers - 1, p.workers), 4LL);
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

// Two e4m3 values held as fp16, as bf16 times 2^-112: the exponent's and the
// three upper fraction bits move to their places, and the biases differ by 112.
// `keep` has kKv8Halves' bits of the halves to keep; the others become zero.
// NaN keeps its all-ones exponent, of five bits, which is a finite value then.
constexpr uint32_t kKv8Halves = 0x8FFF8FFFu;
__device__ __forceinline__ uint32_t f16_to_small_bf16(uint32_t w, uint32_t keep) {
  const v2s r = __builtin_bit_cast(v2s, w) >> 3;
  return __builtin_bit_cast(uint32_t, r) & keep;
}
// Which halves of such a pair are NaN (e4m3 has no infinities), as 1 in bit 0 and bit 16.
__device__ __forceinline__ uint32_t small_bf16_nans(uint32_t w) {
  return ((w & 0x0FFF0FFFu) + 0x00800080u) >> 12 & 0x00010001u;
}

// The largest x of the four lane groups (of lanes l % 16 alike).
__device__ __forceinline__ float kv8_group_max(float x) {
  const uint32_t b = __float_as_uint(x);
  const v2u r = __builtin_bit_cast(v2u, __builtin_amdgcn_permlane32_swap(b, b, false, false));
  const uint32_t c = __float_as_uint(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
  const v2u s = __builtin_bit_cast(v2u, __builtin_amdgcn_permlane16_swap(c, c, false, false));
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// A wave's running state for 16 MT rows: lane l holds, for each tile of 16,
// row l % 16, dimensions 16 i + 4 (l / 16) + e of u in u[i][e], and its own
// lane group's part of l.
template <int D, int MT>
struct Kv8State {
  v4f u[MT][D / 16];
  float m[MT], l[MT];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) u[t][i] = v4f{0.f, 0.f, 0.f, 0.f};
      m[t] = -__builtin_huge_valf();
      l[t] = 0.f;
    }
  }
};

// Where a lane's rows stand: keys [lo, hi) that its row of each tile sees.
template <int MT>
struct Kv8Rows {
  int lo[MT], hi[MT];
};

// The block that holds the 16 keys of this lane group's run, and its scales as
// they are in memory.
struct Kv8Run {
  int page;
  float ks, vs;
};

__device__ __forceinline__ Kv8Run kv8_run(const Kv8Cache& c, int head, int page) {
  const size_t at = (size_t)max(page, 0) * c.h_kv + head;
  return Kv8Run{page, c.k_scales[at], c.v_scales[at]};
}

// What a step needs of them: t = s ks + lv; 1 / vs; whether the block is there.
struct Kv8Scale {
  float ks, lv, inv_vs;
  int there;
};

__device__ __forceinline__ Kv8Scale kv8_scale_of(const Kv8Run& run, float scale_log2) {
  const bool there = run.page >= 0;
  const float vs = there ? fmaxf(run.vs, kKv8MinVs) : 1.f;
  return Kv8Scale{run.ks * scale_log2, __builtin_amdgcn_logf(vs), __builtin_amdgcn_rcpf(vs), there};
}

// Whether a step needs the wide form for its blocks: one is not there, or value
// scales are far apart; `top` is the log2 of the largest so far and takes this
// step's in.  Most steps leave by one test.
__device__ __forceinline__ bool kv8_far(const Kv8Scale& sc, float& top) {
  if (!__any(!sc.there || sc.lv > top || sc.lv < top - kKv8Near)) return false;
  top = fmaxf(top, kv8_group_max(sc.there ? sc.lv : -__builtin_huge_valf()));
  return __any(!sc.there || sc.lv < top - kKv8Near);
}

// What remains of a step when its raw products s[4 j + e] with keys run_v + 4 j
// + e are there: t = s ks + lv, the reference, p, and the second product,
// narrow or (WIDE) wide and with masks.  load_v(i, o) gives the lane's values of
// dimension 16 i + a at keys 16 g + 8 o .. (a = lane % 16, g = lane / 16) in fp16.
// WIDE: some row may not see some of the keys, or the sequence end inside the
// step (such steps are the first and last ones of a run), or the value scales are
// far apart.
template <int D, int MT, bool WIDE, class LoadV>
__device__ __forceinline__ void kv8_rest_of_step(int kv, int run_v, const Kv8Scale& sc, const Kv8Rows<MT>& rows,
                                                 float (&s)[MT][16], Kv8State<D, MT>& st, LoadV load_v) {
  float ks = sc.ks, lv = sc.lv;
  uint32_t seen[MT];  // bit i: the row sees key run_v + i
  if constexpr (WIDE) {
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      // keys [lo, hi) of the 16, none if the block is not there
      const int lo = min(max(rows.lo[t] - run_v, 0), 16), hi = sc.there ? min(max(rows.hi[t] - run_v, 0), 16) : 0;
      seen[t] = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[t][i] = seen[t] >> i & 1u ? s[t][i] * ks + lv : -__builtin_huge_valf();
    }
    ks = 1.f;
    lv = 0.f;
  }
  v4u pw[MT][2], rest[MT][2];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    float m = s[t][0];
#pragma unroll
    for (int i = 1; i < 16; ++i) m = fmaxf(m, s[t][i]);
    m = m * ks + lv;
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    // The reference follows the maximum only when a row's p would pass
    // 2^kKv8Slack, and is put 2^kKv8Lead below it: few steps pay for scaling u.
    if (__any(m > st.m[t] + kKv8Slack)) {
      m = fmaxf(m - kKv8Lead, st.m[t]);
      const float shrink = __builtin_amdgcn_exp2f(st.m[t] - (m == -__builtin_huge_valf() ? 0.f : m));
      st.l[t] *= shrink;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) st.u[t][i] *= shrink;
      st.m[t] = m;
    }
    const float ref = st.m[t] == -__builtin_huge_valf() ? 0.f : st.m[t];  // nothing seen yet: any finite reference
    const float off = lv - ref + (WIDE ? kKv8WideLog2 : 0.f);
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float p0 = __builtin_amdgcn_exp2f(s[t][i] * ks + off), p1 = __builtin_amdgcn_exp2f(s[t][i + 1] * ks + off);
      sum[0] += p0;
      sum[1] += p1;
      if constexpr (!WIDE) {
        pw[t][i / 8][(i / 2) & 3] = pack2_f16(p0, p1);
      } else {
        const uint32_t both = pack2_bf16(p0, p1);
        pw[t][i / 8][(i / 2) & 3] = both;
        rest[t][i / 8][(i / 2) & 3] = pack2_bf16(p0 - __uint_as_float(both << 16), p1 - __uint_as_float(both & 0xFFFF0000u));
      }
    }
    st.l[t] += (sum[0] + sum[1]) * (WIDE ? kKv8WideInv : 1.f) * sc.inv_vs;
  }
  if constexpr (!WIDE) {
    v4u v[2][2];
    v[0][0] = load_v(0, 0);
    v[0][1] = load_v(0, 1);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      if (i + 1 < D / 16) {
        v[(i + 1) & 1][0] = load_v(i + 1, 0);
        v[(i + 1) & 1][1] = load_v(i + 1, 1);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < MT; ++t)
          st.u[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, v[i & 1][h]),
                                                                __builtin_bit_cast(v8h, pw[t][h]), st.u[t][i], 0, 0, 0);
    }
    return;
  }
  // Values past the sequence's end, or of a block that is not there, may be
  // anything: zero them.  A NaN of a token that some rows see and others do
  // not must reach the former only, and 0 * NaN would reach both: such values
  // are zeroed, and a second product counts, per row and dimension, the NaN
  // that the row sees.
  uint32_t keep[8];  // of each pair of the lane's 16 keys
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = sc.there ? kv - (run_v + 2 * i) : 0;
    keep[i] = (n >= 2 ? 0xFFFFFFFFu : n == 1 ? 0xFFFFu : 0u) & kKv8Halves;
  }
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    __builtin_amdgcn_sched_barrier(0);
    v4u w[2] = {load_v(i, 0), load_v(i, 1)};
    uint32_t bad = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e / 4][e % 4] = f16_to_small_bf16(w[e / 4][e % 4], keep[e]);
      bad |= small_bf16_nans(w[e / 4][e % 4]);
    }
    if (__any(bad != 0)) {
      v4u ind[2];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t nan = small_bf16_nans(w[e / 4][e % 4]);
        w[e / 4][e % 4] &= ~(nan * 0xFFFFu);
        ind[e / 4][e % 4] = nan * 0x3F80u;
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        v4f cnt = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v4u sw;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sw[e] = (seen[t] >> (8 * h + 2 * e) & 1u) * 0x3F80u | (seen[t] >> (8 * h + 2 * e + 1) & 1u) * 0x3F800000u;
          cnt = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, ind[h]), __builtin_bit_cast(v8bf, sw),
                                                       cnt, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) st.u[t][i][e] = cnt[e] > 0.f ? __builtin_nanf("") : st.u[t][i][e];
      }
    }
    const v8bf v0 = __builtin_bit_cast(v8bf, w[0]), v1 = __builtin_bit_cast(v8bf, w[1]);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      v4f u = st.u[t][i];
      u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, __builtin_bit_cast(v8bf, rest[t][0]), u, 0, 0, 0);
      u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, __builtin_bit_cast(v8bf, rest[t][1]), u, 0, 0, 0);
      u = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, __builtin_bit_cast(v8bf, pw[t][0]), u, 0, 0, 0);
      st.u[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, __builtin_bit_cast(v8bf, pw[t][1]), u, 0, 0, 0);
    }
  }
}

// The raw products of a step of 64 keys with 16 MT rows.  load_k(j, h, o) gives
// the lane's values h * 64 + 16 g + 8 o .. of key (a / 4) * 16 + 4 j + a % 4,
// load_q(t, i) B fragment i of the lane's row of tile t.
template <int D, int MT, class LoadQ, class LoadK>
__device__ __forceinline__ void kv8_scores(float (&s)[MT][16], LoadQ load_q, LoadK load_k) {
  v8bf qf[MT][D / 32];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < D / 32; ++i) qf[t][i] = load_q(t, i);
  // The next product's operands are on their way while one runs; a fence a
  // product keeps the compiler from fetching more than registers hold.
  v8bf k[2][D / 32];
  auto fetch = [&](int j) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) k[j & 1][i] = load_k(j, i / 2, i % 2);
  };
  fetch(0);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j + 1 < 4) fetch(j + 1);
    __builtin_amdgcn_sched_barrier(0);
    v4f acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int t = 0; t < MT; ++t)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[j & 1][i], qf[t][i], acc[t], 0, 0, 0);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][4 * j + e] = acc[t][e];
  }
  __builtin_amdgcn_sched_barrier(0);
}

// The B fragments of one row of q.
template <int D>
__device__ __forceinline__ void kv8_load_q(const Kv8AttnParams& p, const Kv8Seq& sq, int head, int row, v8bf (&qf)[D / 32]) {
  const int g = (threadIdx.x & 63) >> 4;
  const uint16_t* src = p.q + (long long)(sq.first + row / p.group) * p.q_stride +
                        (long long)(head * p.group + row % p.group) * D + g * 16;
#pragma unroll
  for (int h = 0; h < D / 64; ++h) {
    qf[2 * h] = __builtin_bit_cast(v8bf, *(const v4u*)(src + h * 64));
    qf[2 * h + 1] = __builtin_bit_cast(v8bf, *(const v4u*)(src + h * 64 + 8));
  }
}

// Whether a step from token `base` on needs masks, given the keys [all_lo,
// all_hi) that every row sees (all_hi is at most kv).
__device__ __forceinline__ bool kv8_masked(int base, int all_lo, int all_hi) {
  return base < all_lo || base + kKv8Step > all_hi;
}

// A wave's loads of one step straight from the cache into registers.
template <int D>
struct Kv8Regs {
  v4u k[4][D / 64], v[D / 16];

  __device__ __forceinline__ void load_k(const Kv8Cache& c, int head, int base, int page) {
    const int lane = threadIdx.x & 63, a = lane & 15, g = lane >> 4;
    const int run = base + (a >> 2) * 16;
    const uint8_t* src = c.k_codes + ((size_t)max(page, 0) * c.h_kv + head) * (size_t)(c.block * D) +
                         (((run & (c.block - 1)) + (a & 3)) * D + g * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < D / 64; ++h) k[j][h] = *(const v4u*)(src + j * 4 * D + h * 64);
  }
  __device__ __forceinline__ void load_v(const Kv8Cache& c, int head, int base, int page) {
    const int lane = threadIdx.x & 63, a = lane & 15, g = lane >> 4;
    const int run = base + g * 16;
    const uint8_t* src = c.v_codes + ((size_t)max(page, 0) * c.h_kv + head) * (size_t)(c.block * D) +
                         (a * c.block + (run & (c.block - 1)));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) v[i] = *(const v4u*)(src + i * 16 * c.block);
  }
};

// The blocks of this lane's runs in a step: of its row of K (keys (a / 4) * 16
// of the step on) and of its lane group (keys 16 g on).
__device__ __forceinline__ void kv8_pages(const Kv8Cache& c, int seq, int kv, int base, int* page_k, int* page_v) {
  const int lane = threadIdx.x & 63;
  const int run_k = base + ((lane & 15) >> 2) * 16, run_v = base + (lane >> 4) * 16;
  const int pk = kv8_page(c, seq, run_k), pv = kv8_page(c, seq, run_v);
  *page_k = run_k < kv ? pk : -1;
  *page_v = run_v < kv ? pv : -1;
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
// tile's steps wholly are written out; of the others, the last workgroup of a
// tile joins all parts.  The shares come from the lengths on the device:
// nothing of the launch depends on them, and the longest sequence spreads over
// as many workgroups as its part of the batch's keys is worth.
//
// Parts pass between XCDs, whose L2s do not see each other's lines, by stores
// and loads at agent scope (SC1): each thread waits until its stores are
// complete, a barrier and a relaxed counter at the same scope follow, and the
// workgroup that finds all others counted loads the parts, in workgroup order,
// after a barrier behind its own count.  A tile's counter is its first
// workgroup's: no other tile starts in that one and goes on.  (With a
// second kernel for the joining 1 x 777 keys took 11.4 us against 8.9, 32 x
// 4096 47 against 43, 4 x 65536 107 against 101.)
template <int D>
__global__ __launch_bounds__(256) void kv8_attn_kernel(Kv8AttnParams p) {
  constexpr int kPitch = D + 4;
  __shared__ float s_u[4][16][kPitch];
  __shared__ float s_m[4][16], s_l[4][16];
  __shared__ long long box[6];
  __shared__ int s_last;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, a = lane & 15, g = lane >> 4;
  // rows of sequences without keys
  for (int i = blockIdx.x; i < p.batch; i += p.workers) {
    const Kv8Seq s = kv8_seq(p, i);
    if (s.steps > 0) continue;
    for (int e = tid; e < s.count * p.h_q * (D / 2); e += 256)
      ((uint32_t*)p.out)[(size_t)s.first * p.h_q * (D / 2) + e] = 0u;
    if (p.lse)
      for (int e = tid; e < s.count * p.h_q; e += 256) p.lse[(size_t)s.first * p.h_q + e] = -__builtin_huge_valf();
  }
  const Kv8Chunk chunk = kv8_chunk(p, 0, box);
  long long total = chunk.total;
  for (int i = 256; i < p.batch; i += 256) total += kv8_chunk(p, i, box).total;
  const long long share = kv8_share(p, total);
  const long long begin = blockIdx.x * share, end = min(begin + share, total);
  if (begin >= end) return;
  long long at = begin;
  int seq;
  long long seq0;  // first unit of seq
  kv8_find(p, chunk, at, &seq, &seq0, box);
  Kv8Seq sq = kv8_seq(p, seq);
  long long units = kv8_units(p, sq);
  const __amdgpu_buffer_rsrc_t rs_u =
      __builtin_amdgcn_make_buffer_rsrc(p.part_u, 0, p.workers * 2 * 16 * D * 4, kBufferRsrcWord3);
  const __amdgpu_buffer_rsrc_t rs_ml =
      __builtin_amdgcn_make_buffer_rsrc(p.part_ml, 0, p.workers * 2 * 16 * 2 * 4, kBufferRsrcWord3);
  while (at < end) {
    while (at >= seq0 + units) {
      seq0 += units;
      ++seq;
      sq = kv8_seq(p, seq);
      units = kv8_units(p, sq);
    }
    const long long rel = at - seq0;
    const int tile_no = (int)kv8_div(rel, sq.steps);
    const int head = tile_no / sq.tiles, tile = tile_no % sq.tiles;
    const int t0 = (int)(rel - (long long)tile_no * sq.steps);
    const int t1 = (int)min((long long)sq.steps, t0 + (end - at));

    // this lane's row: its query, and the keys it sees
    const int rows = sq.count * p.group, row = min(tile * 16 + a, rows - 1);
    v8bf qf[1][D / 32];
    kv8_load_q<D>(p, sq, head, row, qf[0]);
    Kv8Rows<1> see;
    kv8_sees(p, sq, row / p.group, &see.lo[0], &see.hi[0]);
    // keys that every row of the tile sees, and that any row sees
    int all_lo, all_hi, any_lo, any_hi;
    kv8_sees(p, sq, min(tile * 16 + 15, rows - 1) / p.group, &all_lo, &any_hi);
    kv8_sees(p, sq, tile * 16 / p.group, &any_lo, &all_hi);
    Kv8State<D, 1> st;
    st.clear();
    // Steps that any row sees.  K of the next step is loaded as soon as this
    // step's product has freed its registers, and so is V: each is in flight
    // while the rest of the step computes.
    const int first = max(t0, any_lo / kKv8Step - sq.step0) + wave;
    const int last = min(t1, (any_hi + kKv8Step - 1) / kKv8Step - sq.step0);
    if (first < last) {
      Kv8Regs<D> regs;
      float top = -__builtin_huge_valf();  // log2 of the largest value scale so far
      int base = (sq.step0 + first) * kKv8Step, pk, pv, next_pk, next_pv;
      kv8_pages(p.c, seq, sq.kv, base, &pk, &pv);
      kv8_pages(p.c, seq, sq.kv, base + 4 * kKv8Step, &next_pk, &next_pv);
      regs.load_k(p.c, head, base, pk);
      Kv8Run run = kv8_run(p.c, head, pv);
      regs.load_v(p.c, head, base, pv);
      for (int t = first; t < last; t += 4) {
        const bool more = t + 4 < last;
        const Kv8Scale now = kv8_scale_of(run, p.scale_log2);
        const int here = base;
        base += 4 * kKv8Step;
        pk = next_pk;
        pv = next_pv;
        kv8_pages(p.c, seq, sq.kv, base + 4 * kKv8Step, &next_pk, &next_pv);
        float scores[1][16];
        kv8_scores<D, 1>(scores, [&](int t, int i) { return qf[t][i]; }, [&](int j, int h, int o) {
          return e4m3_to_bf16(regs.k[j][h][2 * o], regs.k[j][h][2 * o + 1]);
        });
        auto rest = [&](auto form) {
          kv8_rest_of_step<D, 1, decltype(form)::value>(sq.kv, here + g * 16, now, see, scores, st, [&](int i, int o) {
            if (i == 0 && o == 0 && more) {
              regs.load_k(p.c, head, base, pk);
              run = kv8_run(p.c, head, pv);
            }
            return __builtin_bit_cast(v4u, e4m3_to_f16(regs.v[i][2 * o], regs.v[i][2 * o + 1]));
          });
        };
        // decided after the scores, when the scales are there (before them 32 x
        // 4096 took 46.6 us against 44.4, with heads of 64 30.6 against 27.3)
        const bool far = kv8_far(now, top);
        if (far || kv8_masked(here, all_lo, all_hi)) rest(std::true_type{}); else rest(std::false_type{});
        if (more) regs.load_v(p.c, head, base, pv);
      }
    }
    // the waves' states, merged in LDS
    st.l[0] += __shfl_xor(st.l[0], 16, 64);
    st.l[0] += __shfl_xor(st.l[0], 32, 64);
    __syncthreads();
    if (g == 0) {
      s_m[wave][a] = st.m[0];
      s_l[wave][a] = st.l[0];
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) *(v4f*)&s_u[wave][a][i * 16 + g * 4] = st.u[0][i];
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
        const int slot = ((int)blockIdx.x * 2 + (at == begin ? 0 : 1)) * 16 + r;
        const bool live = tile * 16 + r < rows;
        if (live) {
#pragma unroll
          for (int i = 0; i < D / 16; i += 4)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v4f{u[i], u[i + 1], u[i + 2], u[i + 3]}), rs_u,
                                                   (slot * D + part * (D / 16) + i) * 4, 0, kCpolSc1);
          if (part == 0)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(v2u, v2f{m, l}), rs_ml, slot * 8, 0, kCpolSc1);
        }
        // the tile's steps, and the workgroups that have some of them
        const long long s0 = seq0 + (long long)tile_no * sq.steps;
        const int w0 = (int)kv8_div(s0, share), w1 = (int)kv8_div(s0 + sq.steps - 1, share);
        wait_vmem_all();
        __syncthreads();
        if (tid == 0)
          s_last = __hip_atomic_fetch_add(p.arrived + w0, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == w1 - w0;
        __syncthreads();
        if (s_last) {
          if (tid == 0) __hip_atomic_store(p.arrived + w0, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);  // for the next call
          // only the first of them can have had another tile before this one
          const int slot0 = (w0 * 2 + (s0 > w0 * share ? 1 : 0)) * 16 + r;
          auto slot_of = [&](int w) { return w == w0 ? slot0 : w * 32 + r; };
          auto load_ml = [&](int w) {
            const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs_ml, slot_of(w) * 8, 0, kCpolSc1);
            return __builtin_bit_cast(v2f, v);
          };
          if (live) {
            // reference and sum of the row: its 16 threads take every 16th part each
            m = -__builtin_huge_valf();
            for (int w = w0 + part; w <= w1; w += 16) m = fmaxf(m, load_ml(w)[0]);
#pragma unroll
            for (int s = 8; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor(m, s, 64));
            const float all = m == -__builtin_huge_valf() ? 0.f : m;
            l = 0.f;
            for (int w = w0 + part; w <= w1; w += 16) {
              const v2f ml = load_ml(w);
              l += ml[1] * __builtin_amdgcn_exp2f(ml[0] - all);
            }
#pragma unroll
            for (int s = 8; s >= 1; s >>= 1) l += __shfl_xor(l, s, 64);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) u[i] = 0.f;
#pragma unroll 4
            for (int w = w0; w <= w1; ++w) {
              const float f = __builtin_amdgcn_exp2f(load_ml(w)[0] - all);
#pragma unroll
              for (int i = 0; i < D / 16; i += 4) {
                const auto v = __builtin_amdgcn_raw_buffer_load_b128(rs_u, (slot_of(w) * D + part * (D / 16) + i) * 4, 0, kCpolSc1);
                const v4f x = __builtin_bit_cast(v4f, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) u[i + e] += x[e] * f;
              }
            }
          }
          kv8_write<D>(p, sq, head, tile * 16 + r, part, u, m, l);
        }
      }
    }
    at += t1 - t0;
  }
}

// Where the 16-byte piece `part` of row `row` lies in an LDS tile of rows of
// `kParts` pieces (a multiple of 8): the 16 lanes that read one piece each of
// rows 0..15 of a tile then fall on all 64 banks once.
template <int kParts>
__device__ __forceinline__ int kv8_slot(int row, int part) {
  return row * kParts + (part ^ (kParts == 8 ? (row >> 1) & 7 : row & 15));
}

// Prompts: one workgroup takes 64 MT rows of one key/value head, 16 MT of them
// a wave, and walks all keys that they see.  Each step's codes are widened once
// for the four waves (K to bf16, V to fp16) on their way to LDS, in two
// buffers: while one is worked on, the next step's pieces are on their way to
// registers, and from there to the other.  (Codes in LDS, widened by each wave,
// take a quarter less LDS time but 96 more of some 400 vector instructions a
// step: 308 us for prompts of 2048; widened, and fetched one product ahead,
// 293.) Wave w
// brings keys 16 w .. 16 w + 15 of a step, K and V: they are of one block, so
// its number, its scales and all addresses are uniform in the wave.
template <int D, int MT>
__global__ __launch_bounds__(256, 2) void kv8_prompt_kernel(Kv8AttnParams p) {
  constexpr int kRows = 64 * MT, kParts = D / 8, kPer = D / 64;
  __shared__ v4u s_k[2][64 * kParts], s_v[2][D * 8];  // pieces of 8 values
  __shared__ Kv8Scale s_scale[2][4];
  __shared__ float s_vs[4][2];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, a = lane & 15, g = lane >> 4;
  const int head = blockIdx.x, seq = blockIdx.y;
  const Kv8Seq sq = kv8_seq(p, seq);
  const int rows = sq.count * p.group;
  // every sequence's last tile, which sees the most keys, starts first
  const int row0 = ((rows + kRows - 1) / kRows - 1 - (int)blockIdx.z) * kRows;
  if (row0 < 0) return;
  const Kv8Cache& c = p.c;

  // keys that any row of the workgroup sees, that all see, and that any of this wave's rows sees
  int any_lo, any_hi, all_lo, all_hi, wave_lo = 0, wave_hi = 0, unused;
  kv8_sees(p, sq, row0 / p.group, &any_lo, &all_hi);
  kv8_sees(p, sq, (min(row0 + kRows, rows) - 1) / p.group, &all_lo, &any_hi);
  const int wave0 = row0 + wave * 16 * MT, wave1 = min(wave0 + 16 * MT, rows) - 1;  // none if wave0 > wave1
  if (wave0 <= wave1) {
    kv8_sees(p, sq, wave1 / p.group, &unused, &wave_hi);
    kv8_sees(p, sq, wave0 / p.group, &wave_lo, &unused);
  }
  v8bf qf[MT][D / 32];
  Kv8Rows<MT> see;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int row = min(wave0 + t * 16 + a, rows - 1);
    kv8_load_q<D>(p, sq, head, row, qf[t]);
    kv8_sees(p, sq, row / p.group, &see.lo[t], &see.hi[t]);
  }
  Kv8State<D, MT> st;
  st.clear();

  // This wave's 16 keys of a step.  The table is read two steps ahead and the
  // scales one, by vector loads although they are uniform: scalar loads share
  // their counter with LDS, whose every wait would wait for them.
  int zero = 0;
  asm("" : "+v"(zero));
  int found, page;
  Kv8Run run;
  v4u held_k[kPer], held_v[kPer];
  auto look = [&](int base) {
    found = c.table[(size_t)seq * c.max_blocks + min((base + wave * 16) >> c.block_log2, c.max_blocks - 1) + zero];
  };
  auto fetch = [&](int base) {
    const int key = base + wave * 16;
    const int at = __builtin_amdgcn_readfirstlane(found);
    page = (key < sq.kv) & ((unsigned)at < (unsigned)c.num_blocks) ? at : -1;
    look(base + kKv8Step);
    const size_t tile = (size_t)max(page, 0) * c.h_kv + head;
    run = Kv8Run{page, c.k_scales[tile + zero], c.v_scales[tile + zero]};
    const uint8_t* k = c.k_codes + tile * (size_t)(c.block * D) + (key & (c.block - 1)) * D;
    const uint8_t* v = c.v_codes + tile * (size_t)(c.block * D) + (key & (c.block - 1));
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      held_k[i] = *(const v4u*)(k + (uint32_t)((lane + 64 * i) * 16));
      held_v[i] = *(const v4u*)(v + (uint32_t)((lane + 64 * i) * c.block));
    }
  };
  // Keys of a block that the table does not have become zeros with lv = -inf:
  // p = 0, without a mask.
  auto put = [&](int buf) {
    const uint32_t keep = page < 0 ? 0u : 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int key = (lane + 64 * i) / (D / 16), part = (lane + 64 * i) % (D / 16) * 2;
      // row 16 j + a of the tile is the key that lane a takes in product j
      const int row = (key >> 2) * 16 + wave * 4 + (key & 3);
      const v4u k = held_k[i] & keep, v = held_v[i] & keep;
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        s_k[buf][kv8_slot<kParts>(row, part + o)] = __builtin_bit_cast(v4u, e4m3_to_bf16(k[2 * o], k[2 * o + 1]));
        s_v[buf][kv8_slot<8>(lane + 64 * i, wave * 2 + o)] = __builtin_bit_cast(v4u, e4m3_to_f16(v[2 * o], v[2 * o + 1]));
      }
    }
    if (lane == 0) {
      Kv8Scale sc = kv8_scale_of(run, p.scale_log2);
      if (page < 0) sc = Kv8Scale{0.f, -__builtin_huge_valf(), 1.f, 0};
      s_scale[buf][wave] = sc;
    }
  };
  const int first = any_lo / kKv8Step, last = (any_hi + kKv8Step - 1) / kKv8Step;
  if (first < last) {
    look(first * kKv8Step);
    fetch(first * kKv8Step);
    // the smallest and the largest value scale of the blocks that the workgroup sees
    float least = __builtin_huge_valf(), most = 0.f;
    const int j1 = min((min(any_hi, sq.kv) - 1) >> c.block_log2, c.max_blocks - 1);
#pragma unroll 4
    for (int j = (any_lo >> c.block_log2) + tid; j <= j1; j += 256) {
      const int at = c.table[(size_t)seq * c.max_blocks + j];
      if ((unsigned)at >= (unsigned)c.num_blocks) continue;
      const float vs = fmaxf(c.v_scales[(size_t)at * c.h_kv + head], kKv8MinVs);
      least = fminf(least, vs);
      most = fmaxf(most, vs);
    }
#pragma unroll
    for (int i = 32; i >= 1; i >>= 1) {
      least = fminf(least, __shfl_xor(least, i, 64));
      most = fmaxf(most, __shfl_xor(most, i, 64));
    }
    if (lane == 0) {
      s_vs[wave][0] = least;
      s_vs[wave][1] = most;
    }
    put(0);
    __syncthreads();
    int s = first;
    auto steps = [&](int until, auto form) {
#pragma unroll 1
      for (; s < until; ++s) {
        const int base = s * kKv8Step, buf = (s - first) & 1;
        fetch(base + kKv8Step);  // past the last step: no block, or one that nobody will use
        if (base < wave_hi && base + kKv8Step > wave_lo) {
          const v4u* k_at = s_k[buf];
          const v4u* v_at = s_v[buf];
          const Kv8Scale now = s_scale[buf][g];
          float scores[MT][16];
          kv8_scores<D, MT>(scores, [&](int t, int i) { return qf[t][i]; }, [&](int j, int h, int o) {
            return __builtin_bit_cast(v8bf, k_at[kv8_slot<kParts>(j * 16 + a, h * 8 + g * 2 + o)]);
          });
          kv8_rest_of_step<D, MT, decltype(form)::value>(sq.kv, base + g * 16, now, see, scores, st, [&](int i, int o) {
            return v_at[kv8_slot<8>(i * 16 + a, g * 2 + o)];
          });
        }
        put(buf ^ 1);
        __syncthreads();
      }
    };
    // Wide steps, steps that every row of the workgroup sees wholly, wide
    // steps; all wide if value scales are far apart.  (Decided for each step,
    // from LDS and before its first product, it took the narrow steps 4 %.)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      least = fminf(least, s_vs[w][0]);
      most = fmaxf(most, s_vs[w][1]);
    }
    const bool far = __any(most > least * kKv8NearRatio);  // uniform, and known to be
    const int whole0 = far ? last : min(max((all_lo + kKv8Step - 1) / kKv8Step, first), last);
    const int whole1 = max(all_hi / kKv8Step, whole0);
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
      steps(part == 0 ? whole0 : last, std::true_type{});
      if (part == 0) steps(min(whole1, last), std::false_type{});
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    float l = st.l[t];
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    const int row = wave0 + t * 16 + a;
    if (row >= rows) continue;
    const size_t at = (size_t)(sq.first + row / p.group) * p.h_q + head * p.group + row % p.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;  // l == 0: the row sees no key
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      *(v2u*)(p.out + at * D + i * 16 + g * 4) = v2u{pack2_bf16(st.u[t][i][0] * inv, st.u[t][i][1] * inv),
                                                     pack2_bf16(st.u[t][i][2] * inv, st.u[t][i][3] * inv)};
    if (p.lse && g == 0) p.lse[at] = (st.m[t] + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
  }
}

}  // namespace dg
