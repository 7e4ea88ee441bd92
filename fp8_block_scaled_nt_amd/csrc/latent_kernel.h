// Attention whose keys and values come from one shared latent vector a token,
// the paged cache of those vectors, and the rotation of their rope parts.
//
// A token is a latent c of L values and a rope part r of P = L / 8 values,
// both shared by all heads:
//
//   latent [num_blocks][block][L]   bf16, or e4m3 codes with
//   scales [num_blocks][block][L / 128], powers of two, for each token and 128 values
//   rope   [num_blocks][block][P]   bf16
//
// Absorbed, a head's key is (c, r) and its value c.  Expanded, an
// up-projection gives each head a key part and a value of L / 4 values each.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_kernel.h"
#include "kv8_kernel.h"
#include "quant_kernel.h"
#include "w4_kernel.h"

namespace dg {

struct LatentCache {
  uint8_t* latent;  // bf16 or e4m3
  uint16_t* rope;
  float* scales;        // null: latents are bf16
  const int32_t* table;  // [batch][max_blocks]
  int block, block_log2, num_blocks, max_blocks;
};

// The block of sequence `seq` that holds token `token` >= 0, or -1 where the table has none.
__device__ __forceinline__ int latent_page(const LatentCache& c, int seq, int token) {
  if (c.max_blocks == 0) return -1;
  const int j = token >> c.block_log2;
  const int page = c.table[(size_t)seq * c.max_blocks + min(j, c.max_blocks - 1)];
  return (j < c.max_blocks) & ((unsigned)page < (unsigned)c.num_blocks) ? page : -1;
}

// Which sequence packed row `row` is of, by the running sums cu: how many of
// cu[1..batch] it has passed.  The wave's lanes look at 64 of them at a time.
// batch: none.
__device__ __forceinline__ int latent_seq_of(const int32_t* cu, int batch, int row) {
  const int lane = threadIdx.x & 63;
  int seq = 0;
  for (int j = 0; j < batch; j += 64) {
    const int end = cu[min(j + lane, batch - 1) + 1];
    seq += __popcll(__ballot(j + lane < batch && end <= row));
  }
  return seq;
}

// ---- append

struct LatentAppendParams {
  const uint16_t* latent;  // bf16 rows, *_stride elements from token to token
  const uint16_t* rope;
  long long latent_stride, rope_stride;
  LatentCache c;
  const int32_t* ctx;
  const int32_t* cu;
  const float* angles;  // [positions][P]: P / 2 cosines, P / 2 sines
  int positions;
  const uint16_t* norm;  // bf16 [L] or null
  float eps;
  const uint16_t* q;  // rope parts of the queries, or null
  uint16_t* q_out;
  long long q_stride, q_head_stride, q_out_stride, q_out_head_stride;
  int h_q, batch, total, most;
};

// Eight pairs (a, b) turned by their angles: (a cos - b sin, a sin + b cos) in
// fp32, rounded once.  PAIRS: x[0], x[1] hold them as neighbours, else x[0]
// the a's and x[1] the b's.
template <bool PAIRS>
__device__ __forceinline__ void latent_rotate(v4u (&x)[2], const v4f (&c)[2], const v4f (&n)[2]) {
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = x[i / 4][i % 4];
      const float a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xFFFF0000u);
      const float cs = c[i / 4][i % 4], sn = n[i / 4][i % 4];
      x[i / 4][i % 4] = pack2_bf16(a * cs - b * sn, a * sn + b * cs);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t wa = x[0][i], wb = x[1][i];
      const float a0 = __uint_as_float(wa << 16), a1 = __uint_as_float(wa & 0xFFFF0000u);
      const float b0 = __uint_as_float(wb << 16), b1 = __uint_as_float(wb & 0xFFFF0000u);
      const float c0 = c[i / 2][2 * i % 4], c1 = c[i / 2][2 * i % 4 + 1];
      const float n0 = n[i / 2][2 * i % 4], n1 = n[i / 2][2 * i % 4 + 1];
      x[0][i] = pack2_bf16(a0 * c0 - b0 * n0, a1 * c1 - b1 * n1);
      x[1][i] = pack2_bf16(a0 * n0 + b0 * c0, a1 * n1 + b1 * c1);
    }
  }
}

// One wave takes one token: its latent, its rope part, and (blockIdx.y) some
// of the queries' heads.  A lane turns eight pairs of a head; the cosines and
// sines that it needs are the same for every head, so they are read once, and
// the norm's sum needs no LDS.  Few tokens are bound by the launch and a chain
// of loads (lengths, table, write): 64 tokens of 512, 8 heads 4.2 us.  Many are
// bound by memory: 4 prompts up to 4096 of 512 into e4m3, 32 heads 28.8 us, 121
// MB read and written (4.2 TB/s).
constexpr int kLatentHeads = 32;  // query heads of one wave

template <int L, bool F8, bool PAIRS>
__global__ __launch_bounds__(256) void latent_append_kernel(LatentAppendParams p) {
  constexpr int P = L / 8, kPer = P / 16;  // lanes of one head
  const int lane = threadIdx.x & 63;
  const int t = __builtin_amdgcn_readfirstlane((int)blockIdx.x * 4 + (int)(threadIdx.x >> 6));
  if (t >= p.total) return;
  const int j = lane % kPer;
  const bool first = blockIdx.y == 0;
  // everything that does not hang on the token's place is on its way before it is known
  v4u x = {0, 0, 0, 0};
  if (first && lane * 8 < L) x = *(const v4u*)(p.latent + (long long)t * p.latent_stride + lane * 8);
  const int seq = __builtin_amdgcn_readfirstlane(latent_seq_of(p.cu, p.batch, t));
  if (seq >= p.batch) return;
  const int i = t - p.cu[seq];
  if (i < 0 || i >= p.most) return;
  const long long pos64 = (long long)p.ctx[seq] + i;
  if (pos64 < 0 || pos64 >= p.positions) return;
  const int pos = (int)pos64;
  const float* at = p.angles + (size_t)pos * P + j * 8;
  const v4f cs[2] = {*(const v4f*)at, *(const v4f*)(at + 4)};
  const v4f sn[2] = {*(const v4f*)(at + P / 2), *(const v4f*)(at + P / 2 + 4)};
  const int o0 = PAIRS ? j * 16 : j * 8, o1 = PAIRS ? j * 16 + 8 : P / 2 + j * 8;
  if (p.q) {
    const int last = min((int)(blockIdx.y + 1) * kLatentHeads, p.h_q);
#pragma unroll 2
    for (int h = blockIdx.y * kLatentHeads + lane / kPer; h < last; h += 64 / kPer) {
      const uint16_t* src = p.q + (long long)t * p.q_stride + (long long)h * p.q_head_stride;
      uint16_t* dst = p.q_out + (long long)t * p.q_out_stride + (long long)h * p.q_out_head_stride;
      v4u y[2] = {*(const v4u*)(src + o0), *(const v4u*)(src + o1)};
      latent_rotate<PAIRS>(y, cs, sn);
      *(v4u*)(dst + o0) = y[0];
      *(v4u*)(dst + o1) = y[1];
    }
  }
  if (!first) return;
  const int page = latent_page(p.c, seq, pos);
  if (page < 0) return;
  const size_t row = ((size_t)page << p.c.block_log2) + (pos & (p.c.block - 1));
  if (lane < kPer) {
    const uint16_t* src = p.rope + (long long)t * p.rope_stride;
    v4u y[2] = {*(const v4u*)(src + o0), *(const v4u*)(src + o1)};
    latent_rotate<PAIRS>(y, cs, sn);
    *(v4u*)(p.c.rope + row * P + o0) = y[0];
    *(v4u*)(p.c.rope + row * P + o1) = y[1];
  }
  if (p.norm || F8) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(x[e] << 16);
      v[2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
    }
    if (p.norm) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[e] * v[e];
#pragma unroll
      for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s, 64);
      const float inv = 1.f / sqrtf(sum * (1.f / L) + p.eps);
      const v4u w = *(const v4u*)(p.norm + lane * 8 % L);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = v[e] * inv * __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
    if constexpr (F8) {
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]) < __builtin_huge_valf() ? fabsf(v[e]) : 0.f);
#pragma unroll
      for (int s = 8; s >= 1; s >>= 1) amax = fmaxf(amax, __shfl_xor(amax, s, 64));
      const float scale = kv8_scale(amax), inv = 1.f / scale;  // powers of two
      if (lane * 8 < L) {
        *(uint2*)(p.c.latent + row * L + lane * 8) =
            make_uint2(kv8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                       kv8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
        if (lane % 16 == 0) p.c.scales[row * (L / 128) + lane / 16] = scale;
      }
      return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pack2_bf16(v[2 * e], v[2 * e + 1]);
  }
  if constexpr (!F8)
    if (lane * 8 < L) *(v4u*)(p.c.latent + (row * L + lane * 8) * 2) = x;
}

// ---- gather

struct LatentGatherParams {
  LatentCache c;
  const int32_t* starts;  // first token of each sequence, or null: 0
  const int32_t* cu;
  uint16_t* latent;  // bf16 [total][L]
  uint16_t* rope;    // bf16 [total][P]
  int batch, total;
};

// Eight codes times a power of two, as bf16: exact but for results outside bf16's range.
__device__ __forceinline__ v4u latent_widen(uint32_t lo, uint32_t hi, float scale) {
  v4u r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true));
  return r;
}

// One wave takes eight rows; a lane takes 16 bytes of a token at a time, so
// that a load brings 1 KB of one to four tokens, and all of them are on their
// way together.  Bound by memory: 4 x up to 32768 tokens of 512 out of e4m3 40.3
// us, 4.2 TB/s read and written (one row a wave 46.5 us a call); 7 x up to 777 of
// 256 3.6 us, the launch and a chain of three loads.
constexpr int kLatentGather = 8;  // rows of a wave

template <int L, bool F8>
__global__ __launch_bounds__(256) void latent_gather_kernel(LatentGatherParams p) {
  constexpr int P = L / 8, kLanes = F8 ? L / 16 : L / 8, kAt = 64 / kLanes;  // lanes of a token, tokens of a load
  const int lane = threadIdx.x & 63;
  const int row0 = __builtin_amdgcn_readfirstlane(((int)blockIdx.x * 4 + (int)(threadIdx.x >> 6)) * kLatentGather);
  if (row0 >= p.total) return;
  const int seq0 = __builtin_amdgcn_readfirstlane(latent_seq_of(p.cu, p.batch, row0));
  // where row t lies in the cache, or -1
  auto place = [&](int t) -> long long {
    int seq = seq0;
    while (seq < p.batch && p.cu[seq + 1] <= t) ++seq;  // as a rule none: t is of the wave's first sequence
    if (t >= p.total || seq >= p.batch) return -1;
    const int i = t - p.cu[seq];
    const long long pos = (long long)(p.starts ? p.starts[seq] : 0) + i;
    if (i < 0 || pos < 0 || pos > 0x7FFFFFFFLL) return -1;
    const int page = latent_page(p.c, seq, (int)pos);
    return page < 0 ? -1 : ((long long)page << p.c.block_log2) + ((int)pos & (p.c.block - 1));
  };
  // lane t of the first eight finds row t's place for all
  const long long mine = place(row0 + lane % kLatentGather);
  auto place_of = [&](int t) { return __shfl(mine, t, 64); };
  v4u x[kLatentGather / kAt];
  float scale[kLatentGather / kAt];
  const int part = lane % kLanes;
#pragma unroll
  for (int i = 0; i < kLatentGather / kAt; ++i) {
    const long long at = max(place_of(i * kAt + lane / kLanes), 0LL);  // some token there is: its bytes are not kept
    x[i] = *(const v4u*)(p.c.latent + at * (F8 ? L : 2 * L) + part * 16);
    if constexpr (F8) scale[i] = p.c.scales[at * (L / 128) + part / 8];
  }
  constexpr int kRopeLanes = P / 8, kRopeAt = 64 / kRopeLanes < kLatentGather ? 64 / kRopeLanes : kLatentGather;
  const int r = lane / kRopeLanes % kRopeAt;
  const long long rope_at = place_of(r);
  const v4u rope = *(const v4u*)(p.c.rope + max(rope_at, 0LL) * P + lane % kRopeLanes * 8);
  if (rope_at >= 0 && lane < kRopeAt * kRopeLanes) *(v4u*)(p.rope + (size_t)(row0 + r) * P + lane % kRopeLanes * 8) = rope;
#pragma unroll
  for (int i = 0; i < kLatentGather / kAt; ++i) {
    const int t = i * kAt + lane / kLanes;
    if (place_of(t) < 0) continue;
    uint16_t* const to = p.latent + (size_t)(row0 + t) * L + part * (F8 ? 16 : 8);
    if constexpr (F8) {
      *(v4u*)to = latent_widen(x[i][0], x[i][1], scale[i]);
      *(v4u*)(to + 8) = latent_widen(x[i][2], x[i][3], scale[i]);
    } else {
      *(v4u*)to = x[i];
    }
  }
}

// ---- attention, absorbed
//
//   x[j] = scale * (ql . c[j] + qr . r[j])   over the tokens j that the row sees
//   o    = sum_j e^(x[j] - lse) c[j],  lse = log sum_j e^x[j]
//
// Rows are (query, head) pairs of one sequence, row = query * h_q + head: all
// of them read the same tokens, once.  Per row the kernel carries a reference
// m, u = sum_j 2^(t[j] - m) c[j] and l = sum_j 2^(t[j] - m) in fp32, with
// t[j] = log2(e) x[j].  m stands kLatentLead above the row's largest t when it
// was set and moves when some t passes it: p never passes 1, and few steps pay
// for scaling u.

// A tile that a workgroup began and did not finish: how many parts it has, and
// where the first lies.
struct LatentCut {
  int seq, tile, parts, slot;
};

struct LatentAttnParams {
  const uint16_t* q;   // bf16 latent parts of the queries
  const uint16_t* qr;  // and their rope parts
  long long q_stride, q_head_stride, qr_stride, qr_head_stride;
  LatentCache c;
  const int32_t* kv_lens;
  const int32_t* cu;
  uint16_t* out;  // bf16
  long long out_stride, out_head_stride;
  float* lse;  // [total][h_q] or null
  float scale_log2;
  int causal, batch, total, most, h_q;
  // split work: workgroup w computes its share of the units below
  float* part_u;   // [workers][2][rows of a tile][L], as the lanes hold it
  float* part_ml;  // [workers][2][rows of a tile][2]: m and l
  LatentCut* cut;  // [workers]
  int workers;
  int together;  // > 1: every sequence has so many tiles, and as many neighbouring workgroups take the same steps of each
};

constexpr int kLatentStep = 64;       // tokens of one step
constexpr float kLatentLead = 8.f;    // log2 of how far the reference is put above the largest score
constexpr float kLatentLow = -3e38f;  // the reference of a row that has seen no token: any score passes it

// How LDS rows of tokens are turned so that neither the 16 tokens of a row
// fragment nor the 8 tokens that a transposing read covers at a time meet in a
// bank: 16-byte piece s of token t lies in slot s ^ latent_turn(t).
__device__ __forceinline__ int latent_turn(int t) { return (t & 3) << 1 | (t & 8) | (t >> 2 & 1); }

struct LatentSeq {
  int first, count;  // its queries
  int kv;            // its tokens that the table has room for
  int pos;           // where its first query stands (negative: before the cache)
  int steps, tiles;
};

template <int ROWS>
__device__ __forceinline__ LatentSeq latent_seq(const LatentAttnParams& p, int seq) {
  LatentSeq s;
  const int all = kv8_rows(p.cu, seq, p.total, p.most, &s.first, &s.count);
  const long long room = (long long)p.c.max_blocks << p.c.block_log2;
  const int kv = max(p.kv_lens[seq], 0);
  s.kv = kv < room ? kv : (int)room;
  s.pos = kv - all;
  s.steps = (s.kv + kLatentStep - 1) / kLatentStep;
  s.tiles = (s.count * p.h_q + ROWS - 1) / ROWS;
  return s;
}

// The same in scalar registers, where `seq` is uniform.
__device__ __forceinline__ int latent_uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
template <int ROWS>
__device__ __forceinline__ LatentSeq latent_seq_uniform(const LatentAttnParams& p, int seq) {
  const LatentSeq s = latent_seq<ROWS>(p, seq);
  return LatentSeq{latent_uniform(s.first), latent_uniform(s.count), latent_uniform(s.kv),
                   latent_uniform(s.pos), latent_uniform(s.steps), latent_uniform(s.tiles)};
}

// Tokens [0, hi) that query `i` of the sequence sees.
__device__ __forceinline__ int latent_sees(const LatentAttnParams& p, const LatentSeq& s, int i) {
  return p.causal ? max(min(s.pos + i + 1, s.kv), 0) : s.kv;
}

// Consecutive shares go to one XCD, so that the tiles of one sequence find its
// tokens in that XCD's L2.
__device__ __forceinline__ int latent_worker(int block, int workers) {
  return workers % kNumXcd == 0 ? block % kNumXcd * (workers / kNumXcd) + block / kNumXcd : block;
}

// Channels col + 16 c .. + 3 of one row: u / l; l == 0: the row sees no token.
template <int L, int C>
__device__ __forceinline__ void latent_write(const LatentAttnParams& p, const LatentSeq& sq, int row, int col,
                                             const v4f (&u)[C], float m, float l, bool with_lse) {
  const int i = row / p.h_q, head = row - i * p.h_q;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* const to = p.out + (long long)(sq.first + i) * p.out_stride + (long long)head * p.out_head_stride + col;
#pragma unroll
  for (int c = 0; c < C; ++c)
    *(v2u*)(to + c * 16) = v2u{pack2_bf16(u[c][0] * inv, u[c][1] * inv), pack2_bf16(u[c][2] * inv, u[c][3] * inv)};
  if (p.lse && with_lse)
    p.lse[(size_t)(sq.first + i) * p.h_q + head] =
        l == 0.f ? -__builtin_huge_valf() : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
}

// The halves of a dword of two bf16 that are finite; the others become zero.
__device__ __forceinline__ uint32_t bf16_finite(uint32_t w) {
  w = (w & 0x7F80u) == 0x7F80u ? w & 0xFFFF0000u : w;
  return (w & 0x7F800000u) == 0x7F800000u ? w & 0xFFFFu : w;
}

// 1 in bf16 for each half of a dword of two bf16 that is not finite, else 0.
__device__ __forceinline__ uint32_t bf16_not_finite(uint32_t w) {
  return ((w & 0x7F80u) == 0x7F80u ? 0x3F80u : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0x3F800000u : 0u);
}

typedef __attribute__((address_space(3))) v4u lds_v4u;
typedef __attribute__((address_space(3))) v2u lds_v2u;

// Four bf16 of one channel and four tokens, from token-major rows: lane i of
// 16 gives the address of four channels of token i / 4 and gets channel i.
__device__ __forceinline__ v2u lds_turned(uint32_t at) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(uintptr_t)at));
}

// A barrier that waits for this wave's LDS accesses, and not for the next
// step's DMA as __syncthreads() would.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  block_barrier();
}

// Ends a run of LDS DMAs: the load under EXEC = 0 that each of them begins
// with, so that the vector memory instruction behind the last one is such a
// load too, whatever the compiler puts there (see lds_dma16).
__device__ __forceinline__ void lds_dma_end(v4i_rsrc rs, uint32_t voff) {
  uint64_t exec_save;
  asm volatile("s_and_saveexec_b64 %0, 0\n\tbuffer_load_dword %1, %1, %2, 0 offen\n\ts_mov_b64 exec, %0"
               : "=&s"(exec_save) : "v"(voff), "s"(rs) : "memory", "scc");
}

// Eight wait states: what a vector instruction has to keep from the matrix
// instruction (16x16x32 in bf16, four passes) whose result it reads.  The asm has
// the results as operands, so it stands behind their products.  It is for products
// that a branch over a side block follows: the compiler looks for what still has
// to be waited for from the reader backwards, through the side block first, and
// does not pass the block before the branch a second time, so the way around the
// side block got no wait (the forms of 16 and 32 rows read scores after 2 to 7
// states, and now and then got what the last product had not added yet).
__device__ __forceinline__ void mfma_settle(v4f (&x)[1][1]) { asm volatile("s_nop 7" : "+v"(x[0][0])); }
__device__ __forceinline__ void mfma_settle(v4f (&x)[1][2]) { asm volatile("s_nop 7" : "+v"(x[0][0]), "+v"(x[0][1])); }
__device__ __forceinline__ void mfma_settle(v4f (&x)[2][2]) {
  asm volatile("s_nop 7" : "+v"(x[0][0]), "+v"(x[0][1]), "+v"(x[1][0]), "+v"(x[1][1]));
}

// LDS of the absorbed kernel, in bytes.
template <int L, bool F8, int NT>
struct LatentLds {
  static constexpr int P = L / 8;
  static constexpr int kRow = F8 ? L : 2 * L;                 // a token's latent as it lies in memory
  static constexpr int kLatent = kLatentStep * kRow;
  static constexpr int kRope = kLatentStep * P * 2;
  static constexpr int kScales = F8 ? 4 * 256 : 0;
  static constexpr int kBuffer = kLatent + kRope + kScales;   // two of them
  static constexpr int kWide = 2 * kBuffer;                   // e4m3: the step's latents in bf16
  static constexpr int kP = kWide + (F8 ? kLatentStep * L * 2 : 0);  // p [rows][64], bf16
  // the second pieces of p: [4][rows][16]; for L = 512 they go over the step's
  // rope parts once all waves are done with those
  static constexpr bool kRestOverRope = 16 * P * 2 >= 16 * NT * 32;
  static constexpr int kRest = kP + 16 * NT * 128;
  static constexpr int kMax = kRest + (kRestOverRope ? 0 : 4 * 16 * NT * 32);  // [4][rows] floats
  static constexpr int kFlags = kMax + 4 * 16 * NT * 4;       // [2] a reference moves, [2][4] a group's block is there, [2] a row sees a score of -inf
  static constexpr int kBox = kFlags + 64;
  static constexpr int kBytes = kBox + 64;
};

// A unit of work is a 64-token step of a tile of 16 NT rows; a workgroup of
// four waves takes an equal share of all units, in the order (sequence, tile,
// step).  In a step wave w sends for tokens 16 w .. 16 w + 15 of the next one, and
// has them in LDS at its end; their blocks are looked up four steps ahead.  For
// the scores the waves share out the tokens, and for
// more than 32 rows (RW = 2) tokens and rows, each half of both, as q for all
// rows would not fit in the registers beside u.  p passes through LDS, and
// wave w adds up channels w L / 4 .. of every row.  So a token's latent is
// fetched once for all heads, and q and u never leave the registers.
//
// Tiles that a share's end cuts leave their parts in the workspace, and
// latent_join_kernel adds them up.
//
// p meets c as bf16, 8 bits, as wide as c itself: its error, up to 2^-8 of each
// p and of either sign, is of the size of out's own rounding where a row weighs
// many values that cancel (against 64 bits, relative to all outputs, 0.0017 to
// 0.0023, where out's rounding alone gives 0.0016 to 0.0017) and less elsewhere;
// fp16 would not hold c's range, and a second piece would be another product.  A step that some row does not see
// wholly may be all that a row sees: there p goes in two pieces, 16 bits.
//
// What bounds it, by case (latents of 512, without the join): with few rows HBM -
// 64 x up to 8192 tokens, 16 rows each, bf16 77 us, 5 TB/s, at a copy's rate; with
// 128 rows the CU - 4 x 65536, bf16, 97 to 120 us from run to run as the clock goes;
// 99.7 us is 732 TFLOP/s, and a wave then has 209 thousand cycles (2.1 GHz) for 32
// steps: a third of MFMA, a fifth of VALU work, waits (LDS, barriers: p is shared
// between the waves) 31 %; 32 x up to 4096 in e4m3 59 us, where widening makes it
// 4.1 VALU instructions an MFMA instead of 2.4; 1 x 777 of 256 7.9 us, latency of
// the prologue.
template <int L, bool F8, int NT>
__global__ __launch_bounds__(256, 1) void latent_attn_kernel(LatentAttnParams p) {
  using Lds = LatentLds<L, F8, NT>;
  constexpr int P = L / 8, kRows = 16 * NT, kJ = L / 64, kC = L / 64;  // kC column tiles of 16 a wave
  constexpr int kRopeFrags = P / 32, RW = NT > 2 ? 2 : 1, kN = NT / RW;  // kN row tiles and RW token tiles of a wave's scores
  // u and q together pass the 256 registers that vector instructions reach: q
  // goes to the accumulation registers, where matrix instructions read it
  constexpr bool kQInAcc = NT * L >= 1024;
  extern __shared__ __align__(1024) uint8_t lds[];  // all of it: a row's place has to be a multiple of its size
  float* const s_max = (float*)(lds + Lds::kMax);
  int* const s_flag = (int*)(lds + Lds::kFlags);
  int* const s_there = s_flag + 2;
  int* const s_inf = s_there + 8;
  long long* const box = (long long*)(lds + Lds::kBox);
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, a = lane & 15, g = lane >> 4;
  const int rw = wave / (4 / RW), tw = wave % (4 / RW);

  // rows of sequences without tokens
  for (int i = blockIdx.x; i < p.batch; i += p.workers) {
    const LatentSeq s = latent_seq<kRows>(p, i);
    if (s.steps > 0) continue;
    for (int r = tid / (L / 8); r < s.count * p.h_q; r += 256 / (L / 8)) {
      const int token = s.first + r / p.h_q, head = r % p.h_q;
      *(v4u*)(p.out + token * p.out_stride + head * p.out_head_stride + tid % (L / 8) * 8) = v4u{0, 0, 0, 0};
      if (p.lse && tid % (L / 8) == 0) p.lse[(size_t)token * p.h_q + head] = -__builtin_huge_valf();
    }
  }
  if (tid == 0) p.cut[latent_worker(blockIdx.x, p.workers)] = LatentCut{0, 0, 0, 0};
  // together > 1: a unit is a step of all tiles, shared out to groups of workgroups that read the same tokens at a time
  auto units_of = [&](const LatentSeq& s) { return p.together > 1 ? (s.count > 0 ? (long long)s.steps : 0) : (long long)s.tiles * s.steps; };
  auto chunk_of = [&](int first) {
    const int i = first + tid;
    Kv8Chunk c;
    c.units = i < p.batch ? units_of(latent_seq<kRows>(p, i)) : 0;
    c.before = kv8_scan256(c.units, &c.total, box) - c.units;
    return c;
  };
  Kv8Chunk chunk = chunk_of(0);
  long long total = chunk.total;
  for (int i = 256; i < p.batch; i += 256) total += chunk_of(i).total;
  const int groups = p.workers / p.together;
  const long long share = max(kv8_div(total + groups - 1, groups), 1LL);
  const int worker = latent_worker(blockIdx.x, p.workers), group = worker / p.together;
  const long long begin = group * share, end = min(begin + share, total);
  if (group >= groups || begin >= end) return;
  // the sequence that the first unit is of
  long long at = begin, seq0 = 0;
  int seq;
  {
    long long carry = 0;
    int from = 0;
    while (at >= carry + chunk.total) {
      carry += chunk.total;
      from += 256;
      chunk = chunk_of(from);
    }
    const long long mine = carry + chunk.before;
    if (at >= mine && at < mine + chunk.units) {
      box[4] = from + tid;
      box[5] = mine;
    }
    __syncthreads();
    seq = __builtin_amdgcn_readfirstlane((int)box[4]);
    seq0 = box[5];
  }
  LatentSeq sq = latent_seq_uniform<kRows>(p, seq);
  long long units = units_of(sq);
  int zero = 0;
  asm("" : "+v"(zero));  // loads of the table by vector loads, although they are uniform

  while (at < end) {
    while (at >= seq0 + units) {
      seq0 += units;
      ++seq;
      sq = latent_seq_uniform<kRows>(p, seq);
      units = units_of(sq);
    }
    const long long rel = at - seq0;
    const int past = latent_uniform((int)kv8_div(rel, sq.steps));  // tiles before this one
    const int tile = p.together > 1 ? worker % p.together : past;
    const int t0 = latent_uniform((int)(rel - (long long)past * sq.steps));
    const int t1 = latent_uniform((int)min((long long)sq.steps, t0 + (end - at)));
    const int rows = sq.count * p.h_q, row0 = tile * kRows;

    // B fragments of this wave's rows, and how many tokens each sees
    v8bf qf[kN][2 * kJ], qrf[kN][kRopeFrags];
    int hi[kN];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int row = min(row0 + 16 * (rw * kN + n) + a, rows - 1), i = row / p.h_q, head = row - i * p.h_q;
      const uint16_t* src = p.q + (long long)(sq.first + i) * p.q_stride + (long long)head * p.q_head_stride + g * 16;
      const uint16_t* srcr = p.qr + (long long)(sq.first + i) * p.qr_stride + (long long)head * p.qr_head_stride + g * (P / 4);
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        qf[n][2 * j] = __builtin_bit_cast(v8bf, *(const v4u*)(src + j * 64));
        qf[n][2 * j + 1] = __builtin_bit_cast(v8bf, *(const v4u*)(src + j * 64 + 8));
      }
#pragma unroll
      for (int j = 0; j < kRopeFrags; ++j) qrf[n][j] = __builtin_bit_cast(v8bf, *(const v4u*)(srcr + j * 8));
      hi[n] = latent_sees(p, sq, i);
      if constexpr (kQInAcc) {
#pragma unroll
        for (int j = 0; j < 2 * kJ; ++j) asm("" : "+a"(qf[n][j]));
#pragma unroll
        for (int j = 0; j < kRopeFrags; ++j) asm("" : "+a"(qrf[n][j]));
      }
    }
    const int all_hi = latent_uniform(latent_sees(p, sq, row0 / p.h_q));
    const int any_hi = latent_uniform(latent_sees(p, sq, (min(row0 + kRows, rows) - 1) / p.h_q));
    // every row's u in this wave's channels, and reference; l of this wave's rows and tokens
    v4f u[NT][kC];
    float m[NT], l[kN];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < kC; ++c) u[n][c] = v4f{0.f, 0.f, 0.f, 0.f};
      m[n] = kLatentLow;
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) l[n] = 0.f;
    // the n-th of this wave's row tiles, of what is kept for all
    auto of_wave = [&](const float (&v)[NT], int n) { return RW == 1 || rw == 0 ? v[n] : v[(kN + n) % NT]; };

    const int last = min(t1, (any_hi + kLatentStep - 1) / kLatentStep);
    if (t0 < last) {
      int found;
      auto look = [&](int step) {
        found = p.c.table[(size_t)seq * p.c.max_blocks + min((step * kLatentStep + wave * 16) >> p.c.block_log2, p.c.max_blocks - 1) + zero];
      };
      auto page_of = [&](int step) {
        const int f = __builtin_amdgcn_readfirstlane(found);
        const int j = (step * kLatentStep + wave * 16) >> p.c.block_log2;
        return (j < p.c.max_blocks) & ((unsigned)f < (unsigned)p.c.num_blocks) ? f : -1;
      };
      // This wave's 16 tokens of a step, as they lie in memory, in kDmas
      // pieces; tokens past the sequence's end, or of a block that the table
      // does not have, become zeros.  Where a lane's bytes lie is linear in the
      // bits of the piece's number and the lane, so that one exclusive or tells.
      constexpr int kPieces = Lds::kRow / 16, kPerDma = 64 / kPieces;  // tokens of one DMA
      constexpr int kLatentDmas = 16 / kPerDma, kDmas = kLatentDmas + P / 32 + F8;
      const int lane_l = lane / kPieces * Lds::kRow + ((lane % kPieces ^ (F8 ? lane / kPieces : latent_turn(lane / kPieces))) << 4);
      const int lane_r = P == 64 ? lane / 8 * 128 + ((lane % 8 ^ lane / 16) << 4) : lane / 4 * 64 + ((lane % 4 ^ (lane / 16 & 3)) << 4);
      v4i_rsrc rl, rr, rs;
      uint8_t* to;
      auto stage_at = [&](int step, int page, int buf) {
        const int token = step * kLatentStep + wave * 16;
        const int valid = page < 0 ? 0 : min(max(sq.kv - token, 0), 16);
        const size_t row = ((size_t)max(page, 0) << p.c.block_log2) + (token & (p.c.block - 1));
        to = lds + buf * Lds::kBuffer;
        rl = make_rsrc(p.c.latent + row * Lds::kRow, valid * Lds::kRow);
        rr = make_rsrc(p.c.rope + row * P, valid * P * 2);
        if constexpr (F8) rs = make_rsrc(p.c.scales + row * (L / 128), valid * (L / 128) * 4);
        if (lane == 0) s_there[buf * 4 + wave] = page >= 0;
      };
      auto stage = [&](int i) {
        if (i < kLatentDmas) {
          const int t = i * kPerDma;
          lds_dma16(rl, lane_l ^ (i * 1024 | (F8 ? t : latent_turn(t)) << 4), 0, to + wave * 16 * Lds::kRow + i * 1024);
        } else if (i < kLatentDmas + P / 32) {
          const int r = i - kLatentDmas;
          lds_dma16(rr, lane_r ^ (r * 1024 | (P == 64 ? r * 4 : 0) << 4), 0, to + Lds::kLatent + wave * 16 * P * 2 + r * 1024);
        } else {
          lds_dma4(rs, lane * 4, 0, to + Lds::kLatent + Lds::kRope + wave * 256);
        }
        if (i == kDmas - 1) lds_dma_end(rr, lane);
      };
      // Where a lane's pieces of a step lie: of keys (piece 2 g of a bf16 row, g of
      // a row of codes) and rope parts, of p as it writes and reads it, and of four
      // tokens' channels; other pieces come in by an exclusive or or an offset.
      int group[RW];  // this wave's groups of 16 tokens; where two waves widen a group, it is the first of one of them
#pragma unroll
      for (int r = 0; r < RW; ++r) group[r] = RW == 1 ? wave : tw * 2 + (r ^ rw);
      const uint32_t lane_k = a * Lds::kRow + (F8 ? (g ^ a) << 4 : (2 * g ^ latent_turn(a)) << 4);
      const uint32_t lane_kr = Lds::kLatent + a * P * 2 + ((P == 64 ? 2 * g ^ (a >> 1 & 7) : g ^ (a >> 2 & 3)) << 4);
      const uint32_t lane_p = lds_addr(lds + Lds::kP) + a * 128 + ((g ^ (a >> 1 & 7)) << 4);
      const uint32_t lane_pw = lds_addr(lds + Lds::kP) + (rw * kN * 16 + a) * 128 + (((2 * group[0] + (g >> 1)) ^ (a >> 1 & 7)) << 4) + (g & 1) * 8;
      uint32_t lane_v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tk = 8 * g + 4 * h + (a >> 2);  // of 32; + 32 for the second half of the step
        // piece 2 c + (a % 4) / 2 of the row, c = wave kC + i: i comes in by an exclusive or
        lane_v[h] = tk * (2 * L) + (((2 * wave * kC + (a >> 1 & 1)) ^ latent_turn(tk & 15)) << 4) + (a & 1) * 8;
      }
      __syncthreads();  // the tile before is done with LDS
      if (tid < 2) s_flag[tid] = s_inf[tid] = 0;
      look(t0);
      stage_at(t0, page_of(t0), 0);
      look(t0 + 1);
#pragma unroll
      for (int i = 0; i < kDmas; ++i) stage(i);
      const int page1 = page_of(t0 + 1);
      look(t0 + 2);
      wait_vmem_all();
      int page2 = page_of(t0 + 2);
      look(t0 + 3);
      stage_at(t0 + 1, t0 + 1 < last ? page1 : -1, 1);
      __syncthreads();

      int s = t0;
      auto steps = [&](int until, auto form) {
        constexpr bool MASKED = decltype(form)::value;
#pragma unroll 1
        for (; s < until; ++s) {
          const int buf = latent_uniform(s - t0) & 1;
          uint8_t* const now = lds + buf * Lds::kBuffer;
          uint8_t* const wide = F8 ? lds + Lds::kWide : now;
          // the rest of a lane's addresses is worked out in every step: kept over
          // the loop they would take the registers that q and u need
          int here = lane;
          asm volatile("" : "+v"(here));
          const int a = here & 15, g = here >> 4;
          // Scores: tokens 16 group[r] + a of the step with rows 16 (rw kN + n)
          // + a, 64 channels at a time.  The next step's tokens set out
          // meanwhile, piece by piece between the products, which leave room.
          v4f x[RW][kN];
#pragma unroll
          for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int n = 0; n < kN; ++n) x[r][n] = v4f{0.f, 0.f, 0.f, 0.f};
          // two pieces every 128 channels and then one, the rest beside the second product
          constexpr int kEarly = kJ + kJ / 2 < kDmas ? kJ + kJ / 2 : kDmas;
          auto stage_of = [&](int j, int i) {
            const int piece = j + j / 2 + i;
            if (i < 1 + j % 2 && piece < kEarly) stage(piece);
          };
          bool there[RW];
          uint32_t at_k[RW];
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            there[r] = s_there[buf * 4 + group[r]] != 0;
            at_k[r] = lds_addr(now) + group[r] * (16 * Lds::kRow) + lane_k;
          }
          auto key_at = [&](int j, int h, int r) {
            const uint32_t bits = F8 ? (j & 3) * 64 : (j & 1) * 128 + h * 16;
            return *(const lds_v4u*)(uintptr_t)((at_k[r] ^ bits) + (F8 ? j / 4 : j / 2) * 256);
          };
          v4u k[3][F8 ? 1 : 2][RW];
          auto fetch_k = [&](int j) {
#pragma unroll
            for (int r = 0; r < RW; ++r)
#pragma unroll
              for (int h = 0; h < (F8 ? 1 : 2); ++h) k[j % 3][h][r] = key_at(j, h, r);
          };
          fetch_k(0);
          fetch_k(1);
          float scale[RW][F8 ? L / 128 : 1];
          if constexpr (F8)
#pragma unroll
            for (int r = 0; r < RW; ++r) {
              const float* const sc = (const float*)(now + Lds::kLatent + Lds::kRope + group[r] * 256) + a * (L / 128);
#pragma unroll
              for (int b = 0; b < L / 128; ++b) scale[r][b] = sc[b];
            }
          const uint32_t at_w = lds_addr(wide) + (16 * group[0] + a) * (2 * L) + ((2 * g ^ latent_turn(a)) << 4);  // e4m3
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            if (j + 2 < kJ) fetch_k(j + 2);
            __builtin_amdgcn_sched_barrier(0);
            v4u kk[2][RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) {
              if constexpr (F8) {
                const v4u c = k[j % 3][0][r];
                kk[0][r] = latent_widen(c[0], c[1], scale[r][j / 2]);
                kk[1][r] = latent_widen(c[2], c[3], scale[r][j / 2]);
                if (r == 0)  // kept for the second product
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    *(lds_v4u*)(uintptr_t)((at_w ^ ((j & 1) * 128 + h * 16)) + j / 2 * 256) = kk[h][r];
              } else {
                kk[0][r] = k[j % 3][0][r];
                kk[1][r] = k[j % 3][1][r];
              }
            }
            int i = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int r = 0; r < RW; ++r) {
#pragma unroll
                for (int n = 0; n < kN; ++n)
                  x[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, kk[h][r]), qf[n][2 * j + h], x[r][n], 0, 0, 0);
                stage_of(j, i++);
                if constexpr (!F8) __builtin_amdgcn_sched_barrier(0);
              }
            if constexpr (RW == 1) stage_of(j, i);
          }
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const uint32_t from = lds_addr(now) + group[r] * (16 * P * 2) + lane_kr;
#pragma unroll
            for (int j = 0; j < kRopeFrags; ++j) {
              const v8bf kr = __builtin_bit_cast(v8bf, *(const lds_v4u*)(uintptr_t)(from ^ (j * 16)));
#pragma unroll
              for (int n = 0; n < kN; ++n) x[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kr, qrf[n][j], x[r][n], 0, 0, 0);
            }
          }
          mfma_settle(x);  // for the branch below
          // lane: row 16 (rw kN + n) + a, tokens 4 g + e of a group of 16
          bool inf = false;
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const int token = s * kLatentStep + 16 * group[r] + 4 * g;
            const bool is = __builtin_amdgcn_readfirstlane(there[r]);
            if (MASKED || !is) {
              asm volatile("");  // a branch: most steps leave it out
#pragma unroll
              for (int n = 0; n < kN; ++n) {
                const int seen = is ? hi[n] - token : 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if constexpr (MASKED) inf |= e < seen && x[r][n][e] == -__builtin_huge_valf();
                  x[r][n][e] = e < seen ? x[r][n][e] : -__builtin_huge_valf();
                }
              }
            }
          }
          uint8_t* const s_rest = Lds::kRestOverRope ? now + Lds::kLatent : lds + Lds::kRest;
          constexpr int kRestGroup = Lds::kRestOverRope ? 16 * P * 2 : kRows * 32;
          if constexpr (MASKED && Lds::kRestOverRope) lds_barrier();
          float sum[kN], most = -__builtin_huge_valf();
          auto weigh = [&]() {
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              const int row = 16 * (rw * kN + n) + a;
              const float ref = of_wave(m, n);
              sum[n] = 0.f;
#pragma unroll
              for (int r = 0; r < RW; ++r) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = __builtin_fmaf(x[r][n][e], p.scale_log2, -ref);  // what is masked is -inf: the scale is not 0
                most = fmaxf(most, fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])));
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = __builtin_amdgcn_exp2f(w[e]);
                sum[n] += (w[0] + w[1]) + (w[2] + w[3]);
                const v2u packed = {pack2_bf16(w[0], w[1]), pack2_bf16(w[2], w[3])};
                *(lds_v2u*)(uintptr_t)((lane_pw ^ (r * 32)) + n * 2048) = packed;
                if constexpr (MASKED) {
                  const v2u rest = {pack2_bf16(w[0] - __uint_as_float(packed[0] << 16), w[1] - __uint_as_float(packed[0] & 0xFFFF0000u)),
                                    pack2_bf16(w[2] - __uint_as_float(packed[1] << 16), w[3] - __uint_as_float(packed[1] & 0xFFFF0000u))};
                  *(v2u*)(s_rest + group[r] * kRestGroup + row * 32 + g * 8) = rest;
                }
              }
            }
          };
          weigh();
          if (__any(most > 0.f) && here == 0) s_flag[s & 1] = 1;
          if constexpr (MASKED)
            if (__any(inf) && here == 0) s_inf[s & 1] = 1;
          lds_barrier();
          // u += c^T p^T, this wave's channels; the first operands are on their
          // way before it is known that p stays
          constexpr int kAhead = 4, kPf = MASKED ? 1 : 2;  // steps with masks have two pieces of p: half of the tokens at a time
          v8bf pf[kPf][NT], rest[NT];
          auto fetch_p = [&](int k) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int row = 16 * n + a;
              pf[k % kPf][n] = __builtin_bit_cast(v8bf, *(const volatile lds_v4u*)(uintptr_t)((lane_p ^ (k * 64)) + n * 2048));
              if constexpr (MASKED) rest[n] = *(const v8bf*)(s_rest + (2 * k + (g >> 1)) * kRestGroup + row * 32 + (g & 1) * 16);
            }
          };
          const uint32_t at_v[2] = {lds_addr(wide) + lane_v[0], lds_addr(wide) + lane_v[1]};
          v4u v[kAhead + 1];
          auto fetch_v = [&](int i) {  // column tile i % kC, tokens 32 (i / kC) ..
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const v2u w = lds_turned((at_v[h] ^ (i % kC * 32)) + i / kC * 32 * 2 * L);
              v[i % (kAhead + 1)][2 * h] = w[0];
              v[i % (kAhead + 1)][2 * h + 1] = w[1];
            }
          };
          const int moved = s_flag[s & 1];
          fetch_p(0);
#pragma unroll
          for (int i = 0; i < kAhead; ++i) fetch_v(i);
          if constexpr (!MASKED) fetch_p(1);
          if (moved) {
            // some row's score passed its reference: all waves move it alike
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              float top = -__builtin_huge_valf();
#pragma unroll
              for (int r = 0; r < RW; ++r) top = fmaxf(top, fmaxf(fmaxf(x[r][n][0], x[r][n][1]), fmaxf(x[r][n][2], x[r][n][3])));
              top = fmaxf(top, __shfl_xor(top, 16, 64));
              top = fmaxf(top, __shfl_xor(top, 32, 64)) * p.scale_log2;
              if (g == 0) s_max[tw * kRows + 16 * (rw * kN + n) + a] = top;
            }
            lds_barrier();
            float shrinks[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float top = s_max[16 * n + a];
#pragma unroll
              for (int w = 1; w < 4 / RW; ++w) top = fmaxf(top, s_max[w * kRows + 16 * n + a]);
              const float ref = top > m[n] ? top + kLatentLead : m[n];
              shrinks[n] = top > m[n] ? __builtin_amdgcn_exp2f(m[n] - ref) : 1.f;
              m[n] = ref;
#pragma unroll
              for (int c = 0; c < kC; ++c) u[n][c] *= shrinks[n];
            }
#pragma unroll
            for (int n = 0; n < kN; ++n) l[n] *= of_wave(shrinks, n);
            weigh();
            lds_barrier();
            fetch_p(0);
            if constexpr (!MASKED) fetch_p(1);
          }
          const bool odd = MASKED && s_inf[s & 1] != 0;
          if (tid == 0) s_flag[(s & 1) ^ 1] = 0;
          if (MASKED && tid == 0) s_inf[(s & 1) ^ 1] = 0;
#pragma unroll
          for (int n = 0; n < kN; ++n) l[n] += sum[n];
#pragma unroll
          for (int i = 0; i < 2 * kC; ++i) {
            const int c = i % kC, k = i / kC;
            if (MASKED && i == kC) fetch_p(1);
            if (i + kAhead < 2 * kC) fetch_v(i + kAhead);
            __builtin_amdgcn_sched_barrier(0);
            v4u w = v[i % (kAhead + 1)];
            if constexpr (MASKED) {
              // a token that some rows see and others do not must reach the
              // former only: what is not finite has made their sums NaN already,
              // or is dealt with below
#pragma unroll
              for (int e = 0; e < 4; ++e) w[e] = bf16_finite(w[e]);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                u[n][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), rest[n], u[n][c], 0, 0, 0);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
              u[n][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), pf[k % kPf][n], u[n][c], 0, 0, 0);
            if (kEarly + i < kDmas) stage(kEarly + i);
            if (i == (kDmas - kEarly < kC ? kC : 2 * kC - 1)) stage_at(s + 2, s + 2 < last ? page2 : -1, buf);  // for the next step to send for
          }
          if (odd) {
            // A row sees a token with a score of -inf and a weight of 0: 0 times
            // infinity makes each channel NaN that is infinite there.  A product
            // of what is not finite with what a row sees finds these.
#pragma unroll
            for (int i = 0; i < 2 * kC; ++i) {
              const int c = i % kC, k = i / kC;
              v4u w;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const v2u x = lds_turned((at_v[h] ^ (c * 32)) + k * 32 * 2 * L);
                w[2 * h] = bf16_not_finite(x[0]);
                w[2 * h + 1] = bf16_not_finite(x[1]);
              }
              if (!__any((w[0] | w[1] | w[2] | w[3]) != 0)) continue;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const int row = min(row0 + 16 * n + a, rows - 1);
                const int seen = latent_sees(p, sq, row / p.h_q) - (s * kLatentStep + 32 * k + 8 * g);
                v4u sees;
#pragma unroll
                for (int e = 0; e < 4; ++e) sees[e] = (2 * e < seen ? 0x3F80u : 0u) | (2 * e + 1 < seen ? 0x3F800000u : 0u);
                const v4f count = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, sees),
                                                                         v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) u[n][c][e] = count[e] > 0.f ? __builtin_nanf("") : u[n][c][e];
              }
            }
          }
          static_assert(kDmas - kEarly < 2 * kC, "all pieces have set out before the next ones' places are worked out");
          // the next step has landed, and everybody is done with this one
          wait_vmem_all();
          page2 = page_of(s + 3);
          __syncthreads();
          look(s + 4);
        }
      };
      const int whole = max(min(all_hi / kLatentStep, last), t0);
      steps(whole, std::false_type{});
      steps(last, std::true_type{});
    }
    // l of the lane groups and of the waves that share the tokens
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      l[n] += __shfl_xor(l[n], 16, 64);
      l[n] += __shfl_xor(l[n], 32, 64);
      if (g == 0) s_max[tw * kRows + 16 * (rw * kN + n) + a] = l[n];
    }
    __syncthreads();
    const bool whole_tile = t0 == 0 && t1 == sq.steps;
    // a part that does not start its tile is its workgroup's first; one that does may have another tile before it
    const int slot = worker * 2 + (at == begin ? 0 : 1);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float sum = s_max[16 * n + a];
#pragma unroll
      for (int w = 1; w < 4 / RW; ++w) sum += s_max[w * kRows + 16 * n + a];
      if (whole_tile) {
        const int row = row0 + 16 * n + a;
        if (row >= rows) continue;
        latent_write<L, kC>(p, sq, row, wave * (L / 4) + g * 4, u[n], m[n], sum, wave == 0 && g == 0);
      } else {
        // as the lanes hold it: whole kilobytes
        v4f* const to = (v4f*)(p.part_u + (size_t)slot * (kRows * L)) + lane;
#pragma unroll
        for (int c = 0; c < kC; ++c) to[((wave * kC + c) * NT + n) * 64] = u[n][c];
        if (wave == 0 && g == 0) *(v2f*)(p.part_ml + (size_t)(slot * kRows + 16 * n + a) * 2) = v2f{m[n], sum};
      }
    }
    if (!whole_tile && t0 == 0 && tid == 0) {
      const int g1 = (int)kv8_div(seq0 + (long long)past * sq.steps + sq.steps - 1, share);
      p.cut[worker] = LatentCut{seq, tile, g1 - group + 1, slot};
    }
    at += t1 - t0;
  }
}

// Adds up the parts of the tiles that shares cut, in an order that does not
// change from call to call.  The workgroups share out all pieces of such tiles:
// kPer times 16 rows by 16 channels, of which each wave takes every fourth part.
// (4 x 65536 with 128 heads took 141 us with sixteen workgroups a tile, 123 like
// this.)  Bound by the launch and two chained loads: 4 us where there is one tile,
// 5.8 us behind 64 x 8192, 10.3 to 11.2 us behind 4 x 65536 and 32 x 4096 with 128 heads,
// up to 67 MB of parts that the L2s and the Infinity Cache hold.
template <int L, int NT>
__global__ __launch_bounds__(256) void latent_join_kernel(LatentAttnParams p) {
  constexpr int kRows = 16 * NT, kPer = 4, kPieces = L / 16 * NT / kPer;
  __shared__ int s_tile[256], s_count[4];
  __shared__ float s_ml[4][2][kRows];
  __shared__ v4f s_u[4][kPer][64];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, a = lane & 15, g = lane >> 4;
  int item = blockIdx.x;  // among all pieces, less those of the 256 workgroups before `base`
  for (int base = 0; base < p.workers; base += 256) {
    // the workgroups that began a tile and did not finish it
    const bool cuts = base + tid < p.workers && p.cut[min(base + tid, p.workers - 1)].parts > 0;
    const uint64_t all = __ballot(cuts);
    __syncthreads();
    if (lane == 0) s_count[wave] = __popcll(all);
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wave; ++w) before += s_count[w];
    if (cuts) s_tile[before + __popcll(all & ((1ull << lane) - 1))] = base + tid;
    const int tiles = s_count[0] + s_count[1] + s_count[2] + s_count[3];
    __syncthreads();
    for (; item < tiles * kPieces; item += gridDim.x) {
      const int worker = s_tile[item / kPieces], b0 = item % kPieces * kPer;
      const LatentCut cut = p.cut[worker];
      const LatentSeq sq = latent_seq_uniform<kRows>(p, cut.seq);
      // the parts after the first are their workgroups' first
      auto slot_of = [&](int i) { return (size_t)(i == 0 ? cut.slot : (worker + i * p.together) * 2); };
      float m[NT], l[NT];
      v4f u[kPer];
#pragma unroll
      for (int n = 0; n < NT; ++n) m[n] = kLatentLow, l[n] = 0.f;
#pragma unroll
      for (int b = 0; b < kPer; ++b) u[b] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int i = wave; i < cut.parts; i += 4) {
        const size_t slot = slot_of(i);
        const v4f* const from = (const v4f*)(p.part_u + slot * (kRows * L)) + b0 * 64 + lane;
        v4f x[kPer];
        v2f ml[NT];
#pragma unroll
        for (int b = 0; b < kPer; ++b) x[b] = from[b * 64];
#pragma unroll
        for (int n = 0; n < NT; ++n) ml[n] = *(const v2f*)(p.part_ml + (slot * kRows + 16 * n + a) * 2);
        float was[NT], is[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float top = fmaxf(m[n], ml[n][0]);
          was[n] = __builtin_amdgcn_exp2f(m[n] - top);
          is[n] = __builtin_amdgcn_exp2f(ml[n][0] - top);
          l[n] = l[n] * was[n] + ml[n][1] * is[n];
          m[n] = top;
        }
#pragma unroll
        for (int b = 0; b < kPer; ++b) u[b] = u[b] * was[b % NT] + x[b] * is[b % NT];
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (g == 0) {
          s_ml[wave][0][16 * n + a] = m[n];
          s_ml[wave][1][16 * n + a] = l[n];
        }
#pragma unroll
      for (int b = 0; b < kPer; ++b) s_u[wave][b][lane] = u[b];
      __syncthreads();
      {
        const int block = b0 + wave, n = block % NT, c = block / NT, r = 16 * n + a, row = cut.tile * kRows + r;
        const float top = fmaxf(fmaxf(s_ml[0][0][r], s_ml[1][0][r]), fmaxf(s_ml[2][0][r], s_ml[3][0][r]));
        float sum = 0.f;
        v4f out[1] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = __builtin_amdgcn_exp2f(s_ml[w][0][r] - top);
          sum += s_ml[w][1][r] * f;
          out[0] += s_u[w][wave][lane] * f;
        }
        if (row < sq.count * p.h_q) latent_write<L, 1>(p, sq, row, c * 16 + g * 4, out, top, sum, c == 0 && g == 0);
      }
      __syncthreads();
    }
    item -= tiles * kPieces;
  }
}

// ---- attention, expanded
//
//   x[j] = scale * (qn . kn[j] + qr . r[j]),  o = sum_j e^(x[j] - lse) v[j]
//
// kn, v [D] are a head's own, r [D / 2] is shared by all heads.

struct LatentExpandedParams {
  const uint16_t* q;   // bf16 [total][h][3 D / 2]: key part, rope part
  const uint16_t* kv;  // bf16 [total_kv][h][2 D]: key part, value
  const uint16_t* kr;  // bf16 [total_kv][D / 2]
  long long q_stride, kv_stride, kr_stride;
  const int32_t* cu;
  const int32_t* cu_kv;
  uint16_t* out;  // bf16 [total][h][D]
  float* lse;     // [total][h] or null
  float scale_log2;
  int causal, batch, total, total_kv, most, h;
};

// How the LDS rows are turned here.  The 8 tokens of half a transposing read are
// 0 .. 7 or 8 .. 15 of 16: their pairs of pieces are told apart by t % 8.  A
// row fragment's read passes 16 lanes at a time, lanes 0-3, 12-15 and 20-27 of 32
// and the others: tokens 8 .. 11 take the odd pieces beside those of 4 .. 7, so
// that lanes of two groups, whose pieces differ by one, do not meet either (with 8
// .. 15 in the order of 0 .. 7 a quarter of the LDS cycles were conflicts).
__device__ __forceinline__ int latent_turn8(int t) { return ((t ^ (t >> 1 & 4)) & 7) << 1 | (t >> 3 & 1); }

// Tokens of a step.
constexpr int latent_expanded_step(bool split) { return split ? 128 : 64; }

// A workgroup of four waves takes 64 MT queries of one head, 16 MT of them a
// wave, and walks all tokens that they see.  Keys and values come to LDS as
// they lie in memory, two steps at a time in flight.  The scores' tiles are
// dealt so that a lane ends up with p of tokens 32 k + 4 g .. and 32 k + 16 + 4
// g .., which is what it wants as B operand if the values' transposing reads
// take the tokens in that order: p stays in registers.  p is rounded to bf16, in
// two pieces where a step has masks, as in the absorbed form.
//
// SPLIT: few queries.  A workgroup takes 16 MT of them, all in every wave, and the
// waves share out the tokens: of a step of 128 each brings 32, works on them
// without a barrier, and the four parts meet in LDS at the end.  Bound by the
// latency of a step's DMA, two of them in flight: 1.2 us a step where 8 workgroups
// run (8 heads, 4 queries of 8192 tokens 77 us, 166 with 64 MT queries each), 1.6
// where every CU has one.
//
// Bound by MFMA and the softmax's VALU work taking turns on a SIMD (two waves of
// it overlap in part: 3.3 VALU instructions an MFMA, 28 % of the wave cycles
// wait): 1 x 8192, 32 heads of 128, causal 663 to 714 us, up to 1037 TFLOP/s
// of 1212 of a large library product; 4 x up to 2048 of 4096 290 to 338 us, where a
// tile has half as many steps for its prologue and its steps with masks.
template <int D, int MT, bool SPLIT = false>
__global__ __launch_bounds__(256, 2) void latent_expanded_kernel(LatentExpandedParams p) {
  constexpr int R = D / 2, kRows = SPLIT ? 16 * MT : 64 * MT, kRow = 4 * D, kPieces = kRow / 16;  // bytes and 16-byte pieces of a token's row
  constexpr int kStep = latent_expanded_step(SPLIT), kOwn = kStep / 4;  // tokens of a step, and those that a wave brings
  constexpr int kTok = SPLIT ? kOwn : kStep;                            // and those that it works on
  constexpr int kBuffer = kStep * (kRow + 2 * R), kN = D / 32, kR = R / 32;
  extern __shared__ __align__(1024) uint8_t lds[];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, a = lane & 15, g = lane >> 4;
  const int head = blockIdx.x, seq = blockIdx.y;
  int first, count, first_kv, kv;
  const int all = latent_uniform(kv8_rows(p.cu, seq, p.total, p.most, &first, &count));
  kv8_rows(p.cu_kv, seq, p.total_kv, p.total_kv, &first_kv, &kv);
  first = latent_uniform(first);
  count = latent_uniform(count);
  first_kv = latent_uniform(first_kv);
  kv = latent_uniform(kv);
  // every sequence's last tile, which sees the most tokens, starts first
  const int row0 = ((count + kRows - 1) / kRows - 1 - (int)blockIdx.z) * kRows;
  if (row0 < 0) return;
  const int pos = kv - all;
  auto sees = [&](int i) { return p.causal ? max(min(pos + i + 1, kv), 0) : kv; };
  const int wave0 = SPLIT ? row0 : row0 + wave * 16 * MT;
  const int any_hi = sees(min(row0 + kRows, count) - 1);
  const int wave_hi = wave0 < count ? sees(min(wave0 + 16 * MT, count) - 1) : 0;

  v8bf qf[MT][kN + kR];
  int hi[MT];
#pragma unroll
  for (int n = 0; n < MT; ++n) {
    const int i = min(wave0 + n * 16 + a, count - 1);
    const uint16_t* src = p.q + (long long)(first + i) * p.q_stride + (long long)head * (D + R) + g * 8;
#pragma unroll
    for (int k = 0; k < kN + kR; ++k) qf[n][k] = __builtin_bit_cast(v8bf, *(const v4u*)(src + k * 32));
    hi[n] = sees(i);
  }
  v4f u[MT][D / 16];
  float m[MT], l[MT];
#pragma unroll
  for (int n = 0; n < MT; ++n) {
#pragma unroll
    for (int c = 0; c < D / 16; ++c) u[n][c] = v4f{0.f, 0.f, 0.f, 0.f};
    m[n] = kLatentLow;
    l[n] = 0.f;
  }

  // Where a lane finds its pieces in a step's rows: of a key (token a, channels 8
  // g ..), of a rope part, and of four values (token 4 g + a / 4, channels 4 (a %
  // 4) ..); other channels come in by an exclusive or, other tokens by an offset.
  const uint32_t lane_k = a * kRow + ((g ^ latent_turn8(a)) << 4);
  const uint32_t lane_r = a * 2 * R + ((R == 64 ? g ^ (a >> 1 & 7) : g ^ (a >> 2 & 3)) << 4);
  const int tk = 4 * g + (a >> 2);
  const uint32_t lane_v = tk * kRow + (((D / 8 + (a >> 1 & 1)) ^ latent_turn8(tk)) << 4) + (a & 1) * 8;

  // This wave's tokens of a step.
  auto stage = [&](int step, int buf) {
    uint8_t* const to = lds + buf * kBuffer;
    const uint32_t pitch = (uint32_t)p.kv_stride * 2, pitch_r = (uint32_t)p.kr_stride * 2;
#pragma unroll
    for (int o = 0; o < kOwn; o += 16) {
      const int own = wave * kOwn + o, token = step * kStep + own;
      const int valid = min(max(kv - token, 0), 16);
      const int at = first_kv + min(token, kv);
      const v4i_rsrc rk = make_rsrc(p.kv + (long long)at * p.kv_stride + (long long)head * (2 * D), valid ? (valid - 1) * pitch + kRow : 0);
      constexpr int kPerDma = 64 / kPieces;
#pragma unroll
      for (int i = 0; i < 16 / kPerDma; ++i) {
        const int t = i * kPerDma + lane / kPieces, piece = (lane % kPieces) ^ latent_turn8(t);
        lds_dma16(rk, t * pitch + piece * 16, 0, to + own * kRow + i * 1024);
      }
      const v4i_rsrc rr = make_rsrc(p.kr + (long long)at * p.kr_stride, valid ? (valid - 1) * pitch_r + 2 * R : 0);
#pragma unroll
      for (int i = 0; i < R / 32; ++i) {
        const int t = R == 64 ? i * 8 + lane / 8 : lane / 4;
        const int piece = R == 64 ? lane % 8 ^ (t >> 1 & 7) : lane % 4 ^ (t >> 2 & 3);
        lds_dma16(rr, t * pitch_r + piece * 16, 0, to + kStep * kRow + own * R * 2 + i * 1024);
      }
      if (o + 16 == kOwn) lds_dma_end(rr, lane);
    }
  };
  constexpr int kEvents = kOwn / 16 * (16 / (64 / kPieces) + R / 32) * kVmPerDma + 1;  // of one step, as vmcnt sees them

  const int last = (any_hi + kStep - 1) / kStep;
  if (last > 0) {
    stage(0, 0);
    stage(1, 1);  // past the last step: zeros
    int s = 0;
    auto steps = [&](int until, auto form) {
      constexpr bool MASKED = decltype(form)::value;
#pragma unroll 1
      for (; s < until; ++s) {
        const int base = s * kStep + (SPLIT ? wave * kTok : 0), buf = s & 1;
        wait_vmem<kEvents>();  // this step has landed, the next may be under way
        if constexpr (SPLIT)
          asm volatile("" ::: "memory");
        else
          block_barrier();
        if (base < wave_hi) {
          float t[MT][kTok / 4];
          const uint32_t now = lds_addr(lds + buf * kBuffer);
          const uint32_t at = now + (SPLIT ? wave * kTok * kRow : 0);
          const uint32_t at_r = now + kStep * kRow + (SPLIT ? wave * kTok * 2 * R : 0);
#pragma unroll
          for (int j = 0; j < kTok / 16; ++j) {
            v4f x[MT];
#pragma unroll
            for (int n = 0; n < MT; ++n) x[n] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kN + kR; ++k) {
              const v4u key = k < kN ? *(const lds_v4u*)(uintptr_t)(((at + lane_k) ^ (k * 64)) + j * 16 * kRow)
                                     : *(const lds_v4u*)(uintptr_t)(((at_r + lane_r) ^ ((k - kN) * 64)) + j * 32 * R);
#pragma unroll
              for (int n = 0; n < MT; ++n)
                x[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, key), qf[n][k], x[n], 0, 0, 0);
            }
#pragma unroll
            for (int n = 0; n < MT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) t[n][4 * j + e] = x[n][e];
          }
          v4u pw[MT][kTok / 32], rest[MT][kTok / 32];
          uint32_t seen[MT];
#pragma unroll
          for (int n = 0; n < MT; ++n) {
            // element 4 j + e: token 16 j + 4 g + e
            if constexpr (MASKED) {
              seen[n] = 0;
#pragma unroll
              for (int i = 0; i < kTok / 4; ++i) {
                const bool is = base + 16 * (i / 4) + 4 * g + i % 4 < hi[n];
                t[n][i] = is ? t[n][i] : -__builtin_huge_valf();  // the scale is not 0: it stays so
                seen[n] |= is ? 1u << i : 0u;
              }
            }
            // how far the scores are from the reference; the largest is taken of
            // these, as products' results would be made canonical for it first
            float d[kTok / 4], top = -__builtin_huge_valf();
#pragma unroll
            for (int i = 0; i < kTok / 4; ++i) d[i] = __builtin_fmaf(t[n][i], p.scale_log2, -m[n]);
#pragma unroll
            for (int i = 0; i < kTok / 4; ++i) top = fmaxf(top, d[i]);
            if (__any(top > 0.f)) {
              top = -__builtin_huge_valf();
#pragma unroll
              for (int i = 0; i < kTok / 4; ++i) top = fmaxf(top, t[n][i]);
              top = fmaxf(top, __shfl_xor(top, 16, 64));
              top = fmaxf(top, __shfl_xor(top, 32, 64)) * p.scale_log2;
              const float ref = top > m[n] ? top + kLatentLead : m[n], shrink = top > m[n] ? __builtin_amdgcn_exp2f(m[n] - ref) : 1.f;
              l[n] *= shrink;
#pragma unroll
              for (int c = 0; c < D / 16; ++c) u[n][c] *= shrink;
              m[n] = ref;
#pragma unroll
              for (int i = 0; i < kTok / 4; ++i) d[i] = __builtin_fmaf(t[n][i], p.scale_log2, -ref);
            }
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kTok / 4; i += 2) {
              const float p0 = __builtin_amdgcn_exp2f(d[i]), p1 = __builtin_amdgcn_exp2f(d[i + 1]);
              sum[0] += p0;
              sum[1] += p1;
              const uint32_t both = pack2_bf16(p0, p1);
              pw[n][i / 8][i / 2 & 3] = both;
              if constexpr (MASKED)
                rest[n][i / 8][i / 2 & 3] = pack2_bf16(p0 - __uint_as_float(both << 16), p1 - __uint_as_float(both & 0xFFFF0000u));
            }
            l[n] += sum[0] + sum[1];
          }
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t at_v = (at + lane_v) ^ (c * 32);
#pragma unroll
            for (int k = 0; k < kTok / 32; ++k) {
              v4u v;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const v2u w = lds_turned(at_v + (32 * k + 16 * h) * kRow);
                v[2 * h] = w[0];
                v[2 * h + 1] = w[1];
              }
              if constexpr (MASKED) {
                // What is not finite must reach the rows that see it only: it is
                // zeroed, and a second product finds the rows that see some of it.
                v4u ind, fin;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  fin[e] = bf16_finite(v[e]);
                  ind[e] = bf16_not_finite(v[e]);
                }
                if (__any((ind[0] | ind[1] | ind[2] | ind[3]) != 0)) {
#pragma unroll
                  for (int n = 0; n < MT; ++n) {
                    v4u sw;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      sw[e] = (seen[n] >> (8 * k + 2 * e) & 1u) * 0x3F80u | (seen[n] >> (8 * k + 2 * e + 1) & 1u) * 0x3F800000u;
                    const v4f cnt = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, ind), __builtin_bit_cast(v8bf, sw),
                                                                           v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[n][c][e] = cnt[e] > 0.f ? __builtin_nanf("") : u[n][c][e];
                  }
                }
                v = fin;
#pragma unroll
                for (int n = 0; n < MT; ++n)
                  u[n][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, v), __builtin_bit_cast(v8bf, rest[n][k]), u[n][c], 0, 0, 0);
              }
#pragma unroll
              for (int n = 0; n < MT; ++n)
                u[n][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, v), __builtin_bit_cast(v8bf, pw[n][k]), u[n][c], 0, 0, 0);
            }
          }
        }
        if constexpr (SPLIT) {
          asm volatile("" ::: "memory");
          __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's reads of the buffer have returned
          asm volatile("" ::: "memory");
        } else {
          lds_barrier();  // all are done with this buffer: their reads have returned
        }
        stage(s + 2, buf);
      }
    };
    // steps that every row of the workgroup sees wholly, and those with masks
    steps(min(sees(row0) / kStep, last), std::false_type{});
    steps(last, std::true_type{});
    wait_vmem_all();  // no LDS DMA may be in flight past this point
  }
#pragma unroll
  for (int n = 0; n < MT; ++n) {
    l[n] += __shfl_xor(l[n], 16, 64);
    l[n] += __shfl_xor(l[n], 32, 64);
  }
  // channels c .. + 3 of row n 16 + a; l == 0: it sees no token
  auto write = [&](int n, int c, v4f x, float mx, float sum, bool with_lse) {
    const int i = wave0 + n * 16 + a;
    if (i >= count) return;
    const size_t row = (size_t)(first + i) * p.h + head;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *(v2u*)(p.out + row * D + c) = v2u{pack2_bf16(x[0] * inv, x[1] * inv), pack2_bf16(x[2] * inv, x[3] * inv)};
    if (p.lse && with_lse) p.lse[row] = sum == 0.f ? -__builtin_huge_valf() : (mx + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f;
  };
  if constexpr (SPLIT) {
    // the waves' parts, in their order; wave w adds up a quarter of the channels
    v4f* const s_u = (v4f*)lds;                                     // [4][MT][D / 16][64]
    float* const s_ml = (float*)(lds + 4 * MT * (D / 16) * 1024);  // [4][2][16 MT]
    __syncthreads();
#pragma unroll
    for (int n = 0; n < MT; ++n) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c) s_u[((wave * MT + n) * (D / 16) + c) * 64 + lane] = u[n][c];
      if (g == 0) {
        s_ml[(wave * 2 + 0) * 16 * MT + n * 16 + a] = m[n];
        s_ml[(wave * 2 + 1) * 16 * MT + n * 16 + a] = l[n];
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < MT; ++n) {
      float f[4], top = kLatentLow, sum = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, s_ml[w * 2 * 16 * MT + n * 16 + a]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f[w] = __builtin_amdgcn_exp2f(s_ml[w * 2 * 16 * MT + n * 16 + a] - top);
        sum += s_ml[(w * 2 + 1) * 16 * MT + n * 16 + a] * f[w];
      }
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        const int c = wave * (D / 64) + k;
        v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) x += s_u[((w * MT + n) * (D / 16) + c) * 64 + lane] * f[w];
        write(n, c * 16 + g * 4, x, top, sum, c == 0 && g == 0);
      }
    }
  } else {
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int c = 0; c < D / 16; ++c) write(n, c * 16 + g * 4, u[n][c], m[n], l[n], c == 0 && g == 0);
  }
}

}  // namespace dg
