// delta_chunk.hpp -- what the chunked kernels of the gated delta rule share:
// the chunk's mathematics, its image in the workspace, fp16 pairs and the
// layout of MFMA operands.
//
// A chunk of C = 64 tokens that starts from the state S0 (here dstate x
// headdim), with cs_t the sum of step A up to t (inclusive, chunk-local):
//   N_tj = e^{cs_t - cs_j} k_t . k_j            (j < t)
//   T    = (I + N diag(b))^-1                    (unit lower triangular)
//   X    = V - diag(e^cs) K S0,   R = T X,   U = diag(b) R
//   Y    = scale (diag(e^cs) Q S0 + P R),  P_tj = e^{cs_t - cs_j} (q_t . k_j) b_j  (j <= t)
//   S_C  = e^{cs_C} S0 + K^T diag(e^{cs_C - cs} b) R
// R is what each token adds, v_t minus what the state answers its key; b only
// meets it in P and in the last line, so a b of zero divides nothing.
// T, P and the fades depend on q, k and the gates alone, not on the state, so
// a first kernel (delta_prep_kernel) forms them for all chunks at once; the
// second (delta_walk_kernel) walks each sequence's chunks in order.  The
// columns of S0, X, R and Y (value channels) never meet, so the walk cuts a
// head into tiles of 16 channels.
//
// Operand order.  An accumulator of v_mfma_f32_16x16x32_f16 holds rows 4 lq + i
// (i < 4) of column lr in lane 16 lq + lr.  The same registers, two row tiles
// side by side, are a B (or, transposed, an A) operand whose K index runs
// 4 lq + {0..3}, 16 + 4 lq + {0..3} in a lane: a product does not care in which
// order K runs as long as both operands agree.  So the state, X and U go from
// one product into the next in registers, and the other operands (K, Q, T, P)
// are stored or read in that order ("paired order").
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "common.hpp"

namespace ssm {

constexpr int kDeltaC = 64;  // tokens per chunk

// The chunk image, one per (chunk slot, head): operand fragments in paired
// order, 64 lanes x 16 bytes each.  T and P are lower triangular, so of a
// 64 x 64 matrix only six fragments (row tile t, column pair m <= t / 2) hold
// anything: index kFragOf(t, m).
constexpr int kFrag = 1024;                  // bytes of a fragment
constexpr int kImgThi = 0;                   // T, fp16 hi
constexpr int kImgTlo = 6 * kFrag;           // T, fp16 lo
constexpr int kImgP = 12 * kFrag;            // P, fp16
constexpr int kImgGrow = 18 * kFrag;         // e^{cs_t}
constexpr int kImgLeft = kImgGrow + 256;     // e^{cs_C - cs_t} b_t (0 behind the sequence's end)
constexpr int kImgBytes = kImgGrow + 512;
// The backward's image: the same fragments of T (for its walk forward), then T's and P's transposes (for its walk back;
// P without b), each a pair, and the gates.
constexpr float kBwdPScale = 16.0f;          // P is kept 16 times as large, away from the last places of fp16
// Beside its values' scale the backward's forward walk holds the state 32 times as large: its elements are smaller than
// the values that make them, and the last place of a pair's lo part is 2^-24 (states of 128 x 128 were off by 3.5e-7
// without it, by 2.2e-7 with it).
constexpr float kBwdStateUp = 32.0f;
// T too, whose elements off the diagonal are small, and X (3 x 333 tokens: the gradient of A up to 1.6e-6 off without,
// 3.6e-7 with them).
constexpr float kBwdTUp = 64.0f;
constexpr float kBwdXUp = 16.0f;
constexpr int kBwdBack = 12 * kFrag;         // T^T hi, T^T lo, P^T hi, P^T lo: six fragments each
constexpr int kBwdGates = kBwdBack + 24 * kFrag;
// (64 floats each: e^{cs_t}, scale e^{cs_t}, e^{cs_C - cs_t}, b_t, and cs_t as a pair hi, lo)
constexpr int kBwdImgBytes = kBwdGates + 1536;
__host__ __device__ constexpr int frag_of(int t, int m) { return t < 2 ? t : 2 + 2 * (t - 2) + m; }
// The same of the transposes, upper triangular: row tile t, column pair m >= t / 2.
__host__ __device__ constexpr int back_frag(int t, int m) { return m ? t : 4 + t; }

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4_t mfma_f16(f16x8_t a, f16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Two accumulator tiles as one operand: rounded to fp16 (nearest even), and as
// a pair hi + lo (hi = fp16(v), lo = fp16(v - hi): 22 significant bits).
__device__ __forceinline__ f16x8_t pair_f16(f32x4_t a, f32x4_t b) {
  const f16x4_t x = __builtin_convertvector(a, f16x4_t), y = __builtin_convertvector(b, f16x4_t);
  return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}
// v - h exactly, h an fp16 value: one mixed-precision FMA each (the compiler turns half of them into a conversion and
// a subtraction when it may choose).
__device__ __forceinline__ f32x4_t f16_rest(f32x4_t v, f16x4_t h) {
  const u32x2_t w = __builtin_bit_cast(u32x2_t, h);
  f32x4_t r;
  asm("v_fma_mix_f32 %0, -%1, 1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r[0]) : "v"(w[0]), "v"(v[0]));
  asm("v_fma_mix_f32 %0, -%1, 1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r[1]) : "v"(w[0]), "v"(v[1]));
  asm("v_fma_mix_f32 %0, -%1, 1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r[2]) : "v"(w[1]), "v"(v[2]));
  asm("v_fma_mix_f32 %0, -%1, 1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r[3]) : "v"(w[1]), "v"(v[3]));
  return r;
}
__device__ __forceinline__ void split_f16(f32x4_t a, f32x4_t b, f16x8_t& hi, f16x8_t& lo) {
  const f16x4_t x = __builtin_convertvector(a, f16x4_t), y = __builtin_convertvector(b, f16x4_t);
  hi = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  lo = pair_f16(f16_rest(a, x), f16_rest(b, y));
}

// Eight bf16 values as fp16 (exact from 2^-17 to 65504 in magnitude).
__device__ __forceinline__ u32x4_t bf16x8_as_f16(u32x4_t v) {
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2_t h = __builtin_convertvector((f32x2_t){bf16_lo(v[i]), bf16_hi(v[i])}, f16x2_t);
    r[i] = __builtin_bit_cast(uint32_t, h);
  }
  return r;
}

// K and Q of a chunk in LDS, fp16.  For fragments of rows (16 rows x 32
// columns) each 32-element block is stored in paired order, so that a lane
// reads its two runs with one 16-byte read (two 8-byte runs in one instruction
// take twice as long), rows 4 x odd dwords apart: every bank once.  For
// fragments of columns (transposed reads, eight rows x 32 bytes at a time) K
// is kept a second time, as it is, rows 8 x odd dwords apart: every bank once.
template <int DK> constexpr int kRowLd = DK + 8;
template <int DK> constexpr int kColLd = DK + 16;
// Where run j (four elements) of a 32-element block sits in paired order.
__device__ __forceinline__ constexpr int paired_run(int j) { return j < 4 ? 2 * j : 2 * j - 7; }
// Elements cc .. cc + 7 (cc a multiple of 8) of a row in paired order.
__device__ __forceinline__ void lds_store_paired(uint16_t* row, int cc, u32x4_t v) {
  uint16_t* a = row + (cc & ~31);
  const int j = (cc >> 2) & 7;
  *reinterpret_cast<u32x2_t*>(a + 4 * paired_run(j)) = u32x2_t{v[0], v[1]};
  *reinterpret_cast<u32x2_t*>(a + 4 * paired_run(j + 1)) = u32x2_t{v[2], v[3]};
}
// Columns 32 kk .. + 31 of row r.
template <int DK> __device__ __forceinline__ f16x8_t lds_row_frag(const uint16_t* base, int r, int kk, int lq) {
  return *reinterpret_cast<const f16x8_t*>(base + r * kRowLd<DK> + 32 * kk + 8 * lq);
}
// Transposed LDS read (ds_read_b64_tr_b16): lane i of 16 receives, of the four
// rows that the 16 lanes address as 4 x 4 runs (lane i: row i / 4, run i % 4),
// column i.
__device__ __forceinline__ u32x2_t lds_tr4(const uint16_t* a) {
  typedef short v4i16 __attribute__((ext_vector_type(4)));
  const v4i16 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16*)(a));
  return __builtin_bit_cast(u32x2_t, v);
}
// A fragment whose K index is the row of such an array: rows k0 .. k0 + 31 in paired order, columns 16 d + lr.
template <int DK> __device__ __forceinline__ f16x8_t lds_col_frag(const uint16_t* base, int k0, int d, int lr, int lq) {
  const uint16_t* a = base + (k0 + 4 * lq + (lr >> 2)) * kColLd<DK> + 16 * d + 4 * (lr & 3);
  const u32x2_t x = lds_tr4(a), y = lds_tr4(a + 16 * kColLd<DK>);
  return __builtin_bit_cast(f16x8_t, u32x4_t{x[0], x[1], y[0], y[1]});
}

// A 16-byte buffer store.  The whole offset goes into the lane's: with a scalar register for a part of it the compiler
// takes such a store as done with its data at once, and let the next instruction overwrite them; on the MI355X four
// lanes of every sixteen then stored the new value of the first dword, now and then.
__device__ __forceinline__ void store_b128(u32x4_t v, rsrc_t r, int voff) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, voff, 0, 0);
}

// f(IC<0>) .. f(IC<N - 1>): a loop whose index is a constant in the body.
template <class F, int... I> __device__ __forceinline__ void static_for_each(F&& f, std::integer_sequence<int, I...>) {
  (f(IC<I>{}), ...);
}
template <int N, class F> __device__ __forceinline__ void static_for(F&& f) {
  static_for_each(f, std::make_integer_sequence<int, N>{});
}

// Sequence s of the call: its first token in the flat [batch * L] token axis,
// its length, and its first chunk slot.  Packed offsets are clamped into
// [0, L]; slot cu[s] / 64 + s leaves every sequence room for its chunks, since
// ceil(len / 64) <= floor(end / 64) - floor(start / 64) + 1.
struct DeltaSeq {
  int64_t tok, len, slot;
};
__device__ __forceinline__ DeltaSeq delta_seq(const int64_t* cu, int64_t s, int64_t L, int64_t chunks_per_row) {
  DeltaSeq d;
  if (!cu) {
    d.tok = s * L;
    d.len = L;
    d.slot = s * chunks_per_row;
    return d;
  }
  const int64_t a = cu[s], b = cu[s + 1];
  d.tok = a < 0 ? 0 : (a > L ? L : a);
  const int64_t e = b < d.tok ? d.tok : (b > L ? L : b);
  d.len = e - d.tok;
  d.slot = d.tok / kDeltaC + s;
  return d;
}

// The last sequence of n that starts at or before a chunk slot, by a whole wavefront: 64 places are tried at once.
__device__ __forceinline__ int64_t delta_slot_seq(const int64_t* cu, int64_t n, int64_t L, int64_t slot) {
  const int64_t lane = threadIdx.x & 63;
  int64_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const int64_t step = (hi - lo + 63) / 64, at = lo + (lane + 1) * step;
    const bool before = at <= hi && delta_seq(cu, at, L, 0).slot <= slot;
    const int64_t count = __popcll(__ballot(before));  // (the slots ascend)
    lo += count * step;
    hi = lo + step - 1 < hi ? lo + step - 1 : hi;
  }
  return lo;
}

// What is linear in the values (or in the gradients) may have any magnitude, but passes through fp16 pairs.  So values
// and initial states are scaled by the power of two that brings their largest magnitude to [32, 64) (the backward's to
// [2, 4)), dY and dfinal to [16, 32), and results scaled back, all exactly.  (Above, states and sums have room up to the
// largest fp16, 65504; the lo part of a pair, whose last place is 2^-24, keeps its bits down to 2^-3.)  The scale is 1
// where nothing, or something not finite, is the largest; it stays between 2^-60 and 2^60, so that products of two stay
// in fp32.
__device__ __forceinline__ float unit_scale(unsigned amax_bits, int target) {
  const int e = static_cast<int>(amax_bits >> 23) - 127;
  if (amax_bits == 0u || e > 127) return 1.0f;
  const int s = target - e < -60 ? -60 : (target - e > 60 ? 60 : target - e);
  return __uint_as_float(static_cast<unsigned>(s + 127) << 23);
}
__device__ __forceinline__ float grad_scale(unsigned amax_bits) { return unit_scale(amax_bits, 4); }
// (lower for heads wider than 256: the gradients take dy . u over all channels as an fp16)
__device__ __forceinline__ float value_scale(unsigned amax_bits, int64_t P) {
  const int wide = 56 - __builtin_clzll(static_cast<unsigned long long>(P - 1));  // log2(P / 256), rounded up
  return unit_scale(amax_bits, 1 - (wide > 0 ? wide : 0));
}

// A channel tile that the head does not have is addressed here: behind every
// resource (they are cut to this length, and a chunk's offsets, 64 rows of at
// most 2^23 bytes, stay below half of it), so loads return zero and stores are
// dropped.
constexpr int kPastEnd = 0x40000000;

// Workgroups are dealt round-robin to the eight XCDs; giving each XCD a run of
// consecutive units lets neighbours that read the same rows share its L2.
__device__ __forceinline__ unsigned xcd_order(unsigned i, unsigned n) {
  const unsigned q = n / 8, r = n % 8, x = i % 8;
  return x * q + (x < r ? x : r) + i / 8;
}

// The (sequence, head) unit and block of channels of a walk's workgroup.  Rows of one length go to the XCDs in runs;
// packed sequences are handed out longest first over all of them (in runs, one XCD gets all the heads of the longest
// sequence), so that the last ones are short.
struct DeltaUnit {
  int64_t seq, h, block;
};
__device__ __forceinline__ int64_t key_head(int64_t h, int64_t H, int64_t G) {
  return static_cast<unsigned>(h) / (static_cast<unsigned>(H) / static_cast<unsigned>(G));
}
// (Workgroups are counted in 32 bits, which the host sees to, and divided so: a division of 64 bits is a hundred
// instructions.)
template <class P> __device__ __forceinline__ DeltaUnit delta_unit(const P& p, int64_t blocks) {
  const unsigned nb = static_cast<unsigned>(blocks), H = static_cast<unsigned>(p.H);
  const unsigned id = p.cu ? blockIdx.x : xcd_order(blockIdx.x, static_cast<unsigned>(p.rows) * H * nb);
  const unsigned unit = id / nb, s = unit / H;
  return {p.cu ? p.order[s] : s, unit - s * H, id - unit * nb};
}

struct DeltaChunkParams {
  const void* q;       // [tokens][G][N] bf16
  const void* k;
  const void* v;       // [tokens][H][P] bf16
  const void* delta;   // [tokens][H] bf16 (raw)
  const float* A;      // [H]
  const void* beta;    // [tokens][H] bf16
  const float* bias;   // [H] (nullable)
  const float* h0;     // [rows][H][P][N] (nullable); may be hT
  float* hT;           // (nullable)
  const int64_t* cu;   // (nullable)
  int* order;          // with cu: the sequences, longest first
  void* y;
  char* img;           // [slots][H][kImgBytes]
  unsigned* words;     // workspace header
  // backward: bits of the largest |v| of a chunk (of the first one |initial state| too) [slots][H], of the largest |dy|
  // and |dfinal| of a unit [rows][H]; the scale of a unit's values
  unsigned* vmax;
  unsigned* amax;
  float* vscale;
  int64_t rows;        // sequences
  int64_t L, H, G, P;
  int64_t chunks;      // chunks per batch row (no cu)
  int64_t slots;       // chunk slots in all
  int softplus, sigmoid;
  float scale;
};

// Of the backward (delta_bwd_kernels.hpp).
struct DeltaBwdParams {
  DeltaChunkParams c;
  const void* dy;       // [tokens][H][P] bf16
  const float* dfinal;  // [rows][H][P][N] (nullable)
  void* dq;             // [tokens][G][N] bf16
  void* dk;
  void* dv;             // [tokens][H][P] bf16
  void* ddelta;         // [tokens][H] bf16
  void* dbeta;
  float* dh0;           // [rows][H][P][N] (nullable)
  // kept as operand fragments, [slots][H][tiles][...][kFrag]: S0 [2][KT] (hi, lo), dS [KT] (scaled), R and dV (scaled)
  // [2][2] (hi, lo; two halves of the tokens, channel by channel)
  char* state;
  char* adj;
  char* r;
  char* dvh;
  // parts of dla over a tile's 16 channels, [slots][H][tiles][64]: the terms of S0 and Q, of S0 and K, of dS and K
  float* oterm;
  float* gterm;
  float* lterm;
  float* edge;          // [slots][H][tiles][64]: parts of e^{cs_C} <dS, S0>
  float* part;          // [slots][H][2]: parts of dA and dbias
  int64_t tiles;        // P / 16
};

}  // namespace ssm
