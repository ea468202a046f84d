// delta_walk_kernel.hpp -- the chunked gated delta rule's walk over a
// sequence (delta_chunk.hpp has the mathematics and the operand order).
//
// A wavefront owns a tile of 16 value channels with its whole state (dstate x
// 16, fp32 accumulators) and takes a chunk from S0 to S_C without exchanging
// anything with its neighbours; the W wavefronts of a workgroup share the
// chunk's K, Q, T, P and fades in LDS, double-buffered, so a chunk costs one
// barrier.  Per chunk (dstate 128) 104 MFMAs 16x16x32: K S0 32 (S0 as fp16
// hi + lo), T X 18 (both as pairs, without lo x lo), K^T R 32, Q S0 16 and
// P R 6 (one product each: y is stored with 8 bits).
//
// The chain K S0 -> X -> T X -> R -> K^T R is serial, and only two wavefronts
// share a SIMD, so the order of the instructions matters: fragments are read
// from LDS one step ahead of the products that take them, and scheduling
// fences keep the compiler from moving the reads next to their use (where each
// one's latency would show).  What bounds it is that chain: at dstate 128 a
// chunk takes a wavefront 2.8 us with a SIMD of its own, 4.1 with two on it
// (16384 tokens of 40 heads of 128 channels in 266 us, 1.9 TB/s; the products
// alone would take 60).
//
// Precision.  K and Q convert to fp16 exactly.  Everything on the way from
// state to state is a pair of fp16 (22 bits) with fp32 accumulation.
#pragma once

#include "delta_chunk.hpp"

namespace ssm {

// A tensor's next chunk: where it starts, and the length of the resource over it.  Only the last chunk's has to end
// where the sequence does; past it there is nothing.
struct DeltaStream {
  char* base;
  int64_t step;
  int tail;
  __device__ __forceinline__ DeltaStream(const void* p, int64_t chunk, int64_t last)
      : base(static_cast<char*>(const_cast<void*>(p))), step(chunk), tail(static_cast<int>(last)) {}
  // left: chunks from this one on
  __device__ __forceinline__ rsrc_t take(int left) {
    const rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(base, 0, left > 1 ? kPastEnd : (left == 1 ? tail : 0), kBufWord3);
    base += step;
    return r;
  }
};

// The larger magnitudes of two pairs of bf16, and the largest of a wavefront's (as integers, which order as they do).
__device__ __forceinline__ unsigned max_bf16x2(unsigned a, unsigned b) {
  typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a & 0x7fff7fffu),
                                                                __builtin_bit_cast(u16x2_t, b & 0x7fff7fffu)));
}
__device__ __forceinline__ unsigned finite_bits(unsigned v) { return v < 0x7f800000u ? v : 0u; }
__device__ __forceinline__ unsigned wave_max(unsigned v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = max(v, static_cast<unsigned>(__shfl_xor(static_cast<int>(v), o, 64)));
  return static_cast<unsigned>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
}

template <int DK, bool KEEP> struct DeltaWalkLds {
  __attribute__((aligned(16))) uint16_t k[kDeltaC * kRowLd<DK>];
  __attribute__((aligned(16))) uint16_t kt[kDeltaC * kColLd<DK>];
  __attribute__((aligned(16))) uint16_t q[kDeltaC * kRowLd<DK>];
  __attribute__((aligned(16))) char img[KEEP ? 12 * kFrag + 1024 : kImgBytes];  // KEEP: T and four gates
};

// What the backward's walk takes and writes beside the forward's.
struct DeltaKeep {
  const void* dy;
  const float* dfinal;
  char* state;
  char* r;
  float* oterm;
};
__device__ __forceinline__ DeltaKeep kept(const DeltaChunkParams&) { return {}; }
__device__ __forceinline__ DeltaKeep kept(const DeltaBwdParams& b) { return {b.dy, b.dfinal, b.state, b.r, b.oterm}; }

template <bool KEEP> struct DeltaWalkArgs {
  typedef DeltaChunkParams type;
};
template <> struct DeltaWalkArgs<true> {
  typedef DeltaBwdParams type;
};
__device__ __forceinline__ const DeltaChunkParams& chunk_params(const DeltaChunkParams& p) { return p; }
__device__ __forceinline__ const DeltaChunkParams& chunk_params(const DeltaBwdParams& p) { return p.c; }

// KEEP: the backward's walk over the same chunks.  It stores no y but what the gradients take of each chunk: S0 and R as
// operand fragments, (S0 q) . dy of each token over this tile's channels, and the largest |dy| of the unit.
template <int DK, int W, bool KEEP>
__global__ void __launch_bounds__(64 * W) delta_walk_kernel(typename DeltaWalkArgs<KEEP>::type wp) {
  const DeltaChunkParams& p = chunk_params(wp);
  const DeltaKeep keep = kept(wp);
  constexpr int KT = DK / 32, DT = DK / 16, NTH = 64 * W;
  using Lds = DeltaWalkLds<DK, KEEP>;
  constexpr int GATES = KEEP ? 12 * kFrag : kImgGrow, IMG = KEEP ? kBwdImgBytes : kImgBytes;
  __shared__ Lds lds[2];
  // each wavefront's own values, [token][channel], as they are in memory (bf16): written with the next chunk's
  // operands, read transposed at its start
  __shared__ __attribute__((aligned(16))) uint16_t lds_v[W][kDeltaC * 16];
  __shared__ int lds_first[W][16];  // of each channel, where a chunk's values stop being finite
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t blocks = (p.P + 16 * W - 1) / (16 * W);  // workgroups per unit
  const DeltaUnit un = delta_unit(p, blocks);
  const int64_t seq = un.seq, h = un.h, unit = seq * p.H + h, g = key_head(h, p.H, p.G);
  const int col = static_cast<int>(un.block * W + w) * 16;  // first channel of this wavefront
  const DeltaSeq sq = delta_seq(p.cu, seq, p.L, p.chunks);
  const int nchunks = static_cast<int>((sq.len + kDeltaC - 1) / kDeltaC);
  const int64_t rowe = p.H * p.P, krow = p.G * DK;
  const int rowe32 = static_cast<int>(rowe), krow32 = static_cast<int>(krow);  // the host keeps them below 2^22
  const int yrow = (lr * rowe32 + 4 * lq) * 2;

  // ---- the scale of the values and the state.  KEEP: one of the whole unit, from the largest value of each chunk.  The
  // forward: this tile's own, from the first chunk and the initial state; a chunk whose values leave [0, 1024) in that
  // scale (`limit`) gets a new one, to which the state goes over.  (Looking for the largest value before the walk, as the
  // backward does, would read all of v once more: 15 us of 380 at 16384 tokens of 40 heads.)
  float sc = 1.0f, inv = 1.0f, yscale = p.scale;
  unsigned limit = 0u;  // what |v| may be (fp32 bits)
  bool over = false;    // the next chunk has larger ones
  auto set_scale = [&](float to) {
    sc = to;
    inv = 1.0f / sc;
    yscale = p.scale * inv;
    limit = __float_as_uint(1024.0f * inv);
  };
  if constexpr (KEEP) {
    unsigned top = 0u;
    for (int c = lane; c < nchunks; c += 64) top = max(top, p.vmax[(sq.slot + c) * p.H + h]);
    set_scale(value_scale(wave_max(top), p.P));
    if (tid == 0 && un.block == 0) p.vscale[unit] = sc;
  }

  // ---- the state: channel col + lr, states 16 d + 4 lq .. + 3
  f32x4_t S[DT];
  const int64_t sbase = (unit * p.P + col + lr) * DK + 4 * lq;
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    S[d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (p.h0 && col < p.P)
      S[d] = *reinterpret_cast<const f32x4_t*>(p.h0 + sbase + 16 * d) * (KEEP ? sc * kBwdStateUp : sc);
  }

  // ---- chunk loads, one chunk ahead in registers
  constexpr int PIECES = kDeltaC * DK / 8, PER = (PIECES + NTH - 1) / NTH;
  constexpr int IPIECES = sizeof(Lds::img) / 16, IPER = (IPIECES + NTH - 1) / NTH;
  // byte offset of the channel tile: past every resource when the head has no such tile, where loads return zero and
  // stores are dropped (a branch around each load would make the compiler wait for it)
  const int64_t tiles = p.P / 16;
  const int ctile = col < p.P ? col * 2 : kPastEnd;
  u32x4_t gk[PER], gq[PER], gi[IPER];
  u32x2_t gv[4];
  // Each tensor's chunks in order, as a base that moves on (computing a chunk's address anew took a hundred scalar
  // instructions a chunk).  Past the last chunk the resources are empty, so the loop loads without a branch: a
  // conditional load's registers would be copied, and waited for, where the paths meet.
  const int64_t kb = sq.tok * krow + g * DK, vb = sq.tok * rowe + h * p.P;
  const int64_t last = sq.len - static_cast<int64_t>(nchunks - 1) * kDeltaC;  // tokens of the last chunk
  const int64_t ktail = ((last - 1) * krow + DK) * 2, vtail = ((last - 1) * rowe + p.P) * 2;
  DeltaStream ks(static_cast<const uint16_t*>(p.k) + kb, krow * kDeltaC * 2, ktail);
  DeltaStream qs(static_cast<const uint16_t*>(p.q) + kb, krow * kDeltaC * 2, ktail);
  DeltaStream vs(static_cast<const uint16_t*>(p.v) + vb, rowe * kDeltaC * 2, vtail);
  // y of the forward; KEEP: dY
  DeltaStream ys(static_cast<const uint16_t*>(KEEP ? keep.dy : p.y) + vb, rowe * kDeltaC * 2, vtail);
  DeltaStream is(p.img + (sq.slot * p.H + h) * IMG, p.H * IMG, IMG);
  // what KEEP writes of a chunk (these resources cover one tile; a lane of no tile lies behind them)
  const int64_t cell0 = (sq.slot * p.H + h) * tiles + col / 16, cells = p.H * tiles;
  DeltaStream ss(keep.state + cell0 * (2 * KT * kFrag), cells * (2 * KT * kFrag), 2 * KT * kFrag);
  DeltaStream rs(keep.r + cell0 * (4 * kFrag), cells * (4 * kFrag), 4 * kFrag);
  DeltaStream os(keep.oterm + cell0 * kDeltaC, cells * kDeltaC * 4, kDeltaC * 4);
  const int mine = lane * 16 + (col < p.P ? 0 : kPastEnd);
  float amax = 0.0f;
  // y of a chunk, four consecutive channels of token 16 t + lr in a lane; stored during the chunk after it.  KEEP: dY of
  // the chunk, in the same places.
  u32x2_t yo[4];
  // What passes between memory, registers and LDS for a chunk, as ITEMS: the row pieces of K and Q, the image's
  // pieces, the values and y, two token tiles each.  A step of the loop below takes its share of them: piece by piece
  // into LDS what was loaded a chunk ago, and the same piece of the chunk after out of memory.  (All at once they
  // kept the wavefronts waiting for the CU's one memory path: 64 bytes a clock for 83 KB a chunk.)
  constexpr int LOADS = PER + IPER + 2, ITEMS = LOADS + (KEEP ? 0 : 2);
  rsrc_t rk, rq, ri, rv, ry, rkeep;
  auto load_dy = [&] {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      yo[t] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(ry, yrow + ctile, 32 * t * rowe32, 0));
  };
  auto next_rsrc = [&](int left) { rk = ks.take(left), rq = qs.take(left), ri = is.take(left), rv = vs.take(left); };
  auto load_item = [&](auto item) {
    constexpr int i = decltype(item)::value;
    if constexpr (i < PER) {
      const int e = tid + NTH * i;
      // (a piece behind the 64 rows has no place: it is not read either, the tensor may end before it)
      const int off = PIECES % NTH == 0 || e < PIECES ? (e / (DK / 8)) * krow32 * 2 + (e % (DK / 8)) * 16 : kPastEnd;
      gk[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, 0));
      gq[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rq, off, 0, 0));
    } else if constexpr (i < PER + IPER) {
      constexpr int e = i - PER;
      // KEEP takes T and the gates, not P between them
      const int at = (tid + NTH * e) * 16 + (KEEP && tid + NTH * e >= GATES / 16 ? kBwdGates - GATES : 0);
      gi[e] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ri, at, 0, 0));
    } else if constexpr (i < PER + IPER + 2) {
      constexpr int t = 2 * ((i - PER - IPER) % 2);
      const int at = yrow + ctile;
      gv[t] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(rv, at, 32 * t * rowe32, 0));
      gv[t + 1] =
          __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(rv, at, 32 * (t + 1) * rowe32, 0));
    }
  };
  auto stage_item = [&](Lds& b, auto item) {
    constexpr int i = decltype(item)::value;
    if constexpr (i < PER) {
      const int e = tid + NTH * i, row = e / (DK / 8), cc = (e % (DK / 8)) * 8;
      if (PIECES % NTH == 0 || e < PIECES) {
        const u32x4_t k8 = bf16x8_as_f16(gk[i]), q8 = bf16x8_as_f16(gq[i]);
        lds_store_paired(&b.k[row * kRowLd<DK>], cc, k8);
        *reinterpret_cast<u32x4_t*>(&b.kt[row * kColLd<DK> + cc]) = k8;
        lds_store_paired(&b.q[row * kRowLd<DK>], cc, q8);
      }
    } else if constexpr (i < PER + IPER) {
      const int e = tid + NTH * (i - PER);
      if (IPIECES % NTH == 0 || e < IPIECES) *reinterpret_cast<u32x4_t*>(&b.img[e * 16]) = gi[i - PER];
    } else if constexpr (i < PER + IPER + 2) {
      constexpr int t = 2 * ((i - PER - IPER) % 2);
      *reinterpret_cast<u32x2_t*>(&lds_v[w][(16 * t + lr) * 16 + 4 * lq]) = gv[t];
      *reinterpret_cast<u32x2_t*>(&lds_v[w][(16 * t + 16 + lr) * 16 + 4 * lq]) = gv[t + 1];
      if constexpr (!KEEP) {
        const unsigned m = max_bf16x2(max_bf16x2(gv[t][0], gv[t][1]), max_bf16x2(gv[t + 1][0], gv[t + 1][1]));
        over = over || __any(max(m & 0x7fff0000u, m << 16) > limit);
      }
    } else {
      constexpr int e = i - PER - IPER - 2, t = 2 * (e % 2);
      __builtin_amdgcn_raw_buffer_store_b64(yo[t], ry, yrow + ctile, 32 * t * rowe32, 0);
      __builtin_amdgcn_raw_buffer_store_b64(yo[t + 1], ry, yrow + ctile, 32 * (t + 1) * rowe32, 0);
    }
  };

  // the largest finite |v| of the chunk that this wavefront has staged last
  auto staged_top = [&] {
    int own = threadIdx.x;  // (opaque: what only this needs is not carried through the loop)
    asm volatile("" : "+v"(own));
    const uint16_t* a = &lds_v[w][(own & 15) * 16 + 4 * ((own & 63) >> 4)];
    unsigned m = 0u;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const u32x2_t v = *reinterpret_cast<const u32x2_t*>(a + 256 * t);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        m = max(m, max(finite_bits(v[i] & 0x7fff0000u), finite_bits((v[i] << 16) & 0x7fff0000u)));
    }
    return m;
  };

  if (nchunks > 0) {
    next_rsrc(nchunks);
    static_for<LOADS>([&](auto i) { load_item(i); });
    next_rsrc(nchunks - 1);
    static_for<LOADS>([&](auto i) {
      stage_item(lds[0], i);
      load_item(i);
    });
  }
  if constexpr (KEEP) {
    ry = ys.take(nchunks);
    load_dy();
  }
  __syncthreads();
  if constexpr (!KEEP) {
    if (nchunks > 0) {
      unsigned top = staged_top();
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) top = max(top, finite_bits(__float_as_uint(S[d][r]) & 0x7fffffffu));
      top = wave_max(top);
      set_scale(top == 0u ? 0x1p60f : unit_scale(top, 5));  // nothing yet: the first value sets it
      over = false;
#pragma unroll
      for (int d = 0; d < DT; ++d) S[d] *= sc;
    }
  }
  f16x8_t Sh[KT], Sl[KT];
#pragma unroll
    for (int kk = 0; kk < KT; ++kk) split_f16(S[2 * kk], S[2 * kk + 1], Sh[kk], Sl[kk]);
  for (int c = 0; c < nchunks; ++c) {
    const Lds& b = lds[c & 1];
    Lds& next = lds[(c + 1) & 1];
    auto img_frag = [&](int base, int f) {
      return *reinterpret_cast<const f16x8_t*>(&b.img[base + f * kFrag + lane * 16]);
    };
    auto img_vec = [&](int base, int t) {  // four tokens 16 t + 4 lq .. + 3
      return *reinterpret_cast<const f32x4_t*>(&b.img[base + (16 * t + 4 * lq) * 4]);
    };
    const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    // ---- X = V - diag(e^cs) K S0, and Q S0 (as its transpose) beside it.  Steps (t, kk) in a row; the fragments of
    // step j + 3 are read before the products of step j.
    constexpr int STEPS = 4 * KT;
    f16x8_t kf[4], qf[4];
    auto read_step = [&](int j) {
      kf[j & 3] = lds_row_frag<DK>(b.k, 16 * (j / KT) + lr, j % KT, lq);
      qf[j & 3] = lds_row_frag<DK>(b.q, 16 * (j / KT) + lr, j % KT, lq);
    };
    f16x8_t th[6], tl[6];
    auto read_t = [&](int f) { th[f] = img_frag(kImgThi, f), tl[f] = img_frag(kImgTlo, f); };
    u32x2_t vq[4];
    const float fade = *reinterpret_cast<const float*>(&b.img[GATES + (kDeltaC - 1) * 4]);
#pragma unroll
    for (int j = 0; j < 3; ++j) read_step(j);
#pragma unroll
      for (int t = 0; t < 4; ++t) vq[t] = lds_tr4(&lds_v[w][(16 * t + 4 * lq + (lr >> 2)) * 16 + 4 * (lr & 3)]);
    __builtin_amdgcn_sched_barrier(0);
    next_rsrc(nchunks - c - 2);
    if constexpr (KEEP) {
      ry = ys.take(nchunks - c - 1);
      rkeep = ss.take(1);
    } else {
      ry = ys.take(c > 0 ? 2 : 0);  // of the chunk before, which is whole
      if (c == 0) ys.base -= ys.step;
    }
    // this chunk's share of ITEMS, in slots evenly spread over its products
    constexpr int SLOTS = STEPS + 3 + 2 * KT;
    auto slot = [&](auto place) {
      constexpr int k = decltype(place)::value, i0 = k * ITEMS / SLOTS, i1 = (k + 1) * ITEMS / SLOTS;
      static_for<i1 - i0>([&](auto i) {
        stage_item(next, IC<i0 + decltype(i)::value>{});
        load_item(IC<i0 + decltype(i)::value>{});
      });
      __builtin_amdgcn_sched_barrier(0);
    };
    f32x4_t x[4], o[4], grow[2];
    f16x8_t Xh[2], Xl[2];
    const float vsc = KEEP ? sc * kBwdXUp : sc;
    auto finish_x = [&](int t) {
      const float v[4] = {bf16_lo(vq[t][0]), bf16_hi(vq[t][0]), bf16_lo(vq[t][1]), bf16_hi(vq[t][1])};
#pragma unroll
      for (int r = 0; r < 4; ++r) x[t][r] = __builtin_fmaf(-grow[t & 1][r], x[t][r], v[r] * vsc);
      if (t & 1) split_f16(x[t - 1], x[t], Xh[t >> 1], Xl[t >> 1]);
    };
    static_for<STEPS>([&](auto step) {
      constexpr int j = decltype(step)::value, t = j / KT, kk = j % KT;
      if constexpr (j + 3 < STEPS)
        read_step(j + 3);
      else
        read_t(j + 3 - STEPS);
      if (kk == KT - 1) grow[t & 1] = img_vec(GATES, t) * (KEEP ? kBwdXUp / kBwdStateUp : 1.0f);
      __builtin_amdgcn_sched_barrier(0);
      if (kk == 0) x[t] = o[t] = zero;
      x[t] = mfma_f16(kf[j & 3], Sl[kk], x[t]);
      o[t] = mfma_f16(Sh[kk], qf[j & 3], o[t]);
      x[t] = mfma_f16(kf[j & 3], Sh[kk], x[t]);
      // (S0 q) . dy goes into the gradient of a fade, which needs both parts of S0
      if constexpr (KEEP) o[t] = mfma_f16(Sl[kk], qf[j & 3], o[t]);
      if constexpr (KEEP && j < 2 * KT)
        store_b128(__builtin_bit_cast(u32x4_t, j < KT ? Sh[j] : Sl[j - KT]), rkeep, mine + j * kFrag);
      if constexpr (kk == 0 && t > 0) finish_x(t - 1);
      // the state itself (its operands are copies) fades here, out of the chain
#pragma unroll
      for (int d = j * DT / STEPS; d < (j + 1) * DT / STEPS; ++d) S[d] *= fade;
      slot(IC<j>{});
    });
    finish_x(3);
    // An X that is not finite (a NaN in padding behind the tokens that count, say) would meet T's zeros in the next
    // products, and R's in those of P.  So X from a channel's first such token on is taken out here, and y from there on
    // and the state are set to NaN at the end.
    bool broken = false;
    if constexpr (!KEEP) {
      f16x2_t sum = {static_cast<_Float16>(0.0f), static_cast<_Float16>(0.0f)};  // of zeros times X
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f16x2_t v = {Xh[m][2 * e], Xh[m][2 * e + 1]};
          sum = __builtin_elementwise_fma(v, f16x2_t{static_cast<_Float16>(0.0f), static_cast<_Float16>(0.0f)}, sum);
        }
      broken = __any(sum[0] != sum[0] || sum[1] != sum[1]);
      if (broken) {
        int own = threadIdx.x & 63;  // (opaque, as above)
        asm volatile("" : "+v"(own));
        auto token = [&](int m, int e) { return 32 * m + (e < 4 ? 0 : 16) + 4 * (own >> 4) + (e & 3); };
        int first = kDeltaC;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            first = !(__builtin_fabsf(static_cast<float>(Xh[m][e])) <= 65504.0f) ? min(first, token(m, e)) : first;
        first = min(first, __shfl_xor(first, 16, 64));
        first = min(first, __shfl_xor(first, 32, 64));
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (token(m, e) >= first) Xh[m][e] = Xl[m][e] = static_cast<_Float16>(0.0f);
        lds_first[w][own & 15] = first;
      }
    }
    // ---- R = T X
    __builtin_amdgcn_sched_barrier(0);
    read_t(3);
    read_t(4);
    read_t(5);
    f32x4_t left[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      left[t] = img_vec(KEEP ? GATES + 512 : kImgLeft, t);
      if constexpr (KEEP) left[t] *= img_vec(GATES + 768, t) * kBwdStateUp;
    }
    f16x8_t kc[DT];  // K^T, a half of the tokens at a time
#pragma unroll
    for (int d = 0; d < DT; ++d) kc[d] = lds_col_frag<DK>(b.kt, 0, d, lr, lq);
    __builtin_amdgcn_sched_barrier(0);
    f32x4_t u[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) u[t] = zero;
    auto t_product = [&](int t, int m, int i) {
      const int f = frag_of(t, m);
      u[t] = mfma_f16(i == 2 ? tl[f] : th[f], i == 1 ? Xl[m] : Xh[m], u[t]);
    };
    static_for<3>([&](auto i) {
      t_product(0, 0, i.value);
      t_product(1, 0, i.value);
      t_product(2, 0, i.value);
      t_product(3, 0, i.value);
      slot(IC<STEPS + decltype(i)::value>{});
    });
    // ---- S = e^{cs_C} S + K^T diag(e^{cs_C - cs} b) R
    f16x8_t Uh[2], Ul[2];
    static_for<3>([&](auto i) {
      t_product(2, 1, i.value);
      t_product(3, 1, i.value);
    });
    if constexpr (KEEP) {
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] *= 1.0f / (kBwdXUp * kBwdTUp);
    }
    split_f16(u[0] * left[0], u[1] * left[1], Uh[0], Ul[0]);
    auto state_product = [&](int d, int m) {
      S[d] = mfma_f16(kc[d], Uh[m], S[d]);
      S[d + 1] = mfma_f16(kc[d + 1], Uh[m], S[d + 1]);
      S[d] = mfma_f16(kc[d], Ul[m], S[d]);
      S[d + 1] = mfma_f16(kc[d + 1], Ul[m], S[d + 1]);
    };
    static_for<KT>([&](auto k) {
      constexpr int d = 2 * decltype(k)::value;
      state_product(d, 0);
      kc[d] = lds_col_frag<DK>(b.kt, 32, d, lr, lq);
      kc[d + 1] = lds_col_frag<DK>(b.kt, 32, d + 1, lr, lq);
      slot(IC<STEPS + 3 + decltype(k)::value>{});
    });
    f16x8_t Rf[2];
    split_f16(u[2] * left[2], u[3] * left[3], Uh[1], Ul[1]);
    f16x8_t pf[KEEP ? 1 : 6];
    float og[4];
    if constexpr (KEEP) {
      rkeep = rs.take(1);
      f16x8_t Rl;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        split_f16(u[2 * m], u[2 * m + 1], Rf[m], Rl);
        store_b128(__builtin_bit_cast(u32x4_t, Rf[m]), rkeep, mine + m * kFrag);
        store_b128(__builtin_bit_cast(u32x4_t, Rl), rkeep, mine + (2 + m) * kFrag);
      }
      og[0] = *reinterpret_cast<const float*>(&b.img[GATES + 256 + lane * 4]);
    } else {
      Rf[0] = pair_f16(u[0], u[1]), Rf[1] = pair_f16(u[2], u[3]);
#pragma unroll
      for (int t = 0; t < 4; ++t) og[t] = *reinterpret_cast<const float*>(&b.img[GATES + (16 * t + lr) * 4]);
#pragma unroll
      for (int f = 0; f < 6; ++f) pf[f] = img_frag(kImgP, f);
    }
    __builtin_amdgcn_sched_barrier(0);
    // the next chunk's operands of the state are split under the products of the following tiles
    static_for<KT>([&](auto k) {
      constexpr int kk = decltype(k)::value, d = 2 * kk;
      state_product(d, 1);
      if constexpr (kk > 0) split_f16(S[d - 2], S[d - 1], Sh[kk - 1], Sl[kk - 1]);
      slot(IC<STEPS + 3 + KT + kk>{});
    });
    if constexpr (KEEP) {
      // (S0 q) . dy over these 16 channels: token 16 t + lr's four channels of each lane group, then the groups
      float dots[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float d[4] = {bf16_lo(yo[t][0]), bf16_hi(yo[t][0]), bf16_lo(yo[t][1]), bf16_hi(yo[t][1])};
        dots[t] = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          dots[t] = __builtin_fmaf(o[t][r], d[r], dots[t]);
          amax = __builtin_fmaxf(amax, __builtin_fabsf(d[r]));
        }
      }
      split_f16(S[DT - 2], S[DT - 1], Sh[KT - 1], Sl[KT - 1]);
      load_dy();
      // lane 16 lq + lr ends with token 16 lq + lr
      const bool odd = lq & 1, high = lq & 2;
      const float a0 = (odd ? dots[1] : dots[0]) + __shfl_xor(odd ? dots[0] : dots[1], 16, 64);
      const float a1 = (odd ? dots[3] : dots[2]) + __shfl_xor(odd ? dots[2] : dots[3], 16, 64);
      const float dot = (high ? a1 : a0) + __shfl_xor(high ? a0 : a1, 32, 64);
      rkeep = os.take(1);
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(dot * og[0] * (inv / kBwdStateUp)), rkeep,
                                            lane * 4 + (col < p.P ? 0 : kPastEnd), 0, 0);
    } else {
      // ---- Y^T = ((Q S0)^T diag(e^cs) + R^T P^T) scale
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] *= og[t];
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] = mfma_f16(Rf[0], pf[frag_of(t, 0)], o[t]);
#pragma unroll
      for (int t = 2; t < 4; ++t) o[t] = mfma_f16(Rf[1], pf[frag_of(t, 1)], o[t]);
      split_f16(S[DT - 2], S[DT - 1], Sh[KT - 1], Sl[KT - 1]);
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] *= yscale;
      if (broken) {
        int own = threadIdx.x & 63;
        asm volatile("" : "+v"(own));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int from = lds_first[w][4 * (own >> 4) + r];  // of this lane's channels of y
#pragma unroll
          for (int t = 0; t < 4; ++t) o[t][r] = 16 * t + (own & 15) >= from ? __builtin_nanf("") : o[t][r];
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        yo[t] = u32x2_t{pack_bf16x2(o[t][0], o[t][1]), pack_bf16x2(o[t][2], o[t][3])};
      }
      if (broken || over) {
        int own = threadIdx.x & 15;
        asm volatile("" : "+v"(own));
        float by = broken && lds_first[w][own] < kDeltaC ? __builtin_nanf("") : 1.0f;
        const unsigned top = wave_max(staged_top());
        if (__uint_as_float(top) > __uint_as_float(limit)) {
          const float was = inv;
          set_scale(unit_scale(top, 5));
          by *= sc * was;
        }
        over = false;
#pragma unroll
        for (int d = 0; d < DT; ++d) S[d] *= by;
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) split_f16(S[2 * kk], S[2 * kk + 1], Sh[kk], Sl[kk]);
      }
    }
    __syncthreads();
  }
  if constexpr (KEEP) {
    if (nchunks > 0 && col < p.P) {
      if (keep.dfinal) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const f32x4_t f = *reinterpret_cast<const f32x4_t*>(keep.dfinal + sbase + 16 * d);
#pragma unroll
          for (int r = 0; r < 4; ++r) amax = __builtin_fmaxf(amax, __builtin_fabsf(f[r]));
        }
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) amax = __builtin_fmaxf(amax, __shfl_xor(amax, o, 64));
      // a maximum does not depend on the order of its arguments, so neither does the scale
      if (lane == 0) atomicMax(p.amax + unit, __float_as_uint(amax));
    }
  } else {
    if (nchunks > 0) {
      ry = ys.take(1);
      static_for<2>([&](auto i) { stage_item(lds[0], IC<LOADS + decltype(i)::value>{}); });
    }
    if (p.hT) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
        if (col < p.P) *reinterpret_cast<f32x4_t*>(p.hT + sbase + 16 * d) = S[d] * inv;
    }
  }
}

}  // namespace ssm
