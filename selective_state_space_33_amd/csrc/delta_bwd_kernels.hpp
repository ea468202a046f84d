// delta_bwd_kernels.hpp -- the gradients of the gated delta rule, chunk by
// chunk (delta_chunk.hpp has the forward's mathematics and the operand order).
//
// With dS the adjoint that reaches a chunk's last state S_C, P taken without b
// (P0_tj = scale e^{cs_t - cs_j} q_t . k_j), L_j = e^{cs_C - cs_j}, U = diag(b) R:
//   Y0  = P0^T dY + diag(L) K dS,   dV = T^T diag(b) Y0,
//   dS0 = e^{cs_C} dS + Q^T diag(scale e^cs) dY - K^T diag(e^cs) dV,
//   dq_t = scale (e^{cs_t} S0 dy_t + sum_{j<=t} e^{cs_t - cs_j} (dy_t . u_j) k_j)
//   w_j  = L_j dS r_j + sum_{t>=j} scale e^{cs_t - cs_j} (dy_t . r_j) q_t
//                     - sum_{t>j} e^{cs_t - cs_j} (dv_t . r_j) k_t
//   dk_j = b_j w_j - e^{cs_j} S0 dv_j - sum_{i<j} e^{cs_j - cs_i} (dv_j . u_i) k_i,   db_j = k_j . w_j,
// and the gradient of the log fade of token t collects every term whose path
// crosses it:
//   dla_t = e^{cs_C} <dS, S0> + sum_{s>=t} e^{cs_s} (scale (S0 q_s) . dy_s - (S0 k_s) . dv_s)
//         + sum_{j<t} L_j (dS k_j) . u_j + sum_{j<t<=s} (P0_sj dy_s - N_sj dv_s) . u_j.
// (y . dy - v . dv, summed over the tokens behind t, is the same number, but as
// a small difference of large sums: in a fast-fading head it costs three
// digits.  The pair terms c_sj of the last sum are summed as rows less columns
// in fp64, where those that do not cross t cancel exactly.)  No term divides by
// b or by a fade.
//
// Four kernels: delta_prep_kernel<., true> (T, P0, gates of all chunks);
// delta_walk_kernel<., ., true> walks forward and keeps each chunk's S0 and R;
// delta_bwd_walk_kernel walks back, a wavefront holding 16 channels of dS as the
// forward's holds S, writes dV and keeps it and dS; delta_grad_kernel forms dq,
// dk, db and dla of all chunks at once, a workgroup per chunk and key head,
// which sums its heads in order.  2 x 4096 tokens of 40 heads of 128 channels,
// dstate 128: 86, 277, 350 and 304 us.  The walks are bound by their chunks'
// chain (64 chunks, 4.3 and 5.5 us each, 160 of the 256 CUs), the last by
// latency at two workgroups a CU (740 MB, 2.4 TB/s).
//
// Precision.  What goes from chunk to chunk, dV and every term of dla is a pair
// of fp16 (22 bits) in fp32 accumulators.  dY and what is linear in it may have
// any magnitude, so a unit's dY and final gradient are scaled by the power of
// two that brings their largest element to [16, 32) and the results scaled back,
// both exactly; dq, dk and db, stored as bf16, take their operands as one fp16.
#pragma once

#include "delta_prep_kernel.hpp"
#include "delta_walk_kernel.hpp"

namespace ssm {

// bf16 values as floats, times a scale.
__device__ __forceinline__ f32x4_t bf16x4_f32(u32x2_t v, float s) {
  return f32x4_t{bf16_lo(v[0]) * s, bf16_hi(v[0]) * s, bf16_lo(v[1]) * s, bf16_hi(v[1]) * s};
}
// acc + v * (hi + lo) of a pair, element by element.
__device__ __forceinline__ f32x4_t fma_pair(f32x4_t v, f16x4_t hi, f16x4_t lo, f32x4_t acc) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
    acc[r] = __builtin_fmaf(v[r], static_cast<float>(hi[r]), __builtin_fmaf(v[r], static_cast<float>(lo[r]), acc[r]));
  return acc;
}

// Sums of sixteen values over the 16 lanes of a row: lane lr receives the sum of value lr.  Each step exchanges the half
// of the values that the partner keeps; the masks 15, 7, 2, 1 are the lane permutations a DPP row has.
template <int CTRL> __device__ __forceinline__ float dpp_move(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float sum_rows16(const f32x4_t (&v)[4], int lr) {
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float lo = v[i >> 2][i & 3], hi = v[2 + (i >> 2)][i & 3];
    a[i] = (lr & 8 ? hi : lo) + dpp_move<0x140>(lr & 8 ? lo : hi);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = (lr & 4 ? a[i + 4] : a[i]) + dpp_move<0x141>(lr & 4 ? a[i] : a[i + 4]);
#pragma unroll
  for (int i = 0; i < 2; ++i) c[i] = (lr & 2 ? b[i + 2] : b[i]) + dpp_move<0x4e>(lr & 2 ? b[i] : b[i + 2]);
  return (lr & 1 ? c[1] : c[0]) + dpp_move<0xb1>(lr & 1 ? c[0] : c[1]);
}

// A fragment of rows (paired order) of an array stored plain.
template <int LD> __device__ __forceinline__ f16x8_t plain_row_frag(const uint16_t* base, int r, int kk, int lq) {
  const uint16_t* a = base + r * LD + 32 * kk + 4 * lq;
  const u32x2_t x = *reinterpret_cast<const u32x2_t*>(a), y = *reinterpret_cast<const u32x2_t*>(a + 16);
  return __builtin_bit_cast(f16x8_t, u32x4_t{x[0], x[1], y[0], y[1]});
}

// A tensor's chunks from the last one back, as DeltaStream the other way.
struct DeltaBackStream {
  char* base;
  int64_t step;
  int size, full;
  // the chunk at p (of `last` bytes) first, then those before it, `chunk` bytes apart and `whole` long
  __device__ __forceinline__ DeltaBackStream(const void* p, int64_t chunk, int64_t last, int64_t whole)
      : base(static_cast<char*>(const_cast<void*>(p))),
        step(chunk),
        size(static_cast<int>(last)),
        full(static_cast<int>(whole)) {}
  __device__ __forceinline__ rsrc_t take(bool go) {
    const rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(base, 0, go ? size : 0, kBufWord3);
    base -= go ? step : 0;
    size = go ? full : size;
    return r;
  }
};

template <int DK> struct DeltaBackLds {
  __attribute__((aligned(16))) uint16_t k[kDeltaC * kColLd<DK>];
  __attribute__((aligned(16))) uint16_t q[kDeltaC * kColLd<DK>];
  __attribute__((aligned(16))) char img[24 * kFrag + 1024];  // the transposes of T and P0 (pairs) and four gates
};

// The walk back with the adjoint.  As delta_walk_kernel, a wavefront owns 16 channels and the chunk's operands are staged
// a chunk ahead, item by item between the products.  Per chunk (dstate 128) 176 MFMAs: K dS and K S0 32 each, P0^T dY 12,
// <dS, S0> 12, T^T (b Y0) 18 and 6 for dV's rows, Q^T dY 32, K^T dV 32.  The chain is K dS -> b Y0 -> dV -> K^T dV; the
// rest fills it.  S0 and R are loaded for the chunk before as soon as this chunk has read them.
template <int DK, int W> __global__ void __launch_bounds__(64 * W) delta_bwd_walk_kernel(DeltaBwdParams bp) {
  const DeltaChunkParams& p = bp.c;
  constexpr int KT = DK / 32, DT = DK / 16, NTH = 64 * W, CL = kColLd<DK>;
  using Lds = DeltaBackLds<DK>;
  constexpr int GATES = 24 * kFrag;
  __shared__ Lds lds[2];
  __shared__ __attribute__((aligned(16))) uint16_t lds_y[W][kDeltaC * 16];  // each wavefront's dY, [token][channel]
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t blocks = (p.P + 16 * W - 1) / (16 * W);
  const DeltaUnit un = delta_unit(p, blocks);
  const int64_t seq = un.seq, h = un.h, unit = seq * p.H + h, g = key_head(h, p.H, p.G);
  const int col = static_cast<int>(un.block * W + w) * 16;
  const DeltaSeq sq = delta_seq(p.cu, seq, p.L, p.chunks);
  const int nchunks = static_cast<int>((sq.len + kDeltaC - 1) / kDeltaC);
  const int64_t rowe = p.H * p.P, krow = p.G * DK;
  const int rowe32 = static_cast<int>(rowe), krow32 = static_cast<int>(krow);
  const int yrow = (lr * rowe32 + 4 * lq) * 2;
  const float sc = nchunks > 0 ? grad_scale(p.amax[unit]) : 1.0f, inv = 1.0f / sc;
  // of what R enters too, and of what S0 does
  const float both = nchunks > 0 ? inv / p.vscale[unit] : 1.0f, state = both / kBwdStateUp;

  // ---- dS (scaled): channel col + lr, states 16 d + 4 lq .. + 3
  f32x4_t S[DT];
  const int64_t sbase = (unit * p.P + col + lr) * DK + 4 * lq;
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    S[d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (bp.dfinal && col < p.P) S[d] = *reinterpret_cast<const f32x4_t*>(bp.dfinal + sbase + 16 * d) * sc;
  }

  // ---- chunk loads, one chunk ahead in registers (items and resources as in delta_walk_kernel)
  constexpr int PIECES = kDeltaC * DK / 8, PER = (PIECES + NTH - 1) / NTH;
  constexpr int IPIECES = sizeof(Lds::img) / 16, IPER = (IPIECES + NTH - 1) / NTH;
  const bool has = col < p.P;
  const int ctile = has ? col * 2 : kPastEnd, mine = lane * 16 + (has ? 0 : kPastEnd);
  const int mine4 = lane * 4 + (has ? 0 : kPastEnd);
  // where lane (lq, lr) puts the sum of sum_rows16's value lr, which belongs to token 16 (lr / 4) + 4 lq + lr % 4
  const int term_at = (16 * (lr >> 2) + 4 * lq + (lr & 3)) * 4 + (has ? 0 : kPastEnd);
  const int64_t lastc = nchunks - 1, ltok = sq.tok + lastc * kDeltaC, last = sq.len - lastc * kDeltaC;
  const int64_t kb = ltok * krow + g * DK, vb = ltok * rowe + h * p.P;
  const int64_t kstep = krow * kDeltaC * 2, vstep = rowe * kDeltaC * 2;
  const int64_t ktail = ((last - 1) * krow + DK) * 2, kfull = ((kDeltaC - 1) * krow + DK) * 2;
  const int64_t vtail = ((last - 1) * rowe + p.P) * 2, vfull = ((kDeltaC - 1) * rowe + p.P) * 2;
  const int64_t lcell = (sq.slot + lastc) * p.H + h, tcell = lcell * bp.tiles + col / 16, tcells = p.H * bp.tiles;
  DeltaBackStream ks(static_cast<const uint16_t*>(p.k) + kb, kstep, ktail, kfull);
  DeltaBackStream qs(static_cast<const uint16_t*>(p.q) + kb, kstep, ktail, kfull);
  DeltaBackStream ys(static_cast<const uint16_t*>(bp.dy) + vb, vstep, vtail, vfull);
  DeltaBackStream os(static_cast<const uint16_t*>(bp.dv) + vb, vstep, vtail, vfull);
  DeltaBackStream is(p.img + lcell * kBwdImgBytes + kBwdBack, p.H * kBwdImgBytes, sizeof(Lds::img), sizeof(Lds::img));
  auto tile_stream = [&](const void* base, int bytes) {
    return DeltaBackStream(static_cast<const char*>(base) + tcell * bytes, tcells * bytes, bytes, bytes);
  };
  DeltaBackStream ss = tile_stream(bp.state, 2 * KT * kFrag), rs = tile_stream(bp.r, 4 * kFrag);
  DeltaBackStream as = tile_stream(bp.adj, KT * kFrag), vs = tile_stream(bp.dvh, 4 * kFrag);
  DeltaBackStream ls = tile_stream(bp.lterm, kDeltaC * 4), gs = tile_stream(bp.gterm, kDeltaC * 4);
  DeltaBackStream es = tile_stream(bp.edge, kDeltaC * 4);
  u32x4_t gk[PER], gq[PER], gi[IPER];
  u32x2_t gd[4], yo[4];  // dY of the next chunk; dV of the last, stored during this one
  f16x8_t s0[2 * KT], r0[4];
  constexpr int LOADS = PER + IPER + 2, ITEMS = LOADS + 2;
  rsrc_t rk, rq, ri, ry, ro, rs0, rr0;
  auto next_rsrc = [&](bool go) { rk = ks.take(go), rq = qs.take(go), ri = is.take(go), ry = ys.take(go); };
  auto load_item = [&](auto item) {
    constexpr int i = decltype(item)::value;
    if constexpr (i < PER) {
      const int e = tid + NTH * i;
      const int off = (e / (DK / 8)) * krow32 * 2 + (e % (DK / 8)) * 16;
      gk[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, 0));
      gq[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rq, off, 0, 0));
    } else if constexpr (i < PER + IPER) {
      constexpr int e = i - PER;
      gi[e] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ri, (tid + NTH * e) * 16, 0, 0));
    } else if constexpr (i < LOADS) {
      constexpr int t = 2 * (i - PER - IPER);
      const int at = yrow + ctile;
      gd[t] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(ry, at, 32 * t * rowe32, 0));
      gd[t + 1] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(ry, at, 32 * (t + 1) * rowe32, 0));
    }
  };
  auto stage_item = [&](Lds& b, auto item) {
    constexpr int i = decltype(item)::value;
    if constexpr (i < PER) {
      const int e = tid + NTH * i, at = (e / (DK / 8)) * CL + (e % (DK / 8)) * 8;
      if (PIECES % NTH == 0 || e < PIECES) {
        *reinterpret_cast<u32x4_t*>(&b.k[at]) = bf16x8_as_f16(gk[i]);
        *reinterpret_cast<u32x4_t*>(&b.q[at]) = bf16x8_as_f16(gq[i]);
      }
    } else if constexpr (i < PER + IPER) {
      const int e = tid + NTH * (i - PER);
      if (IPIECES % NTH == 0 || e < IPIECES) *reinterpret_cast<u32x4_t*>(&b.img[e * 16]) = gi[i - PER];
    } else if constexpr (i < LOADS) {
      constexpr int t = 2 * (i - PER - IPER);
      *reinterpret_cast<u32x2_t*>(&lds_y[w][(16 * t + lr) * 16 + 4 * lq]) = gd[t];
      *reinterpret_cast<u32x2_t*>(&lds_y[w][(16 * t + 16 + lr) * 16 + 4 * lq]) = gd[t + 1];
    } else {
      constexpr int t = 2 * (i - LOADS);
      __builtin_amdgcn_raw_buffer_store_b64(yo[t], ro, yrow + ctile, 32 * t * rowe32, 0);
      __builtin_amdgcn_raw_buffer_store_b64(yo[t + 1], ro, yrow + ctile, 32 * (t + 1) * rowe32, 0);
    }
  };
  auto load_s0 = [&](int kk) {
    s0[kk] = __builtin_bit_cast(f16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rs0, mine, kk * kFrag, 0));
    s0[KT + kk] = __builtin_bit_cast(f16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rs0, mine, (KT + kk) * kFrag, 0));
  };
  auto load_r = [&](int m) {
    r0[m] = __builtin_bit_cast(f16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rr0, mine, m * kFrag, 0));
    r0[2 + m] = __builtin_bit_cast(f16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rr0, mine, (2 + m) * kFrag, 0));
  };

  if (nchunks > 0) {
    next_rsrc(true);
    static_for<LOADS>([&](auto i) { load_item(i); });
    rs0 = ss.take(true), rr0 = rs.take(true);
    static_for<KT>([&](auto kk) { load_s0(kk.value); });
    load_r(0);
    load_r(1);
    next_rsrc(nchunks > 1);
    static_for<LOADS>([&](auto i) {
      stage_item(lds[0], i);
      load_item(i);
    });
  }
  __syncthreads();
  f16x8_t Sh[KT], Sl[KT];
#pragma unroll
  for (int kk = 0; kk < KT; ++kk) split_f16(S[2 * kk], S[2 * kk + 1], Sh[kk], Sl[kk]);
  for (int i = 0; i < nchunks; ++i) {
    const Lds& b = lds[i & 1];
    Lds& next = lds[(i + 1) & 1];
    auto img_frag = [&](int f) { return *reinterpret_cast<const f16x8_t*>(&b.img[f * kFrag + lane * 16]); };
    auto gate = [&](int which, int t) {
      return *reinterpret_cast<const f32x4_t*>(&b.img[GATES + which * 256 + (16 * t + 4 * lq) * 4]);
    };
    const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int STEPS = 4 * KT;
    // tokens' tiles in the order 2, 3, 0, 1: T^T takes the last two first
    auto tile_of = [](int j) { return (j / KT + 2) & 3; };
    f16x8_t kf[4];
    auto read_step = [&](int j) { kf[j & 3] = plain_row_frag<CL>(b.k, 16 * tile_of(j) + lr, j % KT, lq); };
    u32x2_t tq[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) tq[t] = lds_tr4(&lds_y[w][(16 * t + 4 * lq + (lr >> 2)) * 16 + 4 * (lr & 3)]);
    f32x4_t outg[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) outg[t] = gate(1, t);
    const float fade = *reinterpret_cast<const float*>(&b.img[GATES + (kDeltaC - 1) * 4]);
    f16x8_t pf[6];
#pragma unroll
    for (int f = 0; f < 6; ++f) pf[f] = img_frag(18 + f);
    __builtin_amdgcn_sched_barrier(0);
    next_rsrc(i + 2 < nchunks);
    ro = os.take(i > 0);  // of the chunk before this one in the walk
    rs0 = ss.take(i + 1 < nchunks), rr0 = rs.take(i + 1 < nchunks);
    const rsrc_t ra = as.take(true);
    constexpr int SLOTS = STEPS + 2 * KT;
    auto slot = [&](auto place) {
      constexpr int k = decltype(place)::value, i0 = k * ITEMS / SLOTS, i1 = (k + 1) * ITEMS / SLOTS;
      static_for<i1 - i0>([&](auto n) {
        stage_item(next, IC<i0 + decltype(n)::value>{});
        load_item(IC<i0 + decltype(n)::value>{});
      });
      __builtin_amdgcn_sched_barrier(0);
    };
    // ---- P0^T dY (16 times as large), and dY's operands (Df is exact: bf16 values scaled by a power of two)
    f32x4_t wy[4];
    f16x8_t Gh[2], Gl[2], Df[2];
    {
      f32x4_t d[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) d[t] = bf16x4_f32(tq[t], sc), wy[t] = zero;
      Df[0] = pair_f16(d[0], d[1]), Df[1] = pair_f16(d[2], d[3]);
#pragma unroll
      for (int part = 0; part < 2; ++part) {
#pragma unroll
        for (int m = 1; m >= 0; --m)
#pragma unroll
          for (int t = 0; t < 2 + 2 * m; ++t) wy[t] = mfma_f16(pf[back_frag(t, m)], Df[m], wy[t]);
        if (part == 0) {
#pragma unroll
          for (int f = 0; f < 6; ++f) pf[f] = img_frag(12 + f);
#pragma unroll
          for (int j = 0; j < 3; ++j) read_step(j);
#pragma unroll
          for (int m = 0; m < 2; ++m) split_f16(d[2 * m] * outg[2 * m], d[2 * m + 1] * outg[2 * m + 1], Gh[m], Gl[m]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    // ---- K dS, and K S0 and <dS, S0> beside it
    f32x4_t x[4], z[4], e0 = zero, e1 = zero, lt[4], left, beta;
    f16x8_t Zh[2], Zl[2], tf[12];
    // b Y0 of a tile, and on the way L (K dS) . u of its tokens
    auto finish = [&](int t) {
      const int m = t >> 1;
      const f32x4_t lx = x[t] * left;
      const f16x8_t hi = r0[m], lo = r0[2 + m];
      lt[t] = t & 1 ? fma_pair(lx * beta, __builtin_shufflevector(hi, hi, 4, 5, 6, 7),
                               __builtin_shufflevector(lo, lo, 4, 5, 6, 7), zero)
                    : fma_pair(lx * beta, __builtin_shufflevector(hi, hi, 0, 1, 2, 3),
                               __builtin_shufflevector(lo, lo, 0, 1, 2, 3), zero);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[t][r] = beta[r] * __builtin_fmaf(wy[t][r], 1.0f / kBwdPScale, lx[r]);
      if (t & 1) {
        split_f16(x[t - 1], x[t], Zh[m], Zl[m]);
        load_r(m);
      }
    };
    static_for<STEPS>([&](auto step) {
      constexpr int j = decltype(step)::value, kk = j % KT;
      const int t = tile_of(j);
      if constexpr (j + 3 < STEPS)
        read_step(j + 3);
      else {  // T^T's fragments of tokens 32 .. 63
        tf[j + 3 - STEPS] = img_frag(back_frag(j + 3 - STEPS, 1));
        tf[6 + j + 3 - STEPS] = img_frag(6 + back_frag(j + 3 - STEPS, 1));
      }
      if (kk == KT - 1) left = gate(2, t), beta = gate(3, t);
      __builtin_amdgcn_sched_barrier(0);
      if (kk == 0) x[t] = z[t] = zero;
      x[t] = mfma_f16(kf[j & 3], Sl[kk], x[t]);
      z[t] = mfma_f16(kf[j & 3], s0[KT + kk], z[t]);
      x[t] = mfma_f16(kf[j & 3], Sh[kk], x[t]);
      z[t] = mfma_f16(kf[j & 3], s0[kk], z[t]);
      if constexpr (j / KT == 0) {
        e0 = mfma_f16(Sl[kk], s0[kk], e0);
        e1 = mfma_f16(Sh[kk], s0[kk], e1);
        e0 = mfma_f16(Sh[kk], s0[KT + kk], e0);
        store_b128(__builtin_bit_cast(u32x4_t, Sh[kk]), ra, mine + kk * kFrag);
      }
      if constexpr (j / KT == 3) load_s0(kk);
      if constexpr (kk == KT - 1 && j + 1 < STEPS) finish(t);
      slot(IC<j>{});
    });
    // ---- dV = T^T (b Y0): the last two tiles' share of it while the rest of b Y0 is finished, Q^T dY between
    f32x4_t u[4], vt[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) u[t] = vt[t] = zero;
    tf[3] = img_frag(back_frag(3, 1)), tf[9] = img_frag(6 + back_frag(3, 1));
#pragma unroll
    for (int t = 0; t < 2; ++t) tf[4 + t] = img_frag(back_frag(t, 0)), tf[10 + t] = img_frag(6 + back_frag(t, 0));
    f16x8_t cf[DT];  // columns of Q, then of K
#pragma unroll
    for (int d = 0; d < DT; ++d) cf[d] = lds_col_frag<DK>(b.q, 0, d, lr, lq);
    f32x4_t grow[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) grow[t] = gate(0, t);
    __builtin_amdgcn_sched_barrier(0);
    auto t_products = [&](int t, int m) {
      const int f = m ? t : 4 + t;
      u[t] = mfma_f16(tf[f], Zh[m], u[t]);
      vt[t] = mfma_f16(Zh[m], tf[f], vt[t]);
      u[t] = mfma_f16(tf[f], Zl[m], u[t]);
      u[t] = mfma_f16(tf[6 + f], Zh[m], u[t]);
    };
    t_products(2, 1);
    t_products(3, 1);
    finish(tile_of(STEPS - 1));
    t_products(0, 1);
    t_products(1, 1);
    __builtin_amdgcn_sched_barrier(0);
    // What the chunk adds to dS, summed apart and added at the end: the products round at the size of what they add
    // (363 us so far, 350 now).
    f32x4_t more[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) more[d] = zero;
    auto state_product = [&](int d, const f16x8_t& hi, const f16x8_t& lo) {
      more[d] = mfma_f16(cf[d], lo, more[d]);
      more[d + 1] = mfma_f16(cf[d + 1], lo, more[d + 1]);
      more[d] = mfma_f16(cf[d], hi, more[d]);
      more[d + 1] = mfma_f16(cf[d + 1], hi, more[d + 1]);
    };
    auto take_more = [&](int d) {
#pragma unroll
      for (int r = 0; r < 4; ++r) S[d][r] = __builtin_fmaf(fade, S[d][r], more[d][r]);
    };
    static_for<KT>([&](auto k) {
      constexpr int d = 2 * decltype(k)::value;
      state_product(d, Gh[0], Gl[0]);
      cf[d] = lds_col_frag<DK>(b.q, 32, d, lr, lq);
      cf[d + 1] = lds_col_frag<DK>(b.q, 32, d + 1, lr, lq);
    });
    t_products(0, 0);
    t_products(1, 0);
    f16x8_t Vh[2], Vl[2], Nh, Nl;
    const rsrc_t rv = vs.take(true);
    f32x4_t gt[4];
    // dV of two tiles: kept as a pair, times -e^cs as the next product's operand; e^cs (S0 k) . dv of its tokens
    auto take_dv = [&](int m) {
      u[2 * m] *= 1.0f / kBwdTUp, u[2 * m + 1] *= 1.0f / kBwdTUp;
      split_f16(u[2 * m], u[2 * m + 1], Nh, Nl);
      store_b128(__builtin_bit_cast(u32x4_t, Nh), rv, mine + m * kFrag);
      store_b128(__builtin_bit_cast(u32x4_t, Nl), rv, mine + (2 + m) * kFrag);
      const f32x4_t v0 = u[2 * m] * -grow[2 * m], v1 = u[2 * m + 1] * -grow[2 * m + 1];
      split_f16(v0, v1, Vh[m], Vl[m]);
      gt[2 * m] = v0 * z[2 * m], gt[2 * m + 1] = v1 * z[2 * m + 1];
    };
    take_dv(1);
    __builtin_amdgcn_sched_barrier(0);
    static_for<KT>([&](auto k) {
      constexpr int d = 2 * decltype(k)::value;
      state_product(d, Gh[1], Gl[1]);
      cf[d] = lds_col_frag<DK>(b.k, 32, d, lr, lq);
      cf[d + 1] = lds_col_frag<DK>(b.k, 32, d + 1, lr, lq);
      slot(IC<STEPS + decltype(k)::value>{});
    });
    take_dv(0);
    // ---- dS = e^{cs_C} dS + Q^T diag(scale e^cs) dY - K^T diag(e^cs) dV
    static_for<KT>([&](auto k) {
      constexpr int d = 2 * decltype(k)::value;
      state_product(d, Vh[1], Vl[1]);
      cf[d] = lds_col_frag<DK>(b.k, 0, d, lr, lq);
      cf[d + 1] = lds_col_frag<DK>(b.k, 0, d + 1, lr, lq);
    });
    __builtin_amdgcn_sched_barrier(0);
    static_for<KT>([&](auto k) {
      constexpr int kk = decltype(k)::value, d = 2 * kk;
      state_product(d, Vh[0], Vl[0]);
      if constexpr (kk > 0) {
        take_more(d - 2);
        take_more(d - 1);
        split_f16(S[d - 2], S[d - 1], Sh[kk - 1], Sl[kk - 1]);
      }
      slot(IC<STEPS + KT + kk>{});
    });
    // ---- the terms of dla, and dV's rows
    rsrc_t rt = ls.take(true);
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sum_rows16(lt, lr) * both), rt, term_at, 0, 0);
    rt = gs.take(true);
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sum_rows16(gt, lr) * -state), rt, term_at, 0, 0);
    e0 += e1;  // its diagonal: each channel's <dS, S0>
    const float diag = (lr & 2) ? ((lr & 1) ? e0[3] : e0[2]) : ((lr & 1) ? e0[1] : e0[0]);
    rt = es.take(true);
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(lq == (lr >> 2) ? diag * fade * state : 0.0f), rt, mine4, 0,
                                          0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      vt[t] *= inv / kBwdTUp;
      yo[t] = u32x2_t{pack_bf16x2(vt[t][0], vt[t][1]), pack_bf16x2(vt[t][2], vt[t][3])};
    }
    take_more(DT - 2);
    take_more(DT - 1);
    split_f16(S[DT - 2], S[DT - 1], Sh[KT - 1], Sl[KT - 1]);
    __syncthreads();
  }
  if (nchunks > 0) {
    ro = os.take(true);
    static_for<2>([&](auto n) { stage_item(lds[0], IC<LOADS + decltype(n)::value>{}); });
  }
  if (bp.dh0 && has) {
#pragma unroll
    for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4_t*>(bp.dh0 + sbase + 16 * d) = S[d] * inv;
  }
}

constexpr int kGradLd = 40;   // halves per row of the 64 x 32 block of dY (4 x odd dwords, as kRowLd)
constexpr int kGradTok = 80;  // of the 32 x 64 blocks of R and dV, [channel][token] (8 x odd dwords, as kColLd)
constexpr int kGradTokLo = 72;  // of their lo parts (a bank twice: a narrower row lets two workgroups share a CU)
constexpr int kGradC = 65;    // floats per row of the 64 x 64 pair terms

template <int DK> struct DeltaGradLds {
  static constexpr int CL = kColLd<DK>;
  __attribute__((aligned(16))) uint16_t k[kDeltaC * CL], q[kDeltaC * CL];
  union {
    struct {
      __attribute__((aligned(16))) uint16_t r[32 * kGradTok], v[32 * kGradTok], rl[32 * kGradTokLo],
          vl[32 * kGradTokLo], y[kDeltaC * kGradLd], s[32 * CL], a[32 * CL];
    };
    struct {
      // once the blocks are read: the pair terms, rows less columns of them, and each wavefront's sums over its tiles
      float c[kDeltaC * kGradC];
      double e[kDeltaC], og[4][kDeltaC], l[4][kDeltaC], edge[4];
    };
    uint16_t out[2][kDeltaC * CL];  // at the end: dq and dk on their way to whole rows
  };
  __attribute__((aligned(16))) float g[6][kDeltaC];  // the image's gates
};

// A fragment whose K index is the channel (rows 0 .. 31 in paired order), columns the tokens 16 t + lr.
template <int LD> __device__ __forceinline__ f16x8_t tok_frag(const uint16_t* base, int t, int lr, int lq) {
  const uint16_t* a = base + (4 * lq + (lr >> 2)) * LD + 16 * t + 4 * (lr & 3);
  const u32x2_t x = lds_tr4(a), y = lds_tr4(a + 16 * LD);
  return __builtin_bit_cast(f16x8_t, u32x4_t{x[0], x[1], y[0], y[1]});
}

__device__ __forceinline__ float sum_wave(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <int DK> __global__ void __launch_bounds__(256, 2) delta_grad_kernel(DeltaBwdParams bp) {
  const DeltaChunkParams& p = bp.c;
  constexpr int KT = DK / 32, DT = DK / 16, CL = kColLd<DK>;
  __shared__ DeltaGradLds<DK> lds;
  uint16_t *const sK = lds.k, *const sQ = lds.q;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lr = lane & 15, lq = lane >> 4;
  const unsigned groups = static_cast<unsigned>(p.G);
  const unsigned id = xcd_order(blockIdx.x, static_cast<unsigned>(p.slots) * groups);
  const int64_t slot = id / groups, g = id % groups, rep = static_cast<unsigned>(p.H) / groups;
  int64_t s = 0;
  if (p.cu) {
    s = delta_slot_seq(p.cu, p.rows, p.L, slot);
  } else {
    s = static_cast<unsigned>(slot) / static_cast<unsigned>(p.chunks);
  }
  const DeltaSeq sq = delta_seq(p.cu, s, p.L, p.chunks);
  const int64_t c0 = (slot - sq.slot) * kDeltaC;
  if (slot < sq.slot || c0 >= sq.len) {  // a slot of no chunk adds nothing to dA and dbias
    for (int e = tid; e < 2 * rep; e += 256) bp.part[(slot * p.H + g * rep) * 2 + e] = 0.0f;
    return;
  }
  const int nt = static_cast<int>(sq.len - c0 < kDeltaC ? sq.len - c0 : kDeltaC);
  const int64_t tok = sq.tok + c0;
  const int64_t krow = p.G * DK, rowe = p.H * p.P;
  const int64_t kb = tok * krow + g * DK, kbytes = ((nt - 1) * krow + DK) * 2;
  constexpr int KPER = kDeltaC * DK / 8 / 256;
  {
    u32x4_t g_k[KPER], g_q[KPER];
    const rsrc_t rk = make_rsrc(static_cast<const uint16_t*>(p.k) + kb, kbytes);
    const rsrc_t rq = make_rsrc(static_cast<const uint16_t*>(p.q) + kb, kbytes);
#pragma unroll
    for (int i = 0; i < KPER; ++i) {
      const int e = tid + 256 * i, row = e / (DK / 8), cc = (e % (DK / 8)) * 8;
      const int off = static_cast<int>((row * krow + cc) * 2);
      g_k[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, 0));
      g_q[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rq, off, 0, 0));
    }
#pragma unroll
    for (int i = 0; i < KPER; ++i) {
      const int e = tid + 256 * i, row = e / (DK / 8), cc = (e % (DK / 8)) * 8;
      *reinterpret_cast<u32x4_t*>(&sK[row * CL + cc]) = bf16x8_as_f16(g_k[i]);
      *reinterpret_cast<u32x4_t*>(&sQ[row * CL + cc]) = bf16x8_as_f16(g_q[i]);
    }
  }
  const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4_t dq[DT], dk[DT];  // in the scale of the head at work
  float unscale = 1.0f;
#pragma unroll
  for (int d = 0; d < DT; ++d) dq[d] = dk[d] = zero;
  const int nb = static_cast<int>((bp.tiles + 1) / 2);  // blocks of 32 channels
  for (int64_t hh = 0; hh < rep; ++hh) {
    const int64_t h = g * rep + hh, cell = slot * p.H + h;
    // What a lane derives from its place is derived anew for every head: carried over the loop, the addresses and the
    // masks of the triangles took a hundred registers more than there are.
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, lr = lane & 15, lq = lane >> 4;
    const float scy = grad_scale(p.amax[s * p.H + h]), sc = scy * p.vscale[s * p.H + h], inv = 1.0f / sc;
    const int tbytes = static_cast<int>(bp.tiles * kFrag);
    const rsrc_t rr = make_rsrc(bp.r + cell * bp.tiles * (4 * kFrag), 4 * tbytes);
    const rsrc_t rv = make_rsrc(bp.dvh + cell * bp.tiles * (4 * kFrag), 4 * tbytes);
    const rsrc_t ry = make_rsrc(static_cast<const uint16_t*>(bp.dy) + tok * rowe + h * p.P, ((nt - 1) * rowe + p.P) * 2);
    const rsrc_t rs = make_rsrc(bp.state + cell * bp.tiles * (2 * KT * kFrag), 2 * KT * tbytes);
    const rsrc_t ra = make_rsrc(bp.adj + cell * bp.tiles * (KT * kFrag), KT * tbytes);
    constexpr int SP = 2 * KT * 64, SPER = (SP + 255) / 256;  // pieces of two tiles of states
    u32x4_t g_r[2], g_v[2], g_y, g_s[SPER], g_a[SPER];
    auto load = [&](int b) {
      const int row = tid >> 2, cc = 32 * b + 8 * (tid & 3);
      // (P is a multiple of 16: a piece is inside or outside)
      const int aty = cc < p.P ? static_cast<int>((row * rowe + cc) * 2) : kPastEnd;
      g_y = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ry, aty, 0, 0));
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // of two tiles: hi, lo x two halves of the tokens x 64 lanes
        const int at = 2 * b + i < bp.tiles ? (2 * b + i) * (4 * kFrag) + tid * 16 : kPastEnd;
        g_r[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rr, at, 0, 0));
        g_v[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rv, at, 0, 0));
      }
#pragma unroll
      for (int i = 0; i < SPER; ++i) {
        const int e = tid + 256 * i, u = e / (KT * 64), f = e % (KT * 64);
        const bool some = e < SP && 2 * b + u < bp.tiles;
        g_s[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                 rs, some ? (2 * b + u) * (2 * KT * kFrag) + f * 16 : kPastEnd, 0, 0));
        g_a[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                 ra, some ? (2 * b + u) * (KT * kFrag) + f * 16 : kPastEnd, 0, 0));
      }
    };
    // dy . r and dv . r.  Of the tiles of this wavefront's tokens (as t, lane by lane) with those before them: a1, a2 at
    // their tile; with those behind them (this wavefront's as j): a1, a2 at theirs; its tile with itself both ways.
    f32x4_t a1[4], a2[4], b1 = zero, b2 = zero, aw[DT];
#pragma unroll
    for (int t = 0; t < 4; ++t) a1[t] = a2[t] = zero;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      aw[d] = zero;
      dq[d] *= sc * unscale, dk[d] *= sc * unscale;  // from the last head's scale to this one's
    }
    unscale = inv;
    load(0);
    f32x4_t g_g = zero;  // the gates, a lane four
    if (tid < 6 * 16) g_g = *reinterpret_cast<const f32x4_t*>(p.img + cell * kBwdImgBytes + kBwdGates + tid * 16);
    // dla's terms of each token (a lane) over every fourth tile
    double og = 0.0, lt = 0.0, edge = 0.0;
    for (int64_t t = w; t < bp.tiles; t += 4) {
      const int64_t at = (cell * bp.tiles + t) * kDeltaC + lane;
      og += static_cast<double>(bp.oterm[at]) - static_cast<double>(bp.gterm[at]);
      lt += bp.lterm[at];
      edge += bp.edge[at];
    }
    for (int b = 0; b < nb; ++b) {
      __syncthreads();  // the last block (or head) is read
      if (b == 0 && tid < 6 * 16) *reinterpret_cast<f32x4_t*>(&lds.g[0][0] + tid * 4) = g_g;
      {
        const int row = tid >> 2, cc = 8 * (tid & 3);
        u32x4_t y8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f16x2_t hv = __builtin_convertvector((f32x2_t){bf16_lo(g_y[i]) * scy, bf16_hi(g_y[i]) * scy}, f16x2_t);
          y8[i] = __builtin_bit_cast(uint32_t, hv);
        }
        lds_store_paired(&lds.y[row * kGradLd], cc, y8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // fragment (hi | lo, half m), lane (channel lr, lq): tokens 32 m + 4 lq .. + 3 and + 16
          const int at = 32 * (w & 1) + 4 * lq, ch = 16 * i + lr;
          uint16_t* dr = w < 2 ? &lds.r[ch * kGradTok + at] : &lds.rl[ch * kGradTokLo + at];
          uint16_t* dv = w < 2 ? &lds.v[ch * kGradTok + at] : &lds.vl[ch * kGradTokLo + at];
          *reinterpret_cast<u32x2_t*>(dr) = u32x2_t{g_r[i][0], g_r[i][1]};
          *reinterpret_cast<u32x2_t*>(dr + 16) = u32x2_t{g_r[i][2], g_r[i][3]};
          *reinterpret_cast<u32x2_t*>(dv) = u32x2_t{g_v[i][0], g_v[i][1]};
          *reinterpret_cast<u32x2_t*>(dv + 16) = u32x2_t{g_v[i][2], g_v[i][3]};
        }
#pragma unroll
        for (int i = 0; i < SPER; ++i) {
          const int e = tid + 256 * i, u = e / (KT * 64), f = e % (KT * 64);
          if (e >= SP) continue;
          // fragment kk, lane (v, quad): states 32 kk + 4 quad .. + 3 and + 16
          const int at = (16 * u + (f & 15)) * CL + 32 * (f >> 6) + 4 * ((f >> 4) & 3);
          const u32x4_t s0 = __builtin_bit_cast(
              u32x4_t, __builtin_bit_cast(f16x8_t, g_s[i]) * static_cast<_Float16>(1.0f / kBwdStateUp));
          *reinterpret_cast<u32x2_t*>(&lds.s[at]) = u32x2_t{s0[0], s0[1]};
          *reinterpret_cast<u32x2_t*>(&lds.s[at + 16]) = u32x2_t{s0[2], s0[3]};
          *reinterpret_cast<u32x2_t*>(&lds.a[at]) = u32x2_t{g_a[i][0], g_a[i][1]};
          *reinterpret_cast<u32x2_t*>(&lds.a[at + 16]) = u32x2_t{g_a[i][2], g_a[i][3]};
        }
      }
      __syncthreads();
      if (b + 1 < nb) load(b + 1);
      auto yrows = [&](int t) {
        return *reinterpret_cast<const f16x8_t*>(&lds.y[(16 * t + lr) * kGradLd + 8 * lq]);
      };
      const f16x8_t rw = tok_frag<kGradTok>(lds.r, w, lr, lq), yw = yrows(w);
      const f16x8_t vw = tok_frag<kGradTok>(lds.v, w, lr, lq), vwl = tok_frag<kGradTokLo>(lds.vl, w, lr, lq);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        // as pairs where the terms go into dla, one fp16 each in the transposes (for dk)
        if (t <= w) {
          const f16x8_t rt = tok_frag<kGradTok>(lds.r, t, lr, lq), rtl = tok_frag<kGradTokLo>(lds.rl, t, lr, lq);
          a1[t] = mfma_f16(rtl, yw, a1[t]);
          a2[t] = mfma_f16(rtl, vw, a2[t]);
          a1[t] = mfma_f16(rt, yw, a1[t]);
          a2[t] = mfma_f16(rt, vwl, a2[t]);
          a2[t] = mfma_f16(rt, vw, a2[t]);
        } else {
          a1[t] = mfma_f16(yrows(t), rw, a1[t]);
          a2[t] = mfma_f16(tok_frag<kGradTok>(lds.v, t, lr, lq), rw, a2[t]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_sched_barrier(0);
      b1 = mfma_f16(yw, rw, b1);
      b2 = mfma_f16(vw, rw, b2);
      // the rows' gates go into the operands (another rounding to fp16), so the products add to dq and dk themselves
      const f16x8_t yo = yw * static_cast<_Float16>(lds.g[1][16 * w + lr]);
      const f16x8_t vg = vw * static_cast<_Float16>(-lds.g[0][16 * w + lr]);
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const f16x8_t sf = lds_col_frag<DK>(lds.s, 0, d, lr, lq), af = lds_col_frag<DK>(lds.a, 0, d, lr, lq);
        dq[d] = mfma_f16(yo, sf, dq[d]);
        dk[d] = mfma_f16(vg, sf, dk[d]);
        aw[d] = mfma_f16(rw, af, aw[d]);
        if (d & 1) __builtin_amdgcn_sched_barrier(0);  // fragments of all d at once would not fit the registers
      }
    }
    __syncthreads();  // the blocks are read: their place takes the pair terms
    // ---- the chunk's own products.  A lane's elements: before and on this wavefront's tile, (j = 16 t + 4 lq + r,
    // token 16 w + lr); behind it, (token 16 t + 4 lq + r, j = 16 w + lr), and so b1, b2
    const float* left = lds.g[2];
    const float* beta = lds.g[3];
    const int me = 16 * w + lr;
    const float hme = lds.g[4][me], lme = lds.g[5][me];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t <= w) {
        // q_t . k_j and k_t . k_j of the pair terms (the operands are exact)
        f32x4_t qk = zero, kk = zero;
#pragma unroll
        for (int e = 0; e < KT; ++e) {
          const f16x8_t kj = plain_row_frag<CL>(sK, 16 * t + lr, e, lq);
          qk = mfma_f16(kj, plain_row_frag<CL>(sQ, me, e, lq), qk);
          kk = mfma_f16(kj, plain_row_frag<CL>(sK, me, e, lq), kk);
        }
        const f32x4_t bj = *reinterpret_cast<const f32x4_t*>(&beta[16 * t + 4 * lq]);
        const f32x4_t hj = *reinterpret_cast<const f32x4_t*>(&lds.g[4][16 * t + 4 * lq]);
        const f32x4_t lj = *reinterpret_cast<const f32x4_t*>(&lds.g[5][16 * t + 4 * lq]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int o = 16 * t + 4 * lq + r;
          // log of the fade from j = o to this token; past the diagonal (in the own tile) it may be anything
          const float x = ((hme - hj[r]) + (lme - lj[r])) * kLog2e;
          if (t < w) {
            const float f = __builtin_amdgcn_exp2f(x) * bj[r];
            a1[t][r] *= p.scale * f;
            a2[t][r] *= -f;
            lds.c[me * kGradC + o] = a1[t][r] * qk[r] + a2[t][r] * kk[r];
          } else {
            const int rel = 4 * lq + r - lr;
            const float f = rel <= 0 ? __builtin_amdgcn_exp2f(x) * bj[r] : 0.0f;
            const float f2 = rel >= 0 ? __builtin_amdgcn_exp2f(-x) : 0.0f;
            a1[t][r] *= p.scale * f;
            a2[t][r] = rel < 0 ? -f * a2[t][r] : 0.0f;
            lds.c[me * kGradC + o] = rel < 0 ? a1[t][r] * qk[r] + a2[t][r] * kk[r] : 0.0f;
            b1[r] *= p.scale * f2;
            b2[r] = rel > 0 ? -f2 * b2[r] : 0.0f;
          }
        }
      } else {
        const f32x4_t ht = *reinterpret_cast<const f32x4_t*>(&lds.g[4][16 * t + 4 * lq]);
        const f32x4_t lt = *reinterpret_cast<const f32x4_t*>(&lds.g[5][16 * t + 4 * lq]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float f = __builtin_amdgcn_exp2f(((ht[r] - hme) + (lt[r] - lme)) * kLog2e);
          a1[t][r] *= p.scale * f;
          a2[t][r] *= -f;
        }
      }
    }
    __syncthreads();
    {
      // rows less columns of the pair terms, four threads a token
      const int t = tid >> 2, part = tid & 3;
      double e = 0.0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int o = part + 4 * i;
        const float v = lds.c[o < t ? t * kGradC + o : o * kGradC + t];
        e += o < t ? static_cast<double>(v) : (o > t ? -static_cast<double>(v) : 0.0);
      }
      e += __shfl_xor(e, 1, 64);
      e += __shfl_xor(e, 2, 64);
      if (part == 0) lds.e[t] = e;
      lds.og[w][lane] = og;
      lds.l[w][lane] = lt;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) edge += __shfl_xor(edge, o, 64);
      if (lane == 0) lds.edge[w] = edge;
    }
    __syncthreads();
    const f32x4_t leftw = *reinterpret_cast<const f32x4_t*>(&left[16 * w + 4 * lq]);
    const f32x4_t betaw = *reinterpret_cast<const f32x4_t*>(&beta[16 * w + 4 * lq]);
    // operands of the halves m of the tokens: this wavefront's as t with what is before (P, -N), as j with what follows
    f16x8_t pt[2], nt2[2], pj[2], nj[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      auto before = [&](const f32x4_t& v, int t) { return t <= w ? v : zero; };
      auto behind = [&](const f32x4_t& v, const f32x4_t& own, int t) { return t > w ? v : (t == w ? own : zero); };
      pt[m] = pair_f16(before(a1[2 * m], 2 * m), before(a1[2 * m + 1], 2 * m + 1));
      nt2[m] = pair_f16(before(a2[2 * m], 2 * m), before(a2[2 * m + 1], 2 * m + 1));
      pj[m] = pair_f16(behind(a1[2 * m], b1, 2 * m), behind(a1[2 * m + 1], b1, 2 * m + 1));
      nj[m] = pair_f16(behind(a2[2 * m], b2, 2 * m), behind(a2[2 * m + 1], b2, 2 * m + 1));
    }
    float db[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      aw[d] *= leftw;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const f16x8_t kc = lds_col_frag<DK>(sK, 32 * m, d, lr, lq);
        if (2 * m <= w) {  // tokens up to this wavefront's
          dq[d] = mfma_f16(pt[m], kc, dq[d]);
          dk[d] = mfma_f16(nt2[m], kc, dk[d]);
        }
        if (2 * m + 1 >= w) {  // and from it on
          aw[d] = mfma_f16(pj[m], lds_col_frag<DK>(sQ, 32 * m, d, lr, lq), aw[d]);
          aw[d] = mfma_f16(nj[m], kc, aw[d]);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float kv = static_cast<float>(
            __builtin_bit_cast(_Float16, sK[(16 * w + 4 * lq + r) * CL + 16 * d + lr]));
        db[r] = __builtin_fmaf(kv, aw[d][r], db[r]);
      }
      dk[d] += aw[d] * betaw;
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) db[r] += __shfl_xor(db[r], o, 64);
      const int j = 16 * w + 4 * lq + r;
      if (lr == 0 && j < nt) {
        const float b = betaw[r], v = db[r] * inv * (p.sigmoid ? b * (1.0f - b) : 1.0f);
        store_vals<BF16, 1>(bp.dbeta, (tok + j) * p.H + h, &v);
      }
    }
    if (w == 0) {
      // ---- the fades' gradient: sums over the tokens behind each, and over those before it, in fp64
      double la = lds.e[lane] * inv + ((lds.og[0][lane] + lds.og[1][lane]) + (lds.og[2][lane] + lds.og[3][lane]));
      double e = (lds.edge[0] + lds.edge[1]) + (lds.edge[2] + lds.edge[3]);
      lt = (lds.l[0][lane] + lds.l[1][lane]) + (lds.l[2][lane] + lds.l[3][lane]);
      const double own = lt;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double dn = __shfl_down(la, o, 64), up = __shfl_up(lt, o, 64);
        la += lane + o < 64 ? dn : 0.0;
        lt += lane >= o ? up : 0.0;
      }
      e += lt - own;  // the tokens before this one
      float dA = 0.0f, db2 = 0.0f;
      if (lane < nt) {
        const float raw = load_elem<BF16>(p.delta, (tok + lane) * p.H + h) + (p.bias ? p.bias[h] : 0.0f);
        const float l = static_cast<float>(la + e);
        const float ds = l * p.A[h];
        db2 = p.softplus ? ds * sigmoid_f(raw) : ds;
        dA = l * (p.softplus ? softplus_f(raw) : raw);
        store_vals<BF16, 1>(bp.ddelta, (tok + lane) * p.H + h, &db2);
      }
      dA = sum_wave(dA);
      db2 = sum_wave(db2);
      if (lane == 0) {
        bp.part[cell * 2] = dA;
        bp.part[cell * 2 + 1] = db2;
      }
    }
  }
  // dq and dk through LDS, so that they leave in whole 16-byte pieces
  __syncthreads();
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int at = (16 * w + 4 * lq + r) * CL + 16 * d + lr;
      lds.out[0][at] = to_bf16(dq[d][r] * unscale);
      lds.out[1][at] = to_bf16(dk[d][r] * unscale);
    }
  __syncthreads();
  const rsrc_t oq = make_rsrc(static_cast<uint16_t*>(bp.dq) + kb, kbytes);
  const rsrc_t ok = make_rsrc(static_cast<uint16_t*>(bp.dk) + kb, kbytes);
#pragma unroll
  for (int i = 0; i < KPER; ++i) {
    const int e = tid + 256 * i, row = e / (DK / 8), cc = (e % (DK / 8)) * 8;
    const int off = static_cast<int>((row * krow + cc) * 2);
    store_b128(*reinterpret_cast<const u32x4_t*>(&lds.out[0][row * CL + cc]), oq, off);
    store_b128(*reinterpret_cast<const u32x4_t*>(&lds.out[1][row * CL + cc]), ok, off);
  }
}

// dA and dbias of a head: the chunks' parts, summed in a fixed order.
__global__ void __launch_bounds__(256) delta_gate_sum_kernel(const float* part, float* dA, float* dbias, int64_t slots,
                                                             int64_t H) {
  __shared__ double lds[2][256];
  const int64_t h = blockIdx.x;
  double a = 0.0, b = 0.0;
  for (int64_t s = threadIdx.x; s < slots; s += 256) {
    a += part[(s * H + h) * 2];
    b += part[(s * H + h) * 2 + 1];
  }
  lds[0][threadIdx.x] = a;
  lds[1][threadIdx.x] = b;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (static_cast<int>(threadIdx.x) < o) {
      lds[0][threadIdx.x] += lds[0][threadIdx.x + o];
      lds[1][threadIdx.x] += lds[1][threadIdx.x + o];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    dA[h] = static_cast<float>(lds[0][0]);
    if (dbias) dbias[h] = static_cast<float>(lds[1][0]);
  }
}

}  // namespace ssm
