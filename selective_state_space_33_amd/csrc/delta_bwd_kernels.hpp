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
// delta_bwd_walk_kernel<., ., false> walks forward and keeps each chunk's S0 and
// R; <., ., true> walks back, a wavefront holding 16 channels of dS as the
// forward's holds S, writes dV and keeps it and dS; delta_grad_kernel forms dq,
// dk, db and dla of all chunks at once, a workgroup per chunk and key head,
// which sums its heads in order.
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

// The scale of a unit's gradients: it brings their largest magnitude to [16, 32), within what fp32 holds on both
// sides; 1 where there is none, or none that is finite.  (What is summed from them stays thousands of times below the
// largest fp16, and the lo part of a pair, whose last place is 2^-24, keeps its bits down to 2^-3.)
__device__ __forceinline__ float grad_scale(unsigned amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23) - 127;
  if (amax_bits == 0u || e > 127) return 1.0f;
  const int s = e < -96 ? 100 : (e > 104 ? -100 : 4 - e);
  return __uint_as_float(static_cast<unsigned>(s + 127) << 23);
}

constexpr int kSkew = 320;               // bytes of a fragment's 16 lanes in LDS
constexpr int kSkewFrag = 4 * kSkew;     // (four column runs of a transposed read then lie on distinct banks)
constexpr int kBwdLdsImg = 24 * kSkewFrag + 1536;

// The image from registers into LDS, fragments skewed.
template <int NTH, int IPER> __device__ __forceinline__ void stage_bwd_img(char* img, const u32x4_t (&gi)[IPER]) {
#pragma unroll
  for (int i = 0; i < IPER; ++i) {
    const int e = threadIdx.x + NTH * i;
    if (e >= kBwdImgBytes / 16) continue;
    const int f = e >> 6, ln = e & 63;
    const int at = f < 24 ? f * kSkewFrag + (ln >> 4) * kSkew + (ln & 15) * 16 : 24 * kSkewFrag + (e - 24 * 64) * 16;
    *reinterpret_cast<u32x4_t*>(img + at) = gi[i];
  }
}
__device__ __forceinline__ f16x8_t bwd_row_frag(const char* img, int f, int lr, int lq) {
  return *reinterpret_cast<const f16x8_t*>(img + f * kSkewFrag + lq * kSkew + lr * 16);
}
// The transpose's fragment: K index the rows 32 m .. + 31 of the matrix whose fragments start at f0, columns 16 ct + lr.
__device__ __forceinline__ f16x8_t bwd_col_frag(const char* img, int f0, int ct, int m, int lr, int lq) {
  const int at = (lr & 3) * kSkew + (4 * lq + (lr >> 2)) * 16 + (ct & 1) * 8;
  const u32x2_t a = lds_tr4(reinterpret_cast<const uint16_t*>(img + (f0 + frag_of(2 * m, ct >> 1)) * kSkewFrag + at));
  const u32x2_t b =
      lds_tr4(reinterpret_cast<const uint16_t*>(img + (f0 + frag_of(2 * m + 1, ct >> 1)) * kSkewFrag + at));
  return __builtin_bit_cast(f16x8_t, u32x4_t{a[0], a[1], b[0], b[1]});
}
__device__ __forceinline__ f32x4_t bwd_gate(const char* img, int base, int t, int lq) {
  return *reinterpret_cast<const f32x4_t*>(img + 24 * kSkewFrag + (base - kBwdGates) + (16 * t + 4 * lq) * 4);
}
__device__ __forceinline__ float bwd_gate1(const char* img, int base, int t) {
  return *reinterpret_cast<const float*>(img + 24 * kSkewFrag + (base - kBwdGates) + t * 4);
}
// A fragment of rows (paired order) of an array stored plain.
template <int LD> __device__ __forceinline__ f16x8_t plain_row_frag(const uint16_t* base, int r, int kk, int lq) {
  const uint16_t* a = base + r * LD + 32 * kk + 4 * lq;
  const u32x2_t x = *reinterpret_cast<const u32x2_t*>(a), y = *reinterpret_cast<const u32x2_t*>(a + 16);
  return __builtin_bit_cast(f16x8_t, u32x4_t{x[0], x[1], y[0], y[1]});
}

// bf16 values as floats, times a scale.
__device__ __forceinline__ f32x4_t bf16x4_f32(u32x2_t v, float s) {
  return f32x4_t{bf16_lo(v[0]) * s, bf16_hi(v[0]) * s, bf16_lo(v[1]) * s, bf16_hi(v[1]) * s};
}

// Sum over the four lane groups of 16 (lanes lr, 16 + lr, ...), in all of them.
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}
// Sum of each component over the 16 lanes lr of a group, in all of them.
__device__ __forceinline__ f32x4_t sum_lanes16(f32x4_t v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1)
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] += __shfl_xor(v[r], o, 64);
  return v;
}
__device__ __forceinline__ float sum_wave(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Walks forward (BACK false) keeping S0, R and y . dy, or back (BACK true) with the adjoint.  One tile of 16 channels a
// wavefront, W of them a workgroup sharing the chunk in LDS.
template <int DK, int W, bool BACK>
__global__ void __launch_bounds__(64 * W) delta_bwd_walk_kernel(DeltaBwdParams bp) {
  const DeltaChunkParams& p = bp.c;
  constexpr int KT = DK / 32, DT = DK / 16, NTH = 64 * W;
  __shared__ __attribute__((aligned(16))) uint16_t sK[kDeltaC * kColLd<DK>];
  __shared__ __attribute__((aligned(16))) uint16_t sQ[kDeltaC * kColLd<DK>];
  __shared__ __attribute__((aligned(16))) char sImg[kBwdLdsImg];
  __shared__ __attribute__((aligned(16))) uint16_t sT[W][kDeltaC * 16];  // forward: V, back: dY, of each wavefront
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t blocks = (p.P + 16 * W - 1) / (16 * W);
  const int64_t id = xcd_order(blockIdx.x, p.rows * p.H * blocks);
  const int64_t unit = id / blocks, seq = unit / p.H, h = unit % p.H, g = h / (p.H / p.G);
  const int tile = static_cast<int>((id % blocks) * W + w), col = tile * 16;
  const bool mine = col < p.P;
  const DeltaSeq sq = delta_seq(p.cu, seq, p.L, p.chunks);
  const int nchunks = static_cast<int>((sq.len + kDeltaC - 1) / kDeltaC);
  const int64_t rowe = p.H * p.P, krow = p.G * DK;
  const int rowe32 = static_cast<int>(rowe), krow32 = static_cast<int>(krow);
  const int yrow = (lr * rowe32 + 4 * lq) * 2;
  const int ctile = mine ? col * 2 : kPastEnd;
  const float sc = BACK && nchunks > 0 ? grad_scale(p.amax[unit]) : 1.0f, inv = 1.0f / sc;

  // ---- forward: S; back: dS (scaled).  Channel col + lr, states 16 d + 4 lq .. + 3
  f32x4_t S[DT];
  const int64_t sbase = (unit * p.P + col + lr) * DK + 4 * lq;
  const float* first = BACK ? bp.dfinal : p.h0;
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    S[d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (first && mine) S[d] = *reinterpret_cast<const f32x4_t*>(first + sbase + 16 * d);
    if constexpr (BACK) S[d] *= sc;
  }
  float amax = 0.0f;

  constexpr int PIECES = kDeltaC * DK / 8, PER = (PIECES + NTH - 1) / NTH;
  constexpr int IPIECES = kBwdImgBytes / 16, IPER = (IPIECES + NTH - 1) / NTH;
  u32x4_t gk[PER], gq[PER], gi[IPER];
  u32x2_t gv[4], gd[4];
  f16x8_t gs[BACK ? 2 * KT : 1], gr[BACK ? 4 : 1];  // back: the chunk's S0 and R
  auto load = [&](int c) {
    const int64_t c0 = static_cast<int64_t>(c) * kDeltaC, tok = sq.tok + c0;
    const bool some = c >= 0 && c < nchunks;
    const int nt = static_cast<int>(sq.len - c0 < kDeltaC ? sq.len - c0 : kDeltaC);
    const int64_t kb = tok * krow + g * DK, kbytes = some ? ((nt - 1) * krow + DK) * 2 : 0;
    const int64_t vb = tok * rowe + h * p.P, vbytes = some ? ((nt - 1) * rowe + p.P) * 2 : 0;
    const rsrc_t rk = make_rsrc(static_cast<const uint16_t*>(p.k) + kb, kbytes);
    const rsrc_t rq = make_rsrc(static_cast<const uint16_t*>(p.q) + kb, kbytes);
    const rsrc_t ri = make_rsrc(p.img + ((sq.slot + c) * p.H + h) * kBwdImgBytes, some ? kBwdImgBytes : 0);
    const rsrc_t rv = make_rsrc(static_cast<const uint16_t*>(p.v) + vb, vbytes);
    const rsrc_t rd = make_rsrc(static_cast<const uint16_t*>(bp.dy) + vb, vbytes);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + NTH * i;
      const int off = (e / (DK / 8)) * krow32 * 2 + (e % (DK / 8)) * 16;
      gk[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, 0));
      gq[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rq, off, 0, 0));
    }
#pragma unroll
    for (int i = 0; i < IPER; ++i)
      gi[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ri, (tid + NTH * i) * 16, 0, 0));
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      gv[t] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(rv, yrow + ctile, 32 * t * rowe32, 0));
      gd[t] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(rd, yrow + ctile, 32 * t * rowe32, 0));
    }
    if constexpr (BACK) {
      const int64_t at = ((sq.slot + c) * p.H + h) * bp.tiles + tile;
      const rsrc_t rs = make_rsrc(bp.state + at * (2 * KT * kFrag), some && mine ? 2 * KT * kFrag : 0);
      const rsrc_t rr = make_rsrc(bp.r + at * (4 * kFrag), some && mine ? 4 * kFrag : 0);
#pragma unroll
      for (int i = 0; i < 2 * KT; ++i)
        gs[i] = __builtin_bit_cast(f16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rs, lane * 16, i * kFrag, 0));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        gr[i] = __builtin_bit_cast(f16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rr, lane * 16, i * kFrag, 0));
    }
  };

  f16x8_t Sh[KT], Sl[KT];
#pragma unroll
  for (int kk = 0; kk < KT; ++kk) split_f16(S[2 * kk], S[2 * kk + 1], Sh[kk], Sl[kk]);
  load(BACK ? nchunks - 1 : 0);
  for (int i = 0; i < nchunks; ++i) {
    const int c = BACK ? nchunks - 1 - i : i;
    const int64_t c0 = static_cast<int64_t>(c) * kDeltaC, tok = sq.tok + c0;
    const int nt = static_cast<int>(sq.len - c0 < kDeltaC ? sq.len - c0 : kDeltaC);
    const int64_t cell = (sq.slot + c) * p.H + h;  // this chunk's place in the workspace
    __syncthreads();                               // the last chunk's operands are read
#pragma unroll
    for (int e0 = 0; e0 < PER; ++e0) {
      const int e = tid + NTH * e0, row = e / (DK / 8), cc = (e % (DK / 8)) * 8;
      if (PIECES % NTH == 0 || e < PIECES) {
        *reinterpret_cast<u32x4_t*>(&sK[row * kColLd<DK> + cc]) = bf16x8_as_f16(gk[e0]);
        *reinterpret_cast<u32x4_t*>(&sQ[row * kColLd<DK> + cc]) = bf16x8_as_f16(gq[e0]);
      }
    }
    stage_bwd_img<NTH, IPER>(sImg, gi);
#pragma unroll
    for (int t = 0; t < 4; ++t) *reinterpret_cast<u32x2_t*>(&sT[w][(16 * t + lr) * 16 + 4 * lq]) = BACK ? gd[t] : gv[t];
    u32x2_t oth[4];  // forward: dY, channels 4 lq .. + 3 of token 16 t + lr
#pragma unroll
    for (int t = 0; t < 4; ++t) oth[t] = gd[t];
    f16x8_t s0[BACK ? 2 * KT : 1], r0[BACK ? 4 : 1];
    if constexpr (BACK) {
#pragma unroll
      for (int e = 0; e < 2 * KT; ++e) s0[e] = gs[e];
#pragma unroll
      for (int e = 0; e < 4; ++e) r0[e] = gr[e];
    }
    __syncthreads();
    load(BACK ? c - 1 : c + 1);

    u32x2_t tq[4];  // this wavefront's V (dY): tokens 16 t + 4 lq .. + 3 of channel lr
#pragma unroll
    for (int t = 0; t < 4; ++t) tq[t] = lds_tr4(&sT[w][(16 * t + 4 * lq + (lr >> 2)) * 16 + 4 * (lr & 3)]);
    const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const float fade = bwd_gate1(sImg, kBwdGrow, kDeltaC - 1);
    // K times the (adjoint) state, 64 x 16; back, K times S0 beside it
    f32x4_t x[4], z[BACK ? 4 : 1];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      x[t] = zero;
      if constexpr (BACK) z[t] = zero;
#pragma unroll
      for (int kk = 0; kk < KT; ++kk) {
        const f16x8_t kf = plain_row_frag<kColLd<DK>>(sK, 16 * t + lr, kk, lq);
        x[t] = mfma_f16(kf, Sl[kk], x[t]);
        if constexpr (BACK) z[t] = mfma_f16(kf, s0[KT + kk], z[t]);
        x[t] = mfma_f16(kf, Sh[kk], x[t]);
        if constexpr (BACK) z[t] = mfma_f16(kf, s0[kk], z[t]);
      }
    }
    const int64_t mytile = cell * bp.tiles + tile;
    if constexpr (!BACK) {
      char* keep = bp.state + mytile * (2 * KT * kFrag) + lane * 16;
      if (mine) {
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
          *reinterpret_cast<f16x8_t*>(keep + kk * kFrag) = Sh[kk];
          *reinterpret_cast<f16x8_t*>(keep + (KT + kk) * kFrag) = Sl[kk];
        }
      }
      // (S0 q) . dy of each token over these 16 channels, and the largest |dy|
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f32x4_t o = zero;
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
          const f16x8_t qf = plain_row_frag<kColLd<DK>>(sQ, 16 * t + lr, kk, lq);
          o = mfma_f16(Sl[kk], qf, o);
          o = mfma_f16(Sh[kk], qf, o);
        }
        const f32x4_t d = bf16x4_f32(oth[t], 1.0f);
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s = __builtin_fmaf(o[r], d[r], s);
          amax = __builtin_fmaxf(amax, __builtin_fabsf(d[r]));
        }
        s = sum_groups(s) * bwd_gate1(sImg, kBwdOut, 16 * t + lr);
        if (mine && lq == 0) bp.oterm[mytile * kDeltaC + 16 * t + lr] = s;
        const f32x4_t grow = bwd_gate(sImg, kBwdGrow, t, lq), v = bf16x4_f32(tq[t], 1.0f);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[t][r] = __builtin_fmaf(-grow[r], x[t][r], v[r]);
      }
      // R = T X, kept as a pair
      f16x8_t Xh[2], Xl[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) split_f16(x[2 * m], x[2 * m + 1], Xh[m], Xl[m]);
      f32x4_t u[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        u[t] = zero;
#pragma unroll
        for (int m = 0; m <= t / 2; ++m) {
          const f16x8_t th = bwd_row_frag(sImg, frag_of(t, m), lr, lq);
          const f16x8_t tl = bwd_row_frag(sImg, 6 + frag_of(t, m), lr, lq);
          u[t] = mfma_f16(th, Xh[m], u[t]);
          u[t] = mfma_f16(th, Xl[m], u[t]);
          u[t] = mfma_f16(tl, Xh[m], u[t]);
        }
      }
      char* kr = bp.r + mytile * (4 * kFrag) + lane * 16;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        f16x8_t Rh, Rl;
        split_f16(u[2 * m], u[2 * m + 1], Rh, Rl);
        if (mine) {
          *reinterpret_cast<f16x8_t*>(kr + m * kFrag) = Rh;
          *reinterpret_cast<f16x8_t*>(kr + (2 + m) * kFrag) = Rl;
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] *= bwd_gate(sImg, kBwdBeta, t, lq);  // U
      // S = e^{cs_C} S + K^T diag(L) U
#pragma unroll
      for (int d = 0; d < DT; ++d) S[d] *= fade;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        f16x8_t Uh, Ul;
        split_f16(u[2 * m] * bwd_gate(sImg, kBwdLeft, 2 * m, lq), u[2 * m + 1] * bwd_gate(sImg, kBwdLeft, 2 * m + 1, lq),
                  Uh, Ul);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const f16x8_t kc = lds_col_frag<DK>(sK, 32 * m, d, lr, lq);
          S[d] = mfma_f16(kc, Uh, S[d]);
          S[d] = mfma_f16(kc, Ul, S[d]);
        }
      }
    } else {
      char* keep = bp.adj + mytile * (KT * kFrag) + lane * 16;
      if (mine) {
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) *reinterpret_cast<f16x8_t*>(keep + kk * kFrag) = Sh[kk];
      }
      // e^{cs_C} <dS, S0>
      {
        float s = 0.0f;
#pragma unroll
        for (int kk = 0; kk < KT; ++kk)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const f16x8_t hi = s0[kk], lo = s0[KT + kk];
            s = __builtin_fmaf(S[2 * kk][r], static_cast<float>(hi[r]) + static_cast<float>(lo[r]), s);
            s = __builtin_fmaf(S[2 * kk + 1][r], static_cast<float>(hi[4 + r]) + static_cast<float>(lo[4 + r]), s);
          }
        s = sum_wave(s);
        if (lane == 0 && mine) bp.edge[mytile] = s * fade * inv;
      }
      // diag(b) Y0 = diag(b) (diag(L) K dS + P0^T dY); on the way L (K dS) . u of each token
      f32x4_t d[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        d[t] = bf16x4_f32(tq[t], sc);
        x[t] *= bwd_gate(sImg, kBwdLeft, t, lq);
        const f32x4_t beta = bwd_gate(sImg, kBwdBeta, t, lq);
        f32x4_t l;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int e = 4 * (t & 1) + r;
          l[r] = x[t][r] * (static_cast<float>(r0[t >> 1][e]) + static_cast<float>(r0[2 + (t >> 1)][e])) * beta[r];
        }
        x[t] *= kBwdPScale;
        l = sum_lanes16(l);
        if (mine && lr == 0) *reinterpret_cast<f32x4_t*>(&bp.lterm[mytile * kDeltaC + 16 * t + 4 * lq]) = l * inv;
      }
      const f16x8_t Df[2] = {pair_f16(d[0], d[1]), pair_f16(d[2], d[3])};  // exact: bf16 values scaled by a power of 2
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int m = t / 2; m < 2; ++m) {
          x[t] = mfma_f16(bwd_col_frag(sImg, 12, t, m, lr, lq), Df[m], x[t]);
          x[t] = mfma_f16(bwd_col_frag(sImg, 18, t, m, lr, lq), Df[m], x[t]);
        }
        x[t] *= bwd_gate(sImg, kBwdBeta, t, lq) * (1.0f / kBwdPScale);
      }
      // dV = T^T diag(b) Y0, kept as a pair; its transpose (rows of channels, from the hi parts) to store as bf16
      f16x8_t Zh[2], Zl[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) split_f16(x[2 * m], x[2 * m + 1], Zh[m], Zl[m]);
      f32x4_t u[4];
      const rsrc_t ro = make_rsrc(static_cast<uint16_t*>(bp.dv) + tok * rowe + h * p.P, ((nt - 1) * rowe + p.P) * 2);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        u[t] = zero;
        f32x4_t vt = zero;
#pragma unroll
        for (int m = t / 2; m < 2; ++m) {
          const f16x8_t th = bwd_col_frag(sImg, 0, t, m, lr, lq), tl = bwd_col_frag(sImg, 6, t, m, lr, lq);
          u[t] = mfma_f16(th, Zh[m], u[t]);
          u[t] = mfma_f16(th, Zl[m], u[t]);
          u[t] = mfma_f16(tl, Zh[m], u[t]);
          vt = mfma_f16(Zh[m], th, vt);
        }
        vt *= inv;
        __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{pack_bf16x2(vt[0], vt[1]), pack_bf16x2(vt[2], vt[3])}, ro,
                                              yrow + ctile, 32 * t * rowe32, 0);
        // e^cs (S0 k) . dv of each token
        const f32x4_t grow = bwd_gate(sImg, kBwdGrow, t, lq);
        const f32x4_t gt = sum_lanes16(u[t] * z[t] * grow);
        if (mine && lr == 0) *reinterpret_cast<f32x4_t*>(&bp.gterm[mytile * kDeltaC + 16 * t + 4 * lq]) = gt * inv;
      }
      char* kv = bp.dvh + mytile * (4 * kFrag) + lane * 16;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        f16x8_t Vh, Vl;
        split_f16(u[2 * m], u[2 * m + 1], Vh, Vl);
        if (mine) {
          *reinterpret_cast<f16x8_t*>(kv + m * kFrag) = Vh;
          *reinterpret_cast<f16x8_t*>(kv + (2 + m) * kFrag) = Vl;
        }
      }
      // dS = e^{cs_C} dS + Q^T diag(scale e^cs) dY - K^T diag(e^cs) dV
#pragma unroll
      for (int e = 0; e < DT; ++e) S[e] *= fade;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        f16x8_t Gh, Gl, Vh, Vl;
        split_f16(d[2 * m] * bwd_gate(sImg, kBwdOut, 2 * m, lq), d[2 * m + 1] * bwd_gate(sImg, kBwdOut, 2 * m + 1, lq),
                  Gh, Gl);
        split_f16(u[2 * m] * -bwd_gate(sImg, kBwdGrow, 2 * m, lq),
                  u[2 * m + 1] * -bwd_gate(sImg, kBwdGrow, 2 * m + 1, lq), Vh, Vl);
#pragma unroll
        for (int e = 0; e < DT; ++e) {
          const f16x8_t qc = lds_col_frag<DK>(sQ, 32 * m, e, lr, lq), kc = lds_col_frag<DK>(sK, 32 * m, e, lr, lq);
          S[e] = mfma_f16(qc, Gh, S[e]);
          S[e] = mfma_f16(qc, Gl, S[e]);
          S[e] = mfma_f16(kc, Vh, S[e]);
          S[e] = mfma_f16(kc, Vl, S[e]);
        }
      }
    }
#pragma unroll
    for (int kk = 0; kk < KT; ++kk) split_f16(S[2 * kk], S[2 * kk + 1], Sh[kk], Sl[kk]);
  }
  if constexpr (!BACK) {
    // the largest magnitude of the unit's dY and dfinal
    if (nchunks > 0 && mine) {
      if (bp.dfinal) {
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const f32x4_t f = *reinterpret_cast<const f32x4_t*>(bp.dfinal + sbase + 16 * d);
#pragma unroll
          for (int r = 0; r < 4; ++r) amax = __builtin_fmaxf(amax, __builtin_fabsf(f[r]));
        }
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) amax = __builtin_fmaxf(amax, __shfl_xor(amax, o, 64));
      // a maximum does not depend on the order of its arguments, so neither does the scale
      if (lane == 0 && p.amax) atomicMax(p.amax + unit, __float_as_uint(amax));
    }
  } else {
    if (bp.dh0 && mine) {
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4_t*>(bp.dh0 + sbase + 16 * d) = S[d] * inv;
    }
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

template <int DK> __global__ void __launch_bounds__(256, 2) delta_grad_kernel(DeltaBwdParams bp) {
  const DeltaChunkParams& p = bp.c;
  constexpr int KT = DK / 32, DT = DK / 16, CL = kColLd<DK>;
  __shared__ DeltaGradLds<DK> lds;
  uint16_t *const sK = lds.k, *const sQ = lds.q;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t id = xcd_order(blockIdx.x, p.slots * p.G);
  const int64_t slot = id / p.G, g = id % p.G, rep = p.H / p.G;
  int64_t s = 0;
  if (p.cu) {
    int64_t hi = p.rows - 1;
    while (s < hi) {
      const int64_t mid = (s + hi + 1) / 2;
      if (delta_seq(p.cu, mid, p.L, 0).slot <= slot)
        s = mid;
      else
        hi = mid - 1;
    }
  } else {
    s = slot / p.chunks;
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
  u32x4_t g_k[KPER], g_q[KPER];
  {
    const rsrc_t rk = make_rsrc(static_cast<const uint16_t*>(p.k) + kb, kbytes);
    const rsrc_t rq = make_rsrc(static_cast<const uint16_t*>(p.q) + kb, kbytes);
#pragma unroll
    for (int i = 0; i < KPER; ++i) {
      const int e = tid + 256 * i, row = e / (DK / 8), cc = (e % (DK / 8)) * 8;
      const int off = static_cast<int>((row * krow + cc) * 2);
      g_k[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, 0));
      g_q[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rq, off, 0, 0));
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
    const float sc = grad_scale(p.amax[s * p.H + h]), inv = 1.0f / sc;
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
    if (hh == 0) {  // K and Q, loaded ahead of all of this
#pragma unroll
      for (int i = 0; i < KPER; ++i) {
        const int e = tid + 256 * i, row = e / (DK / 8), cc = (e % (DK / 8)) * 8;
        *reinterpret_cast<u32x4_t*>(&sK[row * CL + cc]) = bf16x8_as_f16(g_k[i]);
        *reinterpret_cast<u32x4_t*>(&sQ[row * CL + cc]) = bf16x8_as_f16(g_q[i]);
      }
    }
    // dla's terms of each token (a lane) over every fourth tile
    double og = 0.0, lt = 0.0, edge = 0.0;
    for (int64_t t = w; t < bp.tiles; t += 4) {
      const int64_t at = (cell * bp.tiles + t) * kDeltaC + lane;
      og += static_cast<double>(bp.oterm[at]) - static_cast<double>(bp.gterm[at]);
      lt += bp.lterm[at];
      edge += bp.edge[cell * bp.tiles + t];
    }
    for (int b = 0; b < nb; ++b) {
      __syncthreads();  // the last block (or head) is read
      if (b == 0 && tid < 6 * 16) *reinterpret_cast<f32x4_t*>(&lds.g[0][0] + tid * 4) = g_g;
      {
        const int row = tid >> 2, cc = 8 * (tid & 3);
        u32x4_t y8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f16x2_t hv = __builtin_convertvector((f32x2_t){bf16_lo(g_y[i]) * sc, bf16_hi(g_y[i]) * sc}, f16x2_t);
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
          *reinterpret_cast<u32x2_t*>(&lds.s[at]) = u32x2_t{g_s[i][0], g_s[i][1]};
          *reinterpret_cast<u32x2_t*>(&lds.s[at + 16]) = u32x2_t{g_s[i][2], g_s[i][3]};
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
    __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4_t*>(&lds.out[0][row * CL + cc]), oq, off, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const u32x4_t*>(&lds.out[1][row * CL + cc]), ok, off, 0, 0);
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
