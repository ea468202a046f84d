// delta_walk_kernel.hpp -- the chunked gated delta rule's walk over a
// sequence (delta_chunk.hpp has the mathematics and the operand order).
//
// A wavefront owns NC tiles of 16 value channels with their whole state
// (dstate x 16 NC, fp32 accumulators) and takes a chunk from S0 to S_C without
// exchanging anything with its neighbours; the W wavefronts of a workgroup
// share the chunk's K, Q, T, P and fades in LDS, double-buffered, so a chunk
// costs one barrier.  Per chunk and tile (dstate 128) 104 MFMAs 16x16x32:
// K S0 32 (S0 as fp16 hi + lo), T X 18 (both as pairs, without lo x lo),
// K^T U 32, Q S0 16 and P U 6 (one product each: y is stored with 8 bits).
//
// Precision.  K and Q convert to fp16 exactly.  Everything on the way from
// state to state is a pair of fp16 (22 bits) with fp32 accumulation.
#pragma once

#include "delta_chunk.hpp"

namespace ssm {

template <int DK, int W, int NC> struct DeltaWalkLds {
  // K twice: by rows for K S0 (paired order, 16-byte fragment reads: a row
  // stride of 4 x odd dwords), and plain for the transposed reads of K^T U
  // (8 x odd dwords: eight rows of a read touch all banks once).
  static constexpr int SP = DK + 8, ST = DK + 16;
  __attribute__((aligned(16))) uint16_t k[kDeltaC * SP];
  __attribute__((aligned(16))) uint16_t kt[kDeltaC * ST];
  __attribute__((aligned(16))) uint16_t q[kDeltaC * SP];
  __attribute__((aligned(16))) char img[kImgBytes];
};

template <int DK, int W, int NC>
__global__ void __launch_bounds__(64 * W) delta_walk_kernel(DeltaChunkParams p) {
  constexpr int KT = DK / 32, DT = DK / 16, NTH = 64 * W;
  using Lds = DeltaWalkLds<DK, W, NC>;
  constexpr int SP = Lds::SP, ST = Lds::ST;
  __shared__ Lds lds[2];
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t blocks = (p.P + 16 * NC * W - 1) / (16 * NC * W);  // workgroups per unit
  const int64_t id = xcd_order(blockIdx.x, p.rows * p.H * blocks);
  const int64_t unit = id / blocks, seq = unit / p.H, h = unit % p.H, g = h / (p.H / p.G);
  const int col = static_cast<int>((id % blocks) * W + w) * 16 * NC;  // first channel of this wavefront
  const DeltaSeq sq = delta_seq(p.cu, seq, p.L, p.chunks);
  const int nchunks = static_cast<int>((sq.len + kDeltaC - 1) / kDeltaC);
  const int64_t rowe = p.H * p.P, krow = p.G * DK;

  // ---- the state: channel col + 16 n + lr, states 16 d + 4 lq .. + 3
  f32x4_t S[NC][DT];
  const int64_t sbase = (unit * p.P + col + lr) * DK + 4 * lq;
#pragma unroll
  for (int n = 0; n < NC; ++n)
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      S[n][d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      if (p.h0 && col + 16 * n < p.P)
        S[n][d] = *reinterpret_cast<const f32x4_t*>(p.h0 + sbase + 16 * n * DK + 16 * d);
    }

  // ---- chunk loads, one chunk ahead in registers
  constexpr int PER = kDeltaC * DK / 8 / NTH;
  constexpr int IPER = (kImgBytes / 16 + NTH - 1) / NTH;
  u32x4_t gk[PER], gq[PER], gi[IPER];
  uint16_t gv[NC][4][4];
  auto load = [&](int c) {
    const int64_t c0 = static_cast<int64_t>(c) * kDeltaC, tok = sq.tok + c0;
    const int nt = static_cast<int>(sq.len - c0 < kDeltaC ? sq.len - c0 : kDeltaC);
    const int64_t kb = tok * krow + g * DK, kbytes = ((nt - 1) * krow + DK) * 2;
    const rsrc_t rk = make_rsrc(static_cast<const uint16_t*>(p.k) + kb, kbytes);
    const rsrc_t rq = make_rsrc(static_cast<const uint16_t*>(p.q) + kb, kbytes);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + NTH * i, row = e / (DK / 8), cc = (e % (DK / 8)) * 8;
      const int off = static_cast<int>((row * krow + cc) * 2);
      gk[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rk, off, 0, 0));
      gq[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rq, off, 0, 0));
    }
    const u32x4_t* im = reinterpret_cast<const u32x4_t*>(p.img + ((sq.slot + c) * p.H + h) * kImgBytes);
#pragma unroll
    for (int i = 0; i < IPER; ++i) {
      const int e = tid + NTH * i;
      if (e < kImgBytes / 16) gi[i] = im[e];
    }
    // rows behind the sequence's end read as zero
    const rsrc_t rv = make_rsrc(static_cast<const uint16_t*>(p.v) + tok * rowe + h * p.P, ((nt - 1) * rowe + p.P) * 2);
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          gv[n][t][r] = 0;
          if (col + 16 * n < p.P)
            gv[n][t][r] = __builtin_amdgcn_raw_buffer_load_b16(
                rv, static_cast<int>(((16 * t + 4 * lq + r) * rowe + col + 16 * n + lr) * 2), 0, 0);
        }
  };
  auto stage = [&](Lds& b) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + NTH * i, row = e / (DK / 8), cc = (e % (DK / 8)) * 8;
      const u32x4_t k8 = bf16x8_as_f16(gk[i]), q8 = bf16x8_as_f16(gq[i]);
      const int j = (cc >> 2) & 7, blk = cc & ~31;  // this piece's runs j, j + 1 of its 32-element block
      uint16_t* kp = &b.k[row * SP + blk];
      uint16_t* qp = &b.q[row * SP + blk];
      *reinterpret_cast<u32x2_t*>(kp + 4 * paired_run(j)) = u32x2_t{k8[0], k8[1]};
      *reinterpret_cast<u32x2_t*>(kp + 4 * paired_run(j + 1)) = u32x2_t{k8[2], k8[3]};
      *reinterpret_cast<u32x2_t*>(qp + 4 * paired_run(j)) = u32x2_t{q8[0], q8[1]};
      *reinterpret_cast<u32x2_t*>(qp + 4 * paired_run(j + 1)) = u32x2_t{q8[2], q8[3]};
      *reinterpret_cast<u32x4_t*>(&b.kt[row * ST + cc]) = k8;
    }
#pragma unroll
    for (int i = 0; i < IPER; ++i) {
      const int e = tid + NTH * i;
      if (e < kImgBytes / 16) *reinterpret_cast<u32x4_t*>(&b.img[e * 16]) = gi[i];
    }
  };

  if (nchunks > 0) {
    load(0);
    stage(lds[0]);
  }
  __syncthreads();
  for (int c = 0; c < nchunks; ++c) {
    const Lds& b = lds[c & 1];
    const int64_t c0 = static_cast<int64_t>(c) * kDeltaC, tok = sq.tok + c0;
    const int nt = static_cast<int>(sq.len - c0 < kDeltaC ? sq.len - c0 : kDeltaC);
    float v[NC][4][4];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[n][t][r] = __uint_as_float(static_cast<uint32_t>(gv[n][t][r]) << 16);
    if (c + 1 < nchunks) load(c + 1);

    auto row_frag = [&](const uint16_t* a, int t, int kk) {
      return *reinterpret_cast<const f16x8_t*>(&a[(16 * t + lr) * SP + 32 * kk + 8 * lq]);
    };
    auto img_frag = [&](int base, int f) {
      return *reinterpret_cast<const f16x8_t*>(&b.img[base + f * kFrag + lane * 16]);
    };
    auto img_vec = [&](int base, int t) {  // four tokens 16 t + 4 lq .. + 3
      return *reinterpret_cast<const f32x4_t*>(&b.img[base + (16 * t + 4 * lq) * 4]);
    };
    const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    f16x8_t Sh[NC][KT], Sl[NC][KT];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int kk = 0; kk < KT; ++kk) split_f16(S[n][2 * kk], S[n][2 * kk + 1], Sh[n][kk], Sl[n][kk]);

    // ---- X = diag(b) (V - diag(e^cs) K S0), and Q S0 (as its transpose) beside it
    f32x4_t x[NC][4], o[NC][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int n = 0; n < NC; ++n) x[n][t] = o[n][t] = zero;
#pragma unroll
      for (int kk = 0; kk < KT; ++kk) {
        const f16x8_t kf = row_frag(b.k, t, kk), qf = row_frag(b.q, t, kk);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          x[n][t] = mfma_f16(kf, Sh[n][kk], x[n][t]);
          x[n][t] = mfma_f16(kf, Sl[n][kk], x[n][t]);
          o[n][t] = mfma_f16(Sh[n][kk], qf, o[n][t]);
        }
      }
      const f32x4_t grow = img_vec(kImgGrow, t), beta = img_vec(kImgBeta, t);
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[n][t][r] = beta[r] * __builtin_fmaf(-grow[r], x[n][t][r], v[n][t][r]);
    }
    // ---- U = T X
    f32x4_t u[NC][4];
    {
      f16x8_t Xh[NC][2], Xl[NC][2];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m) split_f16(x[n][2 * m], x[n][2 * m + 1], Xh[n][m], Xl[n][m]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int n = 0; n < NC; ++n) u[n][t] = zero;
#pragma unroll
        for (int m = 0; m <= t / 2; ++m) {
          const f16x8_t th = img_frag(kImgThi, frag_of(t, m)), tl = img_frag(kImgTlo, frag_of(t, m));
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            u[n][t] = mfma_f16(th, Xh[n][m], u[n][t]);
            u[n][t] = mfma_f16(th, Xl[n][m], u[n][t]);
            u[n][t] = mfma_f16(tl, Xh[n][m], u[n][t]);
          }
        }
      }
    }
    // ---- S = e^{cs_C} S + K^T diag(e^{cs_C - cs}) U
    {
      const float fade = *reinterpret_cast<const float*>(&b.img[kImgGrow + (kDeltaC - 1) * 4]);
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int d = 0; d < DT; ++d) S[n][d] *= fade;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        f16x8_t Uh[NC], Ul[NC];
        const f32x4_t l0 = img_vec(kImgLeft, 2 * m), l1 = img_vec(kImgLeft, 2 * m + 1);
#pragma unroll
        for (int n = 0; n < NC; ++n) split_f16(u[n][2 * m] * l0, u[n][2 * m + 1] * l1, Uh[n], Ul[n]);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const f16x8_t kf = lds_col_frag(b.kt, 32 * m, 16 * d, ST, lr, lq);
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            S[n][d] = mfma_f16(kf, Uh[n], S[n][d]);
            S[n][d] = mfma_f16(kf, Ul[n], S[n][d]);
          }
        }
      }
    }
    // ---- Y^T = scale (e^cs (Q S0)^T + U^T P^T): four consecutive channels of token 16 t + lr in a lane
    {
      f16x8_t Uf[NC][2];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m) Uf[n][m] = pair_f16(u[n][2 * m], u[n][2 * m + 1]);
      const rsrc_t ry = make_rsrc(static_cast<uint16_t*>(p.y) + tok * rowe + h * p.P, ((nt - 1) * rowe + p.P) * 2);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float grow = *reinterpret_cast<const float*>(&b.img[kImgGrow + (16 * t + lr) * 4]);
#pragma unroll
        for (int n = 0; n < NC; ++n) o[n][t] *= grow;
#pragma unroll
        for (int m = 0; m <= t / 2; ++m) {
          const f16x8_t pf = img_frag(kImgP, frag_of(t, m));
#pragma unroll
          for (int n = 0; n < NC; ++n) o[n][t] = mfma_f16(Uf[n][m], pf, o[n][t]);
        }
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          o[n][t] *= p.scale;
          if (col + 16 * n < p.P)
            __builtin_amdgcn_raw_buffer_store_b64(
                u32x2_t{pack_bf16x2(o[n][t][0], o[n][t][1]), pack_bf16x2(o[n][t][2], o[n][t][3])}, ry,
                static_cast<int>(((16 * t + lr) * rowe + col + 16 * n + 4 * lq) * 2), 0, 0);
        }
      }
    }
    if (c + 1 < nchunks) stage(lds[(c + 1) & 1]);
    __syncthreads();
  }
  if (p.hT) {
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int d = 0; d < DT; ++d)
        if (col + 16 * n < p.P) *reinterpret_cast<f32x4_t*>(p.hT + sbase + 16 * n * DK + 16 * d) = S[n][d];
  }
}

}  // namespace ssm
