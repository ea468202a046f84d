// delta_prep_kernel.hpp -- the part of the chunked gated delta rule that does
// not depend on the state: per chunk and head T = (I + N diag(b))^-1, P and
// the fades (delta_chunk.hpp), all chunks in parallel.
//
// One workgroup of four wavefronts per (chunk, head).  K of the chunk sits in
// LDS as it comes (bf16, so the products K K^T and K Q^T are exact up to their
// fp32 sums), of Q each wavefront keeps one row tile in registers; it forms a
// row of M tiles and a column of P tiles, five in all, then M takes K's place
// (18 KB a workgroup: six of them share a CU, which hides their serial parts;
// with Q in LDS too, 35 KB and four, it took 115 us where it takes 100: 16384
// tokens of 40 heads, dstate 128, 360 MB).  cs is summed in fp64 and kept
// as a pair of floats: differences of neighbours deep in a fast-fading chunk
// would otherwise lose bits.  The inverse is a forward substitution: the four
// 16 x 16 diagonal blocks at once in one wavefront (a lane a column), then
// block column j in wavefront j, T_ij = -T_ii sum_l M_il T_lj, on fp32 MFMA
// (16x16x4), whose accumulators again serve as the next product's operand.
// T replaces M block by block: T_ii in place, T_ij in the unused block (j, i).
#pragma once

#include "delta_chunk.hpp"
#include "delta_step_kernel.hpp"

namespace ssm {

constexpr int kPrepLd = 68;  // floats per row of the 64 x 64 fp32 arrays (16-byte aligned, banks staggered)

// acc + A B over 16: A rows from LDS (row-major fp32, this lane's row at a), B an accumulator tile.
__device__ __forceinline__ f32x4_t mfma_f32_tile(const float* a, f32x4_t b, f32x4_t acc) {
  const f32x4_t av = *reinterpret_cast<const f32x4_t*>(a);
#pragma unroll
  for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(av[r], b[r], acc, 0, 0, 0);
  return acc;
}

// e^x, the whole part of its exponent to base 2 taken off first (an fp32 argument of 8 is off by 2^-22, and so its power).
__device__ __forceinline__ float exp_f64(double x) {
  const double a = x * 1.4426950408889634, n = __builtin_rint(a);
  return __builtin_ldexpf(__builtin_amdgcn_exp2f(static_cast<float>(a - n)), static_cast<int>(fmin(fmax(n, -1000.0), 1000.0)));
}

// Block column J of T; sM holds M below the diagonal and the T_ii on it.
template <int J> __device__ __forceinline__ void prep_column(float* sM, int lr, int lq) {
  f32x4_t t[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) t[J][r] = sM[(16 * J + 4 * lq + r) * kPrepLd + 16 * J + lr];
#pragma unroll
  for (int i = J + 1; i < 4; ++i) {
    f32x4_t z = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int l = J; l < i; ++l) z = mfma_f32_tile(&sM[(16 * i + lr) * kPrepLd + 16 * l + 4 * lq], t[l], z);
    t[i] = mfma_f32_tile(&sM[(16 * i + lr) * kPrepLd + 16 * i + 4 * lq], z, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      t[i][r] = -t[i][r];
      sM[(16 * J + 4 * lq + r) * kPrepLd + 16 * i + lr] = t[i][r];  // in block (J, i)
    }
  }
}

// BWD: the image of the backward's walks instead (P without b, as a pair; the gates one by one).
template <int DK, bool BWD> __global__ void __launch_bounds__(256) delta_prep_kernel(DeltaChunkParams p) {
  constexpr int IMG = BWD ? kBwdImgBytes : kImgBytes, GATES = BWD ? kBwdGates : kImgGrow;
  constexpr int SB = DK + 8;  // bf16 row stride
  constexpr int ROWS = kDeltaC * SB * 2, MAT = kDeltaC * kPrepLd * 4;  // bytes
  __shared__ __attribute__((aligned(16))) char sMem[ROWS > MAT ? ROWS : MAT];
  uint16_t* const sK = reinterpret_cast<uint16_t*>(sMem);
  float* const sM = reinterpret_cast<float*>(sMem);
  __shared__ __attribute__((aligned(16))) float sChi[kDeltaC], sClo[kDeltaC], sBeta[kDeltaC];
  __shared__ unsigned sTop;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int lr = lane & 15, lq = lane >> 4;
  if (p.words && blockIdx.x == 0 && tid < 4) p.words[tid] = 0u;
  if (tid == 0) sTop = 0u;
  const unsigned heads = static_cast<unsigned>(p.H);
  const unsigned id32 = xcd_order(blockIdx.x, static_cast<unsigned>(p.slots) * heads);
  const int64_t id = id32, slot = id32 / heads, h = id32 % heads, g = key_head(h, p.H, p.G);
  // the sequence of this slot: the last one that starts at or before it
  int64_t s = 0;
  if (p.cu) {
    s = delta_slot_seq(p.cu, p.rows, p.L, slot);
  } else {
    s = static_cast<unsigned>(slot) / static_cast<unsigned>(p.chunks);
  }
  const DeltaSeq sq = delta_seq(p.cu, s, p.L, p.chunks);
  const int64_t c0 = (slot - sq.slot) * kDeltaC;
  if (slot < sq.slot || c0 >= sq.len) return;  // a slot of no chunk (the same for the whole workgroup)
  const int nt = static_cast<int>(sq.len - c0 < kDeltaC ? sq.len - c0 : kDeltaC);
  const int64_t tok = sq.tok + c0;

  // BWD: the first of this thread's pieces of the values (three wavefronts take them): on their way until they are needed
  const int64_t vrow = p.H * p.P;
  const rsrc_t rv = make_rsrc(static_cast<const uint16_t*>(p.v) + tok * vrow + h * p.P, ((nt - 1) * vrow + p.P) * 2);
  const int pieces = static_cast<int>(p.P / 8);
  auto value_piece = [&](int e) {  // (past the 64th row: past the resource)
    const int row = e / pieces;
    const int at = row < kDeltaC ? static_cast<int>((row * vrow + (e - row * pieces) * 8) * 2) : kPastEnd;
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rv, at, 0, 0));
  };
  constexpr int EARLY = 6;
  u32x4_t vv[EARLY];
  // ---- K and Q (rows behind the end are zero) and the gates.  Of Q a wavefront takes one row tile alone.
  const int tt = 3 - w;
  bf16x8_t qf[DK / 32];
  {
    const int64_t rowe = p.G * DK;
    const int64_t base = tok * rowe + g * DK, bytes = ((nt - 1) * rowe + DK) * 2;
    const rsrc_t rk = make_rsrc(static_cast<const uint16_t*>(p.k) + base, bytes);
    const rsrc_t rq = make_rsrc(static_cast<const uint16_t*>(p.q) + base, bytes);
    constexpr int PER = kDeltaC * DK / 8 / 256;
    u32x4_t kv[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + 256 * i, row = e / (DK / 8), col = (e % (DK / 8)) * 8;
      kv[i] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rk, static_cast<int>((row * rowe + col) * 2), 0, 0));
    }
#pragma unroll
    for (int kk = 0; kk < DK / 32; ++kk)
      qf[kk] = __builtin_bit_cast(
          bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(
                        rq, static_cast<int>(((16 * tt + lr) * rowe + 32 * kk + 8 * lq) * 2), 0, 0));
    if constexpr (BWD) {
#pragma unroll
      for (int i = 0; i < EARLY; ++i) vv[i] = value_piece(w > 0 ? tid - 64 + 192 * i : kDeltaC * pieces);
    }
    if (w == 0) {
      const bool live = lane < nt;
      double step = 0.0;
      float b = 0.0f;
      if (live) {
        const float raw = load_elem<BF16>(p.delta, (tok + lane) * p.H + h) + (p.bias ? p.bias[h] : 0.0f);
        // The gradient of A is a sum over all tokens of terms of either sign, and all of them move with the steps: an
        // fp32 softplus that is 7e-8 too large on average shows in it.
        step = !p.softplus ? raw : BWD ? fmax(static_cast<double>(raw), 0.0) + log1p(exp(-fabs(static_cast<double>(raw))))
                                       : softplus_f(raw);
        const float braw = load_elem<BF16>(p.beta, (tok + lane) * p.H + h);
        b = p.sigmoid ? sigmoid_f(braw) : braw;
      }
      double cs = step * static_cast<double>(p.A[h]);
      cs = live ? cs : 0.0;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double up = __shfl_up(cs, o, 64);
        cs += lane >= o ? up : 0.0;
      }
      const double end = __shfl(cs, 63, 64);
      const float chi = static_cast<float>(cs);
      sChi[lane] = chi;
      sClo[lane] = static_cast<float>(cs - static_cast<double>(chi));
      sBeta[lane] = b;
      float* img = reinterpret_cast<float*>(p.img + id * IMG + GATES);
      const float grow = exp_f64(cs);
      img[lane] = grow;
      const float left = exp_f64(end - cs);
      if constexpr (BWD) {
        img[64 + lane] = p.scale * grow;
        img[128 + lane] = left;
        img[192 + lane] = b;
        img[256 + lane] = chi;
        img[320 + lane] = static_cast<float>(cs - static_cast<double>(chi));
        if (c0 == 0 && lane == 0) p.amax[s * p.H + h] = 0u;  // before the walk that takes the maximum
      } else {
        img[64 + lane] = left * b;
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = tid + 256 * i, row = e / (DK / 8), col = (e % (DK / 8)) * 8;
      *reinterpret_cast<u32x4_t*>(&sK[row * SB + col]) = kv[i];
    }
  }
  __syncthreads();

  auto frag = [&](const uint16_t* a, int tile, int kk) {
    return *reinterpret_cast<const bf16x8_t*>(&a[(16 * tile + lr) * SB + 32 * kk + 8 * lq]);
  };
  // e^{cs_t - cs_j}
  auto fade = [&](int t, int j) {
    return __builtin_amdgcn_exp2f(((sChi[t] - sChi[j]) + (sClo[t] - sClo[j])) * kLog2e);
  };
  // ---- M = N diag(b): row tile w, column tiles 0 .. w
  f32x4_t m[4];
#pragma unroll
  for (int jt = 0; jt < 4; ++jt) {
    m[jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (jt > w) continue;
#pragma unroll
    for (int kk = 0; kk < DK / 32; ++kk)
      m[jt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(sK, w, kk), frag(sK, jt, kk), m[jt], 0, 0, 0);
    const int j = 16 * jt + lr;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * lq + r;
      // An entry that is not finite stays out of the inverse, where it would reach the rows before its own: the state
      // and y of its token and all behind it take it from K, P or the fades.
      const float v = sBeta[j] * fade(t, j) * m[jt][r];
      m[jt][r] = j < t && __builtin_fabsf(v) <= 3.4e38f ? v : 0.0f;
    }
  }
  // ---- P of token tile tt.  Backward: P^T, from tiles of Q K^T, which leave four consecutive t of token j = lr in a lane,
  // half a fragment; the half above the diagonal's tile is zero
  if constexpr (BWD) {
    auto put = [&](int jt, f32x4_t v) {
      f16x8_t hi, lo;
      split_f16(v, v, hi, lo);
      char* out = p.img + id * IMG + kBwdBack + (12 + back_frag(jt, tt / 2)) * kFrag + lane * 16 + (tt & 1) * 8;
      *reinterpret_cast<f16x4_t*>(out) = __builtin_shufflevector(hi, hi, 0, 1, 2, 3);
      *reinterpret_cast<f16x4_t*>(out + 6 * kFrag) = __builtin_shufflevector(lo, lo, 0, 1, 2, 3);
    };
    for (int jt = 0; jt <= tt; ++jt) {
      f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kk = 0; kk < DK / 32; ++kk)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[kk], frag(sK, jt, kk), acc, 0, 0, 0);
      const int j = 16 * jt + lr;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 16 * tt + 4 * lq + r;
        acc[r] = j <= t ? p.scale * kBwdPScale * fade(t, j) * acc[r] : 0.0f;
      }
      put(jt, acc);
    }
    if (!(tt & 1)) put(tt + 1, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
  } else {
    // the tiles of K Q^T leave four consecutive j of token t = lr in a lane, half a fragment
    const int t = 16 * tt + lr;
    for (int m2 = 0; m2 <= tt / 2; ++m2) {
      f32x4_t half[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int jt = 2 * m2 + u;
        f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
        if (jt <= tt) {
#pragma unroll
          for (int kk = 0; kk < DK / 32; ++kk)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(sK, jt, kk), qf[kk], acc, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 16 * jt + 4 * lq + r;
            acc[r] = j <= t ? sBeta[j] * fade(t, j) * acc[r] : 0.0f;
          }
        }
        half[u] = acc;
      }
      // fp16: P meets R (fp16 too) in y alone, which is stored with 8 significant bits
      *reinterpret_cast<f16x8_t*>(p.img + id * IMG + kImgP + frag_of(tt, m2) * kFrag + lane * 16) =
          pair_f16(half[0], half[1]);
    }
  }
  __syncthreads();  // K is read
#pragma unroll
  for (int jt = 0; jt < 4; ++jt)
    if (jt <= w) {
#pragma unroll
      for (int r = 0; r < 4; ++r) sM[(16 * w + 4 * lq + r) * kPrepLd + 16 * jt + lr] = m[jt][r];
    }
  __syncthreads();
  if (w == 0) {
    // ---- the diagonal blocks' inverses: lane (block, column c) solves (I + M_bb) x = e_c
    const int b0 = 16 * lq, c = lr;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float acc0 = i == c ? 1.0f : 0.0f, acc1 = 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) {
        const float mv = sM[(b0 + i) * kPrepLd + b0 + j];
        if (j & 1)
          acc1 = __builtin_fmaf(-mv, x[j], acc1);
        else
          acc0 = __builtin_fmaf(-mv, x[j], acc0);
      }
      x[i] = acc0 + acc1;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) sM[(b0 + i) * kPrepLd + b0 + c] = x[i];
  } else if constexpr (BWD) {
    // ---- meanwhile the largest value (magnitudes order as their bits do)
    unsigned top = 0u;
    auto take = [&](u32x4_t x) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top = max(top, (x[i] << 16) & 0x7fff0000u);
        top = max(top, x[i] & 0x7fff0000u);
      }
    };
#pragma unroll
    for (int i = 0; i < EARLY; ++i) take(vv[i]);
    for (int e = tid - 64 + 192 * EARLY; e < kDeltaC * pieces; e += 192) take(value_piece(e));
    if (p.h0 && c0 == 0) {
      const u32x4_t* s0 = reinterpret_cast<const u32x4_t*>(p.h0 + (s * p.H + h) * p.P * DK);
      for (int64_t e = tid - 64; e < p.P * DK / 4; e += 192) {
        const u32x4_t x = s0[e];
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, x[i] & 0x7fffffffu);
      }
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = max(top, static_cast<unsigned>(__shfl_xor(static_cast<int>(top), o, 64)));
    if (lane == 0) atomicMax(&sTop, top);
  }
  __syncthreads();
  if (w == 0)
    prep_column<0>(sM, lr, lq);
  else if (w == 1)
    prep_column<1>(sM, lr, lq);
  else if (w == 2)
    prep_column<2>(sM, lr, lq);
  __syncthreads();
  if (BWD && tid == 0) p.vmax[id] = sTop;
  // ---- T as fragments, hi + lo
  for (int e = tid; e < 6 * 64; e += 256) {
    const int f = e >> 6, ln = e & 63, row = ln & 15, q4 = 4 * (ln >> 4);
    const int t = f < 2 ? f : 2 + ((f - 2) >> 1), m = f < 2 ? 0 : (f & 1);
    // block (t, j) of T sits at (t, t), or at (j, t) for j < t
    auto block = [&](int j) {
      return *reinterpret_cast<const f32x4_t*>(&sM[(16 * (j < t ? j : t) + row) * kPrepLd + 16 * t + q4]);
    };
    const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const f32x4_t x0 = block(2 * m), x1 = 2 * m + 1 <= t ? block(2 * m + 1) : zero;
    constexpr float up = BWD ? kBwdTUp : 1.0f;
    f16x8_t hi, lo;
    split_f16(x0 * up, x1 * up, hi, lo);
    char* out = p.img + id * IMG + f * kFrag + ln * 16;
    *reinterpret_cast<f16x8_t*>(out + kImgThi) = hi;
    *reinterpret_cast<f16x8_t*>(out + kImgTlo) = lo;
  }
  if constexpr (BWD) {
    // ---- and its transpose's: token j = 16 (row tile) + row, four consecutive t twice
    for (int e = tid; e < 6 * 64; e += 256) {
      const int f = e >> 6, ln = e & 63, row = ln & 15, q4 = 4 * (ln >> 4);
      const int j = f < 4 ? f : f - 4, m = f < 4 ? 1 : 0;
      f32x4_t half[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = 2 * m + u;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          half[u][r] = t < j ? 0.0f : sM[(16 * j + q4 + r) * kPrepLd + 16 * t + row] * kBwdTUp;
      }
      f16x8_t hi, lo;
      split_f16(half[0], half[1], hi, lo);
      char* out = p.img + id * IMG + kBwdBack + f * kFrag + ln * 16;
      *reinterpret_cast<f16x8_t*>(out) = hi;
      *reinterpret_cast<f16x8_t*>(out + 6 * kFrag) = lo;
    }
  }
}

}  // namespace ssm
