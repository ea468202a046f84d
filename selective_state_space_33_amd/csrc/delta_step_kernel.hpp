// delta_step_kernel.hpp -- the gated delta rule token by token.
//
// Per batch row (or packed sequence) and head, with the state S (headdim x
// dstate, fp32), one token is
//     a = exp(step A),  r = v - a S k,  S <- a S + (b r) k^T,  y = scale S q.
// The rows of S (one per value channel) never meet, so a row is all that has
// to stay together: eight lanes hold it, DK / 8 states each, for as many
// tokens as there are.  The two products S k and S q both read the state
// before the update (S_new q = a (S q) + b r (k . q)), so one pass over the
// registers serves both, and their sums over the eight lanes are three DPP
// adds each.
//
// What bounds it: for one token (decode) the state, read and written once:
// every lane loads RPT rows (4 RPT 16-byte loads at dstate 128, all issued
// before the first use), eight lanes a 128-byte line; 256 rows of 40 heads of
// 128 channels, dstate 128 (1.35 GB): 243 us, 5.5 TB/s.  Over several tokens
// the chain through S: ~4 DK/8 FMAs and 6 DPP adds a token.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace ssm {

struct DeltaStepParams {
  const void* q;        // [batch][L][G][N]
  const void* k;        // [batch][L][G][N]
  const void* v;        // [batch][L][H][P]
  const void* delta;    // [batch][L][H] (raw)
  const float* A;       // [H]
  const void* beta;     // [batch][L][H] (raw with sigmoid)
  const float* bias;    // [H] (nullable)
  const float* h0;      // [rows][H][P][N] (nullable: zero); may be hT
  float* hT;            // [rows][H][P][N] (nullable)
  const int64_t* cu;    // [nseq + 1] token offsets of batch row 0 (nullable)
  void* y;              // [batch][L][H][P]
  int64_t L, H, G, P;
  int64_t row_blocks;   // workgroups per (row, head) unit
  int softplus, sigmoid;
  float scale;
};

// Sum over the eight lanes of an aligned group, in all of them.  After the two
// quad steps the four lanes of a quad agree, so the mirrored half row holds the
// other quad's sum.
__device__ __forceinline__ float sum8(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xB1, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4E, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x141, 0xf, 0xf, true));
  return v;
}

// 1 / (1 + e^-x); e^-x = inf for very negative x gives 0.
__device__ __forceinline__ float sigmoid_f(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

constexpr int kDeltaStepWaves = 4;

// RPT: rows of the state per lane group (a wavefront holds 8 RPT rows).
template <class IO, int DK, int RPT>
__global__ void __launch_bounds__(64 * kDeltaStepWaves) delta_step_kernel(DeltaStepParams p) {
  constexpr int NC = DK / 32;  // 4-state pieces of a lane: states 32 c + 4 l .. + 3
  const int tid = threadIdx.x, l8 = tid & 7;
  // (the host keeps the counts in 32 bits)
  const unsigned nb = static_cast<unsigned>(p.row_blocks), heads = static_cast<unsigned>(p.H);
  const unsigned unit = blockIdx.x / nb;
  const int64_t seq = unit / heads, h = unit % heads;
  const int64_t g = static_cast<unsigned>(h) / (heads / static_cast<unsigned>(p.G));
  const int64_t row0 = static_cast<int64_t>(blockIdx.x % nb) * (kDeltaStepWaves * 8 * RPT) + (tid >> 6) * (8 * RPT) +
                       ((tid & 63) >> 3);
  int64_t t0 = seq * p.L, t1 = t0 + p.L;
  if (p.cu) {
    const int64_t a = p.cu[seq], b = p.cu[seq + 1];
    t0 = a < 0 ? 0 : (a > p.L ? p.L : a);
    t1 = b < t0 ? t0 : (b > p.L ? p.L : b);
  }
  const float Ah = p.A[h], bias = p.bias ? p.bias[h] : 0.0f;

  float S[RPT][NC][4];
  const int64_t sbase = (seq * p.H + h) * p.P;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t row = row0 + 8 * i;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p.h0 && row < p.P) s = *reinterpret_cast<const float4*>(p.h0 + (sbase + row) * DK + 32 * c + 4 * l8);
      S[i][c][0] = s.x, S[i][c][1] = s.y, S[i][c][2] = s.z, S[i][c][3] = s.w;
    }
  }

  for (int64_t t = t0; t < t1; ++t) {
    float kv[NC][4], qv[NC][4], vv[RPT];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t at = (t * p.G + g) * DK + 32 * c + 4 * l8;
      unpack<IO, 4>(raw_load<IO, 4>(p.k, at), kv[c]);
      unpack<IO, 4>(raw_load<IO, 4>(p.q, at), qv[c]);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i)
      vv[i] = row0 + 8 * i < p.P ? load_elem<IO>(p.v, (t * p.H + h) * p.P + row0 + 8 * i) : 0.0f;
    const float raw = load_elem<IO>(p.delta, t * p.H + h) + bias;
    const float braw = load_elem<IO>(p.beta, t * p.H + h);
    const float a = __builtin_amdgcn_exp2f((p.softplus ? softplus_f(raw) : raw) * Ah * kLog2e);
    const float b = p.sigmoid ? sigmoid_f(braw) : braw;
    float kq = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) kq = __builtin_fmaf(kv[c][j], qv[c][j], kq);
    kq = sum8(kq);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      float sk = 0.0f, sq = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sk = __builtin_fmaf(S[i][c][j], kv[c][j], sk);
          sq = __builtin_fmaf(S[i][c][j], qv[c][j], sq);
        }
      sk = sum8(sk);
      sq = sum8(sq);
      const float u = b * __builtin_fmaf(-a, sk, vv[i]);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][c][j] = __builtin_fmaf(u, kv[c][j], a * S[i][c][j]);
      if (l8 == 0 && row0 + 8 * i < p.P) {
        const float out = p.scale * __builtin_fmaf(a, sq, u * kq);
        store_vals<IO, 1>(p.y, (t * p.H + h) * p.P + row0 + 8 * i, &out);
      }
    }
  }
  if (p.hT) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int64_t row = row0 + 8 * i;
      if (row < p.P) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
          *reinterpret_cast<float4*>(p.hT + (sbase + row) * DK + 32 * c + 4 * l8) =
              make_float4(S[i][c][0], S[i][c][1], S[i][c][2], S[i][c][3]);
      }
    }
  }
}

}  // namespace ssm
