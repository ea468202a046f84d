// norm_kernels.hpp -- the RMS norms around a state-space layer, each in one
// pass over its rows, forward and backward.
//
// Behind the layer (the norm's groups are heads, or the whole row):
//   gate_first = 0:  y = w n SiLU(z),  n = x rstd(x)
//   gate_first = 1:  y = w n,          n = t rstd(t),  t = x SiLU(z)
// In front of the next block, with the residual stream:
//   a = post_w x rstd(x)  (or x),   r' = r + scale a,   y = w r' rstd(r')
// with rstd(t) = 1 / sqrt(mean of t^2 over the group + eps).  The gradient of
// an RMS norm n = t rstd with m reaching it is rstd (m - n mean(m n)), and
// mean(m n) = rstd mean(m t): one sum beside that of t^2, so a backward needs
// a single reduction of two values (the residual one, with a norm behind the
// block, a second, since that norm's gradient starts from the first's).
//
// Layout.  A team of T threads (a power of two up to 256) holds one group:
// NV vectors of VW consecutive elements each (16 bytes of the narrower
// tensor), at places (t + T j) VW, all in registers from the load to the
// store.  A workgroup serves one column group and walks the rows with all its
// teams, so the weights are loaded once and the weight gradients stay in
// registers until the end; their sums over rows are then formed in a fixed
// order: rows of a team in order, the teams of a workgroup through LDS in
// order, the workgroups by norm_reduce_kernel in order.  All statistics,
// sums and products are fp32; outputs are rounded once, to nearest even.
//
// What bounds them: HBM.  A row costs its loads and stores plus ~10 VALU
// instructions an element (the sigmoid's exp and rcp among them).  A large
// copy moves 4.9 TB/s here; the gated norm over 16384 x 5120 in heads of 128
// 4.5 (111 us), its backward over 16384 x 1536 4.7 and 5 us for the weight's
// sums (53), the residual norm's backward over 12289 x 2560 with a norm behind
// the block 3.9 and 5 (145: 24 elements of four tensors and three sums a
// thread leave a CU two workgroups).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.hpp"

namespace ssm {

constexpr int kNormThreads = 256;

// VW consecutive elements from idx, widened to fp32 (16-byte pieces where VW allows).
template <class IO, int VW> __device__ __forceinline__ void vec_load(const void* base, int64_t idx, float* o) {
  if constexpr (VW == 8 && sizeof(Raw<IO, 1>) == 2) {
    const u32x4_t r = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(base) + idx);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[2 * i] = bf16_lo(r[i]), o[2 * i + 1] = bf16_hi(r[i]);
  } else if constexpr (VW == 8) {
    unpack<IO, 4>(raw_load<IO, 4>(base, idx), o);
    unpack<IO, 4>(raw_load<IO, 4>(base, idx + 4), o + 4);
  } else {
    unpack<IO, VW>(raw_load<IO, VW>(base, idx), o);
  }
}
// The same kept as it is in memory until get(): half the registers of a bf16 vector.
template <class IO, int VW> struct Held {
  Raw<IO, VW> v;
  __device__ __forceinline__ void clear() { v = Raw<IO, VW>{}; }
  __device__ __forceinline__ void load(const void* base, int64_t idx) { v = raw_load<IO, VW>(base, idx); }
  __device__ __forceinline__ void get(float* o) const { unpack<IO, VW>(v, o); }
  __device__ __forceinline__ void again() {}
};
template <> struct Held<BF16, 8> {
  u32x4_t v;
  __device__ __forceinline__ void clear() { v = u32x4_t{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void load(const void* base, int64_t idx) {
    v = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(base) + idx);
  }
  __device__ __forceinline__ void get(float* o) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[2 * i] = bf16_lo(v[i]), o[2 * i + 1] = bf16_hi(v[i]);
  }
  // before a second get(): keeps the compiler from holding the first one's values instead
  __device__ __forceinline__ void again() { asm("" : "+v"(v)); }
};
template <class IO, int VW> __device__ __forceinline__ void vec_store(void* base, int64_t idx, const float* v) {
  if constexpr (VW == 8 && sizeof(Raw<IO, 1>) == 2) {
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(base) + idx) = u32x4_t{
        pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  } else if constexpr (VW == 8) {
    store_vals<IO, 4>(base, idx, v);
    store_vals<IO, 4>(base, idx + 4, v + 4);
  } else {
    store_vals<IO, VW>(base, idx, v);
  }
}

// Sums K values over a team of T threads (T a power of two); every thread of
// the workgroup takes part.  Teams wider than a wavefront go through LDS, in
// alternating halves (`par`), so one barrier a sum is enough.
template <int K> __device__ __forceinline__ void team_sum(float (&v)[K], int T, float (*red)[4][2], int& par) {
  for (int o = 1; o < T && o < 64; o <<= 1) {
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += __shfl_xor(v[i], o, 64);
  }
  if (T > 64) {
    const int w = threadIdx.x >> 6, nw = T >> 6, w0 = w & ~(nw - 1);
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < K; ++i) red[par][w][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      v[i] = red[par][w0][i];
      for (int j = 1; j < nw; ++j) v[i] += red[par][w0 + j][i];
    }
    par ^= 1;
  }
}

// SiLU(z) and its derivative s (1 + z (1 - s)).
__device__ __forceinline__ void silu_parts(float z, float& f, float& d) {
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
  f = z * s;
  d = s * __builtin_fmaf(z, 1.0f - s, 1.0f);
}

// A team's place in the work: the column group, its rows, its elements.
struct NormSplit {
  int64_t rows, dim;
  int group, ngroups;  // dim = group * ngroups
  int T, teams;        // threads per team, teams per workgroup
  int slots;           // workgroups per column group
};

struct GatedNormParams {
  NormSplit s;
  const void* x;
  const void* z;         // nullable: no gate
  const float* weight;   // [group] if shared, else [dim]
  int shared, gate_first;
  float eps;
  void* y;               // forward
  const void* dy;        // backward
  void* dx;
  void* dz;
  float* part;           // [slots][dim] partial weight gradients
  unsigned* words;       // workspace header
};

// One column group's place of this thread: true where vector j exists.
template <int NV, int VW> struct NormLane {
  int64_t col;  // first column of the group
  int at[NV];   // element within the group
  bool on[NV];
  __device__ __forceinline__ NormLane(const NormSplit& s) {
    col = static_cast<int64_t>(blockIdx.x % s.ngroups) * s.group;
    const int t = threadIdx.x & (s.T - 1);
#pragma unroll
    for (int j = 0; j < NV; ++j) at[j] = (t + s.T * j) * VW, on[j] = at[j] < s.group;
  }
};

template <class IO, int VW, int NV>
__global__ void __launch_bounds__(kNormThreads) gated_norm_kernel(GatedNormParams p) {
  __shared__ float red[2][4][2];
  int par = 0;
  const NormSplit s = p.s;
  const NormLane<NV, VW> me(s);
  float w[NV][VW];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < VW; ++i) w[j][i] = 0.0f;
    if (me.on[j]) vec_load<F32, VW>(p.weight, me.at[j] + (p.shared ? 0 : me.col), w[j]);
  }
  const int team = threadIdx.x / s.T;
  const float inv = 1.0f / static_cast<float>(s.group);
  const int64_t step = static_cast<int64_t>(s.slots) * s.teams;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x / s.ngroups) * s.teams; r0 < s.rows; r0 += step) {
    const int64_t row = r0 + team;
    const bool live = row < s.rows;
    const int64_t base = row * s.dim + me.col;
    float x[NV][VW], g[NV][VW], sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < VW; ++i) x[j][i] = 0.0f, g[j][i] = 0.0f;
      if (live && me.on[j]) {
        vec_load<IO, VW>(p.x, base + me.at[j], x[j]);
        if (p.z) vec_load<IO, VW>(p.z, base + me.at[j], g[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        if (p.z) g[j][i] = silu_f(g[j][i]);
        if (p.z && p.gate_first) x[j][i] *= g[j][i];
        if (me.on[j]) sum[0] = __builtin_fmaf(x[j][i], x[j][i], sum[0]);
      }
    team_sum<1>(sum, s.T, red, par);
    const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum[0], inv, p.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!live || !me.on[j]) continue;
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        x[j][i] = x[j][i] * rstd * w[j][i];
        if (p.z && !p.gate_first) x[j][i] *= g[j][i];
      }
      vec_store<IO, VW>(p.y, base + me.at[j], x[j]);
    }
  }
}

// Sums NA accumulators per element over the teams of a workgroup (in order, through LDS) into part[slot][dim].
template <int NV, int VW>
__device__ __forceinline__ void team_partials(const float (&acc)[NV][VW], const NormSplit& s,
                                              const NormLane<NV, VW>& me, float* lds, float* part) {
  const int team = threadIdx.x / s.T;
  __syncthreads();  // an earlier use of lds is read
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (me.on[j]) {
#pragma unroll
      for (int i = 0; i < VW; ++i) lds[team * s.group + me.at[j] + i] = acc[j][i];
    }
  __syncthreads();
  const int64_t out = static_cast<int64_t>(blockIdx.x / s.ngroups) * s.dim + me.col;
  for (int e = threadIdx.x; e < s.group; e += kNormThreads) {
    float v = lds[e];
    for (int k = 1; k < s.teams; ++k) v += lds[k * s.group + e];
    part[out + e] = v;
  }
}

constexpr int kNormMaxElems = 32;  // elements per thread at most

template <class IO, int VW, int NV>
__global__ void __launch_bounds__(kNormThreads) gated_norm_bwd_kernel(GatedNormParams p) {
  __shared__ float red[2][4][2];
  __shared__ float lds[kNormThreads * NV * VW];
  int par = 0;
  if (p.words && blockIdx.x == 0 && threadIdx.x < 4) p.words[threadIdx.x] = 0u;
  const NormSplit s = p.s;
  const NormLane<NV, VW> me(s);
  float w[NV][VW], dw[NV][VW];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < VW; ++i) w[j][i] = dw[j][i] = 0.0f;
    if (me.on[j]) vec_load<F32, VW>(p.weight, me.at[j] + (p.shared ? 0 : me.col), w[j]);
  }
  const int team = threadIdx.x / s.T;
  const float inv = 1.0f / static_cast<float>(s.group);
  const int64_t step = static_cast<int64_t>(s.slots) * s.teams;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x / s.ngroups) * s.teams; r0 < s.rows; r0 += step) {
    const int64_t row = r0 + team;
    const bool live = row < s.rows;
    const int64_t base = row * s.dim + me.col;
    Held<IO, VW> hx[NV], hz[NV], hdy[NV];
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      hx[j].clear(), hz[j].clear(), hdy[j].clear();
      if (live && me.on[j]) {
        hx[j].load(p.x, base + me.at[j]);
        hdy[j].load(p.dy, base + me.at[j]);
        if (p.z) hz[j].load(p.z, base + me.at[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[VW], z[VW], dy[VW];
      hx[j].get(x), hz[j].get(z), hdy[j].get(dy);
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        float f = 1.0f, d = 0.0f;
        if (p.z) silu_parts(z[i], f, d);
        const float t = p.gate_first ? x[i] * f : x[i];
        const float m = (p.gate_first ? dy[i] : dy[i] * f) * w[j][i];
        if (me.on[j]) {
          sum[0] = __builtin_fmaf(t, t, sum[0]);
          sum[1] = __builtin_fmaf(m, t, sum[1]);
        }
      }
    }
    team_sum<2>(sum, s.T, red, par);
    const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum[0], inv, p.eps));
    const float c = sum[1] * inv * rstd;  // mean(m n)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!live || !me.on[j]) continue;
      float x[VW], z[VW], dy[VW];
      hx[j].again(), hz[j].again(), hdy[j].again();
      hx[j].get(x), hz[j].get(z), hdy[j].get(dy);
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        float f = 1.0f, d = 0.0f;
        if (p.z) silu_parts(z[i], f, d);
        const float n = (p.gate_first ? x[i] * f : x[i]) * rstd;
        const float dn = p.gate_first ? dy[i] : dy[i] * f;
        dw[j][i] = __builtin_fmaf(dn, n, dw[j][i]);
        const float dt = rstd * __builtin_fmaf(-n, c, dn * w[j][i]);
        const float dzv = p.gate_first ? dt * x[i] * d : dy[i] * n * w[j][i] * d;
        x[i] = p.gate_first ? dt * f : dt;
        z[i] = dzv;
      }
      vec_store<IO, VW>(p.dx, base + me.at[j], x);
      if (p.dz) vec_store<IO, VW>(p.dz, base + me.at[j], z);
    }
  }
  team_partials<NV, VW>(dw, s, me, lds, p.part);
}

struct ResidualNormParams {
  NormSplit s;
  const void* x;
  const void* residual;      // forward: the stream before (nullable: zero); backward: the one after
  const float* scale;        // [dim] (nullable: 1)
  const float* post_weight;  // [dim] (nullable: no norm behind the block)
  const float* weight;       // [dim]
  float eps;
  void* y;                   // forward
  void* residual_out;
  const void* dy;            // backward
  const void* dres_out;      // nullable: zero
  void* dx;
  void* dres;                // nullable
  float* part;               // [3][slots][dim]: dweight, dscale, dpost_weight
  unsigned* words;
};

// IO: storage of x, y (and dx, dy); RIO: storage of the residual stream.
template <class IO, class RIO, int VW, int NV>
__global__ void __launch_bounds__(kNormThreads) residual_norm_kernel(ResidualNormParams p) {
  __shared__ float red[2][4][2];
  int par = 0;
  const NormSplit s = p.s;
  const NormLane<NV, VW> me(s);
  const int team = threadIdx.x / s.T;
  const float inv = 1.0f / static_cast<float>(s.group);
  const int64_t step = static_cast<int64_t>(s.slots) * s.teams;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * s.teams; r0 < s.rows; r0 += step) {
    const int64_t row = r0 + team;
    const bool live = row < s.rows;
    const int64_t base = row * s.dim;
    float x[NV][VW], r[NV][VW], sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < VW; ++i) x[j][i] = r[j][i] = 0.0f;
      if (live && me.on[j]) {
        vec_load<IO, VW>(p.x, base + me.at[j], x[j]);
        if (p.residual) vec_load<RIO, VW>(p.residual, base + me.at[j], r[j]);
      }
    }
    if (p.post_weight) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VW; ++i) sum[0] = __builtin_fmaf(x[j][i], x[j][i], sum[0]);
      team_sum<1>(sum, s.T, red, par);
      const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum[0], inv, p.eps));
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (me.on[j]) {
          float pw[VW];
          vec_load<F32, VW>(p.post_weight, me.at[j], pw);
#pragma unroll
          for (int i = 0; i < VW; ++i) x[j][i] *= rstd * pw[i];
        }
    }
    sum[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (me.on[j]) {
        float sc[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) sc[i] = 1.0f;
        if (p.scale) vec_load<F32, VW>(p.scale, me.at[j], sc);
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          r[j][i] = __builtin_fmaf(sc[i], x[j][i], r[j][i]);
          sum[0] = __builtin_fmaf(r[j][i], r[j][i], sum[0]);
        }
      }
    team_sum<1>(sum, s.T, red, par);
    const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum[0], inv, p.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!live || !me.on[j]) continue;
      float w[VW];
      vec_load<F32, VW>(p.weight, me.at[j], w);
      vec_store<RIO, VW>(p.residual_out, base + me.at[j], r[j]);
#pragma unroll
      for (int i = 0; i < VW; ++i) r[j][i] *= rstd * w[i];
      vec_store<IO, VW>(p.y, base + me.at[j], r[j]);
    }
  }
}

template <class IO, class RIO, int VW, int NV>
__global__ void __launch_bounds__(kNormThreads) residual_norm_bwd_kernel(ResidualNormParams p) {
  __shared__ float red[2][4][2];
  __shared__ float lds[kNormThreads * NV * VW];
  int par = 0;
  if (p.words && blockIdx.x == 0 && threadIdx.x < 4) p.words[threadIdx.x] = 0u;
  const NormSplit s = p.s;
  const NormLane<NV, VW> me(s);
  float dw[NV][VW], dsc[NV][VW], dpw[NV][VW];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VW; ++i) dw[j][i] = dsc[j][i] = dpw[j][i] = 0.0f;
  const int team = threadIdx.x / s.T;
  const float inv = 1.0f / static_cast<float>(s.group);
  const int64_t step = static_cast<int64_t>(s.slots) * s.teams;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * s.teams; r0 < s.rows; r0 += step) {
    const int64_t row = r0 + team;
    const bool live = row < s.rows;
    const int64_t base = row * s.dim;
    Held<IO, VW> hx[NV], hg[NV];
    float r[NV][VW], dr[NV][VW], sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      hx[j].clear(), hg[j].clear();
#pragma unroll
      for (int i = 0; i < VW; ++i) r[j][i] = dr[j][i] = 0.0f;
      if (live && me.on[j]) {
        hx[j].load(p.x, base + me.at[j]);
        vec_load<RIO, VW>(p.residual, base + me.at[j], r[j]);
        hg[j].load(p.dy, base + me.at[j]);
        if (p.dres_out) vec_load<RIO, VW>(p.dres_out, base + me.at[j], dr[j]);
      }
    }
    // the norm in front: dr += rstd (w dy - n mean(w dy n)), n = r rstd
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (me.on[j]) {
        float w[VW], g[VW];
        vec_load<F32, VW>(p.weight, me.at[j], w);
        hg[j].get(g);
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          sum[0] = __builtin_fmaf(r[j][i], r[j][i], sum[0]);
          sum[1] = __builtin_fmaf(g[i] * w[i], r[j][i], sum[1]);
        }
      }
    team_sum<2>(sum, s.T, red, par);
    const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum[0], inv, p.eps));
    const float c = sum[1] * inv * rstd;
    sum[0] = sum[1] = 0.0f;
    // scale and post_weight of a vector, 1 where there is none
    auto factors = [&](int j, float (&sc)[VW], float (&pw)[VW]) {
#pragma unroll
      for (int i = 0; i < VW; ++i) sc[i] = pw[i] = 1.0f;
      if (p.scale) vec_load<F32, VW>(p.scale, me.at[j], sc);
      if (p.post_weight) vec_load<F32, VW>(p.post_weight, me.at[j], pw);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!me.on[j]) continue;
      float w[VW], sc[VW], pw[VW], g[VW], x[VW];
      vec_load<F32, VW>(p.weight, me.at[j], w);
      factors(j, sc, pw);
      hg[j].again();
      hg[j].get(g), hx[j].get(x);
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const float n = r[j][i] * rstd;
        dw[j][i] = __builtin_fmaf(g[i], n, dw[j][i]);
        dr[j][i] += rstd * __builtin_fmaf(-n, c, g[i] * w[i]);
        sum[0] = __builtin_fmaf(x[i], x[i], sum[0]);
        sum[1] = __builtin_fmaf(dr[j][i] * sc[i] * pw[i], x[i], sum[1]);
      }
      if (live && p.dres) vec_store<RIO, VW>(p.dres, base + me.at[j], dr[j]);
    }
    float xr = 1.0f, xc = 0.0f;
    if (p.post_weight) {
      team_sum<2>(sum, s.T, red, par);
      xr = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum[0], inv, p.eps));
      xc = sum[1] * inv * xr;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!live || !me.on[j]) continue;
      float sc[VW], pw[VW], x[VW];
      factors(j, sc, pw);
      hx[j].again();
      hx[j].get(x);
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        const float n = x[i] * xr;  // x itself without a norm behind the block
        dsc[j][i] = __builtin_fmaf(dr[j][i], n * pw[i], dsc[j][i]);
        dpw[j][i] = __builtin_fmaf(dr[j][i] * sc[i], n, dpw[j][i]);
        // past the post weight, into the block's output
        x[i] = xr * __builtin_fmaf(-n, xc, dr[j][i] * sc[i] * pw[i]);
      }
      vec_store<IO, VW>(p.dx, base + me.at[j], x);
    }
  }
  const int64_t plane = static_cast<int64_t>(s.slots) * s.dim;
  team_partials<NV, VW>(dw, s, me, lds, p.part);
  if (p.scale) team_partials<NV, VW>(dsc, s, me, lds, p.part + plane);
  if (p.post_weight) team_partials<NV, VW>(dpw, s, me, lds, p.part + 2 * plane);
}

// out[plane][c] = the sum of the slots' partials of column c, and of columns c + width, ... too where a weight is
// shared by the groups.  One workgroup per 64 columns and plane; its 16 wavefronts take every 16th (slot, group)
// entry in order and are joined in order through LDS.
constexpr int kNormReduceWaves = 16;
struct NormReduceParams {
  const float* part;   // [planes][slots][dim]
  float* out[3];       // per plane: [width] (nullable)
  int64_t slots, dim, width;
};
__global__ void __launch_bounds__(64 * kNormReduceWaves) norm_reduce_kernel(NormReduceParams p) {
  __shared__ float lds[kNormReduceWaves][64];
  float* out = p.out[blockIdx.y];
  if (!out) return;  // the same for the whole workgroup
  const float* part = p.part + static_cast<int64_t>(blockIdx.y) * p.slots * p.dim;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  const int64_t n = p.slots * (p.dim / p.width);  // entries of a column, `width` floats apart
  float v = 0.0f;
  if (c < p.width) {
#pragma unroll 8
    for (int64_t e = w; e < n; e += kNormReduceWaves) v += part[e * p.width + c];
  }
  lds[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < p.width) {
    for (int k = 1; k < kNormReduceWaves; ++k) v += lds[k][lane];
    out[c] = v;
  }
}

}  // namespace ssm
