// ssm_norm.hip -- C-ABI entry points of the RMS norms around a layer (declared
// with their contracts in include/ssm_scan.h): argument checks, the split of a
// row over threads, the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "host_common.hpp"
#include "norm_kernels.hpp"
#include "ssm_scan.h"

namespace ssm {
namespace {

bool nm_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t nm_al256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int64_t nm_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t nm_elem(ssm_dtype_t dt) { return dt == SSM_DTYPE_F32 ? 4 : 2; }
bool nm_dtype_ok(ssm_dtype_t dt) { return dt == SSM_DTYPE_F32 || dt == SSM_DTYPE_BF16; }

constexpr int64_t kNormHeader = 256;
constexpr int64_t kNormMaxGroup = kNormThreads * kNormMaxElems;  // 8192 elements in a workgroup's registers

struct NormPlan {
  int VW, NV;
  NormSplit s;
};

enum NormPass { kNormFwd, kNormGatedBwd, kNormResidualBwd };

// Workgroups per CU over all column groups, each walking its rows: a forward's
// eight cost nothing but their start.  A backward's each leave a partial row
// of weight gradients, and a second round of them waits for the first: as many
// as the kernel's registers let share a CU, by the elements of a thread (8, 16,
// 24, 32).  16384 x 1536, 24 elements, gated: three 53 us, four 57; 12289 x
// 2560, 24 elements, residual: two 142 us, four 150.
constexpr int kNormMaxPerCu = 5;
int norm_per_cu(NormPass pass, int elems) {
  if (pass == kNormFwd) return 8;
  const int n = (pass == kNormGatedBwd ? 6 : 5) - (elems + 7) / 8;
  return n < 2 ? 2 : n;
}
int64_t norm_slots(int64_t rows, int64_t ngroups, int per_cu) {
  const int64_t want = nm_ceil(per_cu * device_cu_count(), ngroups);
  return want < rows ? want : rows;
}

// VW elements per vector (1 where a pointer or the row does not allow 16-byte
// accesses); T the fewest threads that hold a group in at most four vectors
// each (eight elements with VW = 1; three in the residual backward, where a
// fourth leaves a CU one workgroup), so that a wavefront serves several short
// groups without a barrier; wider teams only while rows alone do not give
// every CU a workgroup (256 rows, residual forward, wider / not: of 2560 4.5 /
// 5.0 us, of 1536 3.7 / 4.8).
NormPlan plan_norm(int64_t rows, int64_t dim, int64_t group, int vw, NormPass pass) {
  NormPlan pl = {};
  pl.VW = vw;
  const int64_t nvec = nm_ceil(group, vw);
  const int64_t pref = vw == 1 ? 8 : (pass == kNormResidualBwd ? 3 : 4), cap = kNormMaxElems / vw;
  int64_t T = 1;
  while (T < 16 && T < nvec) T *= 2;
  while (T < kNormThreads && nm_ceil(nvec, T) > pref) T *= 2;
  const int64_t ngroups = dim / group;
  while (T < kNormThreads && T < nvec && nm_ceil(rows, kNormThreads / T) * ngroups < device_cu_count()) T *= 2;
  int64_t nv = nm_ceil(nvec, T);
  // the instantiated counts
  if (vw == 1)
    while (nv & (nv - 1)) ++nv;
  else if (vw == 4 && nv > 4)
    nv = 8;
  pl.NV = static_cast<int>(nv <= cap ? nv : 0);
  pl.s.rows = rows;
  pl.s.dim = dim;
  pl.s.group = static_cast<int>(group);
  pl.s.ngroups = static_cast<int>(ngroups);
  pl.s.T = static_cast<int>(T);
  pl.s.teams = static_cast<int>(kNormThreads / T);
  const int64_t most = norm_slots(rows, ngroups, norm_per_cu(pass, pl.NV * vw)), slots = nm_ceil(rows, pl.s.teams);
  pl.s.slots = static_cast<int>(slots < most ? slots : most);
  return pl;
}

// Calls f(IC<VW>, IC<NV>) for the plan's instantiation.
template <int VWMAX, class F> hipError_t norm_dispatch(const NormPlan& pl, F&& f) {
  if (pl.VW == VWMAX) {
    switch (pl.NV) {
      case 1: return f(IC<VWMAX>{}, IC<1>{});
      case 2: return f(IC<VWMAX>{}, IC<2>{});
      case 3: return f(IC<VWMAX>{}, IC<3>{});
      case 4: return f(IC<VWMAX>{}, IC<4>{});
      case 8:
        if constexpr (VWMAX == 4) return f(IC<4>{}, IC<8>{});
    }
  } else {
    switch (pl.NV) {
      case 1: return f(IC<1>{}, IC<1>{});
      case 2: return f(IC<1>{}, IC<2>{});
      case 4: return f(IC<1>{}, IC<4>{});
      case 8: return f(IC<1>{}, IC<8>{});
      case 16: return f(IC<1>{}, IC<16>{});
      case 32: return f(IC<1>{}, IC<32>{});
    }
  }
  return hipErrorInvalidValue;
}

template <class P> hipError_t norm_launch(void (*kernel)(P), int64_t grid, const P& p, hipStream_t s) {
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(kNormThreads), 0, s, p);
  return hipGetLastError();
}

template <class IO> hipError_t run_gated(const NormPlan& pl, GatedNormParams& p, bool bwd, hipStream_t stream) {
  constexpr int VWMAX = sizeof(Raw<IO, 1>) == 2 ? 8 : 4;
  p.s = pl.s;
  const int64_t grid = static_cast<int64_t>(pl.s.ngroups) * pl.s.slots;
  return norm_dispatch<VWMAX>(pl, [&](auto vw, auto nv) {
    constexpr int VW = decltype(vw)::value, NV = decltype(nv)::value;
    return bwd ? norm_launch(gated_norm_bwd_kernel<IO, VW, NV>, grid, p, stream)
               : norm_launch(gated_norm_kernel<IO, VW, NV>, grid, p, stream);
  });
}

template <class IO, class RIO>
hipError_t run_residual(const NormPlan& pl, ResidualNormParams& p, bool bwd, hipStream_t stream) {
  constexpr int VWMAX = sizeof(Raw<IO, 1>) == 2 ? 8 : 4;
  p.s = pl.s;
  return norm_dispatch<VWMAX>(pl, [&](auto vw, auto nv) {
    constexpr int VW = decltype(vw)::value, NV = decltype(nv)::value;
    return bwd ? norm_launch(residual_norm_bwd_kernel<IO, RIO, VW, NV>, pl.s.slots, p, stream)
               : norm_launch(residual_norm_kernel<IO, RIO, VW, NV>, pl.s.slots, p, stream);
  });
}

hipError_t run_reduce(const NormReduceParams& p, int planes, hipStream_t stream) {
  hipLaunchKernelGGL(norm_reduce_kernel, dim3(static_cast<unsigned>(nm_ceil(p.width, 64)), planes),
                     dim3(64 * kNormReduceWaves), 0, stream, p);
  return hipGetLastError();
}

// 16-byte accesses: whole vectors in a group and every pointer (null: absent) on a 16-byte border.
template <size_t n> bool nm_vec_ok(int64_t group, int vw, const void* const (&ptrs)[n]) {
  if (group % vw != 0) return false;
  for (const void* q : ptrs)
    if (q && !nm_aligned(q, 16)) return false;
  return true;
}

bool nm_shape_bad(int64_t rows, int64_t dim, int64_t group, float eps) {
  return rows <= 0 || dim <= 0 || group <= 0 || dim % group != 0 || !(eps >= 0.0f) || __builtin_isinf(eps);
}
// Rows below 2^31, so that slots and grids fit 32 bits; the column count likewise.
bool nm_unsupported(int64_t rows, int64_t dim, int64_t group) {
  return group > kNormMaxGroup || rows > 0x7fffffffLL || dim > 0x7fffffffLL;
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" ssm_status_t ssm_gated_norm_fwd(const void* x, const void* z, const float* weight, int shared_flag,
                                           int gate_first_flag, float eps, void* y, int64_t rows, int64_t dim,
                                           int64_t group, ssm_dtype_t dt, hipStream_t stream) {
  if (!x || !weight || !y || nm_shape_bad(rows, dim, group, eps) || !nm_dtype_ok(dt)) return SSM_ERR_INVALID_ARG;
  const size_t es = nm_elem(dt);
  if (!nm_aligned(x, es) || (z && !nm_aligned(z, es)) || !nm_aligned(y, es) || !nm_aligned(weight, 4))
    return SSM_ERR_INVALID_ARG;
  if (nm_unsupported(rows, dim, group)) return SSM_ERR_UNSUPPORTED;
  const int vw = static_cast<int>(16 / es);
  const void* const ptrs[] = {x, z, weight, y};
  const NormPlan pl = plan_norm(rows, dim, group, nm_vec_ok(group, vw, ptrs) ? vw : 1, kNormFwd);
  GatedNormParams p = {};
  p.x = x;
  p.z = z;
  p.weight = weight;
  p.shared = shared_flag ? 1 : 0;
  p.gate_first = gate_first_flag ? 1 : 0;
  p.eps = eps;
  p.y = y;
  const hipError_t e =
      dt == SSM_DTYPE_F32 ? run_gated<F32>(pl, p, false, stream) : run_gated<BF16>(pl, p, false, stream);
  return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

extern "C" size_t ssm_gated_norm_bwd_workspace_size(int64_t rows, int64_t dim, int64_t group, ssm_dtype_t dt) {
  if (nm_shape_bad(rows, dim, group, 0.0f) || !nm_dtype_ok(dt) || nm_unsupported(rows, dim, group)) return 0;
  return kNormHeader + nm_al256(static_cast<size_t>(norm_slots(rows, dim / group, kNormMaxPerCu)) * dim * sizeof(float));
}

extern "C" ssm_status_t ssm_gated_norm_bwd(const void* x, const void* z, const float* weight, int shared_flag,
                                           int gate_first_flag, float eps, const void* dy, void* dx, void* dz,
                                           float* dweight, int64_t rows, int64_t dim, int64_t group, ssm_dtype_t dt,
                                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!x || !weight || !dy || !dx || !dweight || nm_shape_bad(rows, dim, group, eps) || !nm_dtype_ok(dt))
    return SSM_ERR_INVALID_ARG;
  const size_t es = nm_elem(dt);
  if (!nm_aligned(x, es) || (z && !nm_aligned(z, es)) || !nm_aligned(dy, es) || !nm_aligned(dx, es) ||
      (dz && !nm_aligned(dz, es)) || !nm_aligned(weight, 4) || !nm_aligned(dweight, 4))
    return SSM_ERR_INVALID_ARG;
  if (nm_unsupported(rows, dim, group)) return SSM_ERR_UNSUPPORTED;
  if (!workspace || !nm_aligned(workspace, 256) ||
      workspace_bytes < ssm_gated_norm_bwd_workspace_size(rows, dim, group, dt))
    return SSM_ERR_INVALID_ARG;
  const int vw = static_cast<int>(16 / es);
  const void* const ptrs[] = {x, z, weight, dy, dx, dz};
  const NormPlan pl = plan_norm(rows, dim, group, nm_vec_ok(group, vw, ptrs) ? vw : 1, kNormGatedBwd);
  GatedNormParams p = {};
  p.x = x;
  p.z = z;
  p.weight = weight;
  p.shared = shared_flag ? 1 : 0;
  p.gate_first = gate_first_flag ? 1 : 0;
  p.eps = eps;
  p.dy = dy;
  p.dx = dx;
  p.dz = z ? dz : nullptr;
  p.words = static_cast<unsigned*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kNormHeader);
  hipError_t e = dt == SSM_DTYPE_F32 ? run_gated<F32>(pl, p, true, stream) : run_gated<BF16>(pl, p, true, stream);
  if (e != hipSuccess) return SSM_ERR_HIP;
  NormReduceParams r = {};
  r.part = p.part;
  r.out[0] = dweight;
  r.slots = pl.s.slots;
  r.dim = dim;
  r.width = shared_flag ? group : dim;
  e = run_reduce(r, 1, stream);
  return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

extern "C" ssm_status_t ssm_residual_norm_fwd(const void* x, const void* residual, const float* scale,
                                              const float* post_weight, const float* weight, float eps, void* y,
                                              void* residual_out, int64_t rows, int64_t dim, ssm_dtype_t dt,
                                              ssm_dtype_t res_dt, hipStream_t stream) {
  if (!x || !weight || !y || !residual_out || nm_shape_bad(rows, dim, dim, eps) || !nm_dtype_ok(dt) ||
      !nm_dtype_ok(res_dt))
    return SSM_ERR_INVALID_ARG;
  const size_t es = nm_elem(dt), rs = nm_elem(res_dt);
  if (!nm_aligned(x, es) || !nm_aligned(y, es) || (residual && !nm_aligned(residual, rs)) ||
      !nm_aligned(residual_out, rs))
    return SSM_ERR_INVALID_ARG;
  const float* f32s[] = {scale, post_weight, weight};
  for (const float* q : f32s)
    if (q && !nm_aligned(q, 4)) return SSM_ERR_INVALID_ARG;
  if (nm_unsupported(rows, dim, dim) || (dt == SSM_DTYPE_F32 && res_dt != SSM_DTYPE_F32)) return SSM_ERR_UNSUPPORTED;
  const int vw = static_cast<int>(16 / es);
  const void* const ptrs[] = {x, residual, scale, post_weight, weight, y, residual_out};
  const NormPlan pl = plan_norm(rows, dim, dim, nm_vec_ok(dim, vw, ptrs) ? vw : 1, kNormFwd);
  ResidualNormParams p = {};
  p.x = x;
  p.residual = residual;
  p.scale = scale;
  p.post_weight = post_weight;
  p.weight = weight;
  p.eps = eps;
  p.y = y;
  p.residual_out = residual_out;
  const hipError_t e = dt == SSM_DTYPE_F32       ? run_residual<F32, F32>(pl, p, false, stream)
                       : res_dt == SSM_DTYPE_F32 ? run_residual<BF16, F32>(pl, p, false, stream)
                                                 : run_residual<BF16, BF16>(pl, p, false, stream);
  return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

extern "C" size_t ssm_residual_norm_bwd_workspace_size(int64_t rows, int64_t dim, ssm_dtype_t dt,
                                                       ssm_dtype_t res_dt) {
  if (nm_shape_bad(rows, dim, dim, 0.0f) || !nm_dtype_ok(dt) || !nm_dtype_ok(res_dt) ||
      nm_unsupported(rows, dim, dim) || (dt == SSM_DTYPE_F32 && res_dt != SSM_DTYPE_F32))
    return 0;
  return kNormHeader + nm_al256(3 * static_cast<size_t>(norm_slots(rows, 1, kNormMaxPerCu)) * dim * sizeof(float));
}

extern "C" ssm_status_t ssm_residual_norm_bwd(const void* x, const void* residual_out, const float* scale,
                                              const float* post_weight, const float* weight, float eps,
                                              const void* dy, const void* dresidual_out, void* dx, void* dresidual,
                                              float* dscale, float* dpost_weight, float* dweight, int64_t rows,
                                              int64_t dim, ssm_dtype_t dt, ssm_dtype_t res_dt, void* workspace,
                                              size_t workspace_bytes, hipStream_t stream) {
  if (!x || !residual_out || !weight || !dy || !dx || !dweight || nm_shape_bad(rows, dim, dim, eps) ||
      !nm_dtype_ok(dt) || !nm_dtype_ok(res_dt))
    return SSM_ERR_INVALID_ARG;
  const size_t es = nm_elem(dt), rs = nm_elem(res_dt);
  if (!nm_aligned(x, es) || !nm_aligned(dy, es) || !nm_aligned(dx, es) || !nm_aligned(residual_out, rs) ||
      (dresidual_out && !nm_aligned(dresidual_out, rs)) || (dresidual && !nm_aligned(dresidual, rs)))
    return SSM_ERR_INVALID_ARG;
  const float* f32s[] = {scale, post_weight, weight, dscale, dpost_weight, dweight};
  for (const float* q : f32s)
    if (q && !nm_aligned(q, 4)) return SSM_ERR_INVALID_ARG;
  if (nm_unsupported(rows, dim, dim) || (dt == SSM_DTYPE_F32 && res_dt != SSM_DTYPE_F32)) return SSM_ERR_UNSUPPORTED;
  if (!workspace || !nm_aligned(workspace, 256) ||
      workspace_bytes < ssm_residual_norm_bwd_workspace_size(rows, dim, dt, res_dt))
    return SSM_ERR_INVALID_ARG;
  const int vw = static_cast<int>(16 / es);
  const void* const ptrs[] = {x, residual_out, scale, post_weight, weight, dy, dresidual_out, dx, dresidual};
  const NormPlan pl = plan_norm(rows, dim, dim, nm_vec_ok(dim, vw, ptrs) ? vw : 1, kNormResidualBwd);
  ResidualNormParams p = {};
  p.x = x;
  p.residual = residual_out;
  p.scale = scale;
  p.post_weight = post_weight;
  p.weight = weight;
  p.eps = eps;
  p.dy = dy;
  p.dres_out = dresidual_out;
  p.dx = dx;
  p.dres = dresidual;
  p.words = static_cast<unsigned*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kNormHeader);
  hipError_t e = dt == SSM_DTYPE_F32       ? run_residual<F32, F32>(pl, p, true, stream)
                 : res_dt == SSM_DTYPE_F32 ? run_residual<BF16, F32>(pl, p, true, stream)
                                           : run_residual<BF16, BF16>(pl, p, true, stream);
  if (e != hipSuccess) return SSM_ERR_HIP;
  NormReduceParams r = {};
  r.part = p.part;
  r.out[0] = dweight;
  r.out[1] = scale ? dscale : nullptr;
  r.out[2] = post_weight ? dpost_weight : nullptr;
  r.slots = pl.s.slots;
  r.dim = dim;
  r.width = dim;
  e = run_reduce(r, post_weight ? 3 : scale ? 2 : 1, stream);
  return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}
