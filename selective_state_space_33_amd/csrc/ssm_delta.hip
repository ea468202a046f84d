// ssm_delta.hip -- C-ABI entry points of the gated delta rule, forward and
// one-token step (declared with their contracts in include/ssm_scan.h).
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include "delta_host.hpp"
#include "delta_prep_kernel.hpp"
#include "delta_step_kernel.hpp"
#include "delta_walk_kernel.hpp"
#include "host_common.hpp"
#include "order_kernel.hpp"
#include "ssm_scan.h"

namespace ssm {
namespace {

// Rows of the state per wavefront: 8 RPT.  Over a sequence more rows share the
// loads of the keys and queries, once there are wavefronts enough; a single
// token is bound by the state's way in and out, where more wavefronts are
// better.  Heads of 128, dstate 128, 40 heads, RPT 4 / 1: 512 tokens of 4 rows
// (fp32) 667 / 553 us, 256 of 16 489 / 708, 16 of 256 438 / 769; one token of
// 8, 64, 256 rows 8.0 / 7.8, 53 / 51, 263 / 243.
template <class IO, int DK> hipError_t launch_step(DeltaStepParams& p, int64_t units, hipStream_t s) {
  constexpr int RPT = DK <= 128 ? 4 : 2;
  const int64_t wide = kDeltaStepWaves * 8 * RPT, narrow = kDeltaStepWaves * 8;
  if (p.L > 1 && units * ((p.P + wide - 1) / wide) >= 2 * device_cu_count()) {
    p.row_blocks = (p.P + wide - 1) / wide;
    if (units * p.row_blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    hipLaunchKernelGGL((delta_step_kernel<IO, DK, RPT>), dim3(static_cast<unsigned>(units * p.row_blocks)),
                       dim3(64 * kDeltaStepWaves), 0, s, p);
  } else {
    p.row_blocks = (p.P + narrow - 1) / narrow;
    if (units * p.row_blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    hipLaunchKernelGGL((delta_step_kernel<IO, DK, 1>), dim3(static_cast<unsigned>(units * p.row_blocks)),
                       dim3(64 * kDeltaStepWaves), 0, s, p);
  }
  return hipGetLastError();
}

template <class IO> hipError_t run_step(DeltaStepParams& p, int64_t units, int64_t dstate, hipStream_t s) {
  switch (dstate) {
    case 32: return launch_step<IO, 32>(p, units, s);
    case 64: return launch_step<IO, 64>(p, units, s);
    case 96: return launch_step<IO, 96>(p, units, s);
    case 128: return launch_step<IO, 128>(p, units, s);
    case 192: return launch_step<IO, 192>(p, units, s);
    case 256: return launch_step<IO, 256>(p, units, s);
  }
  return hipErrorInvalidValue;
}

DeltaStepParams step_params(const DeltaArgs& a) {
  DeltaStepParams p = {};
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.delta = a.delta;
  p.A = a.A;
  p.beta = a.beta;
  p.bias = a.bias;
  p.h0 = a.h0;
  p.cu = a.cu;
  p.L = a.L;
  p.H = a.heads;
  p.G = a.ngroups;
  p.P = a.headdim;
  p.softplus = a.softplus;
  p.sigmoid = a.sigmoid;
  p.scale = a.scale;
  return p;
}

// ---- the chunked plan
bool delta_chunked(int64_t L, int64_t heads, int64_t headdim, int64_t dstate, int64_t nseq, ssm_dtype_t dt) {
  if (dt != SSM_DTYPE_BF16 || dstate > 128 || headdim % 16 != 0) return false;
  // a chunk's 64 rows, and as much again behind them, are addressed with 32-bit byte offsets
  if (heads * headdim > (1 << 22) || heads * dstate > (1 << 22)) return false;
  const char* e = getenv("SSM_DELTA_CHUNKED");
  if (e) return atoi(e) != 0;
  // Heads 40 x 128, dstate 128, token by token / chunked: one row of 16 tokens 26 / 30 us, of 32 30 / 30, of 64 55 / 30;
  // 256 sequences of 8 372 / 602, of 16 590 / 614, of 32 1030 / 656.
  return L / (nseq > 0 ? nseq : 1) > 16;
}
template <int DK> hipError_t run_chunked(DeltaChunkParams& p, hipStream_t s) {
  const int64_t grid = p.slots * p.H;
  hipLaunchKernelGGL((delta_prep_kernel<DK, false>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t tiles = p.P / 16, units = p.rows * p.H;
  // Four wavefronts a workgroup while every workgroup gets a CU of its own (a SIMD is then one wavefront's), else eight,
  // which share a head's staging.  Whole calls, 40 heads of 128, dstate 128, four / eight: 2 rows of 4096 tokens 256 /
  // 282 us, 4 rows 484 / 346, 8 rows 767 / 661.
  const int64_t small = units * ((tiles + 3) / 4);
  if (tiles > 4 && small > device_cu_count())
    hipLaunchKernelGGL((delta_walk_kernel<DK, 8, false>), dim3(static_cast<unsigned>(units * ((tiles + 7) / 8))),
                       dim3(512), 0, s, p);
  else
    hipLaunchKernelGGL((delta_walk_kernel<DK, 4, false>), dim3(static_cast<unsigned>(small)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" ssm_status_t ssm_delta_update(float* state, const void* q, const void* k, const void* v,
                                         const void* delta, const float* A, const void* beta,
                                         const float* delta_bias, int softplus_flag, int sigmoid_flag, float scale,
                                         void* y, int64_t batch, int64_t heads, int64_t headdim, int64_t ngroups,
                                         int64_t dstate, ssm_dtype_t dt, hipStream_t stream) {
  if (!state || !y) return SSM_ERR_INVALID_ARG;
  const DeltaArgs a = {q,     k,     v, delta, A,     beta,    delta_bias, state,  nullptr, 0,
                       batch, 1,     heads,    headdim, ngroups, dstate,   softplus_flag ? 1 : 0,
                       sigmoid_flag ? 1 : 0, scale, dt};
  const ssm_status_t st = check_delta_args(a, y, state);
  if (st != SSM_OK) return st;
  DeltaStepParams p = step_params(a);
  p.hT = state;
  p.y = y;
  const hipError_t e = dt == SSM_DTYPE_F32 ? run_step<F32>(p, batch * heads, dstate, stream)
                                           : run_step<BF16>(p, batch * heads, dstate, stream);
  return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

extern "C" size_t ssm_delta_fwd_workspace_size(int64_t batch, int64_t L, int64_t heads, int64_t headdim,
                                               int64_t ngroups, int64_t dstate, int64_t nseq, ssm_dtype_t dt) {
  if (!delta_sizes_ok(batch, L, heads, headdim, ngroups, dstate) || (dt != SSM_DTYPE_F32 && dt != SSM_DTYPE_BF16))
    return 0;
  if ((nseq > 0 && batch != 1) || nseq < 0) return 0;
  if (!delta_shape_supported(nseq > 0 ? nseq : batch, L, heads, headdim, dstate)) return 0;
  if (!delta_chunked(L, heads, headdim, dstate, nseq, dt)) return 0;
  if (delta_slots(batch, L, nseq) > 0x7fffffffLL / heads) return 0;
  return kDeltaHeader + delta_order_bytes(nseq) + static_cast<size_t>(delta_slots(batch, L, nseq)) * heads * kImgBytes;
}

extern "C" ssm_status_t ssm_delta_fwd(const void* q, const void* k, const void* v, const void* delta, const float* A,
                                      const void* beta, const float* delta_bias, int softplus_flag,
                                      int sigmoid_flag, float scale, const float* initial_state,
                                      const int64_t* cu_seqlens, int64_t nseq, void* y, float* final_state,
                                      int64_t batch, int64_t L, int64_t heads, int64_t headdim, int64_t ngroups,
                                      int64_t dstate, ssm_dtype_t dt, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
  const DeltaArgs a = {q,     k, v,     delta,   A,       beta,   delta_bias, initial_state, cu_seqlens, nseq,
                       batch, L, heads, headdim, ngroups, dstate, softplus_flag ? 1 : 0, sigmoid_flag ? 1 : 0,
                       scale, dt};
  const ssm_status_t st = check_delta_args(a, y, final_state);
  if (st != SSM_OK) return st;
  if (!delta_chunked(L, heads, headdim, dstate, nseq, dt) || !delta_aligned(y, 8) || !delta_aligned(v, 8)) {
    DeltaStepParams p = step_params(a);
    p.hT = final_state;
    p.y = y;
    const int64_t units = (cu_seqlens ? nseq : batch) * heads;
    const hipError_t e = dt == SSM_DTYPE_F32 ? run_step<F32>(p, units, dstate, stream)
                                             : run_step<BF16>(p, units, dstate, stream);
    return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
  }
  if (delta_slots(batch, L, nseq) > 0x7fffffffLL / heads) return SSM_ERR_UNSUPPORTED;  // a workgroup for each
  const size_t need = ssm_delta_fwd_workspace_size(batch, L, heads, headdim, ngroups, dstate, nseq, dt);
  if (!workspace || workspace_bytes < need || !delta_aligned(workspace, 256)) return SSM_ERR_INVALID_ARG;
  DeltaChunkParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.delta = delta;
  p.A = A;
  p.beta = beta;
  p.bias = delta_bias;
  p.h0 = initial_state;
  p.hT = final_state;
  p.cu = cu_seqlens;
  p.y = y;
  p.words = static_cast<unsigned*>(workspace);
  // the workspace: header, order of packed sequences, images
  p.order = reinterpret_cast<int*>(static_cast<char*>(workspace) + kDeltaHeader);
  p.img = static_cast<char*>(workspace) + kDeltaHeader + delta_order_bytes(nseq);
  p.rows = cu_seqlens ? nseq : batch;
  p.L = L;
  p.H = heads;
  p.G = ngroups;
  p.P = headdim;
  p.chunks = (L + kDeltaC - 1) / kDeltaC;
  p.slots = delta_slots(batch, L, cu_seqlens ? nseq : 0);
  p.softplus = a.softplus;
  p.sigmoid = a.sigmoid;
  p.scale = scale;
  if (cu_seqlens) {
    hipLaunchKernelGGL(packed_order_kernel, dim3(1), dim3(kOrderBins), 0, stream, p.cu, static_cast<int>(nseq), L,
                       p.order);
    if (hipGetLastError() != hipSuccess) return SSM_ERR_HIP;
  }
  hipError_t e = hipErrorInvalidValue;
  switch (dstate) {
    case 32: e = run_chunked<32>(p, stream); break;
    case 64: e = run_chunked<64>(p, stream); break;
    case 96: e = run_chunked<96>(p, stream); break;
    case 128: e = run_chunked<128>(p, stream); break;
  }
  return e == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}
