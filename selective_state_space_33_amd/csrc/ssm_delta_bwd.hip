// ssm_delta_bwd.hip -- C-ABI entry points of the gated delta rule's backward
// (declared with their contracts in include/ssm_scan.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "delta_bwd_kernels.hpp"
#include "delta_host.hpp"
#include "host_common.hpp"
#include "order_kernel.hpp"
#include "ssm_scan.h"

namespace ssm {
namespace {

bool bwd_supported(int64_t batch, int64_t L, int64_t heads, int64_t headdim, int64_t dstate, int64_t nseq,
                   ssm_dtype_t dt) {
  if (dt != SSM_DTYPE_BF16 || dstate > 128 || headdim % 16 != 0) return false;
  // a chunk's rows are addressed with 32-bit byte offsets
  if (heads * headdim > (1 << 22) || heads * dstate > (1 << 22)) return false;
  return delta_slots(batch, L, nseq) <= 0x7fffffffLL / heads;
}

// The workspace: [header][order of packed sequences][largest gradients, values' scales, largest values][images][S0][dS]
// [R][dV][the terms of dla][edges][parts of dA, dbias].
struct BwdLayout {
  size_t order, amax, vscale, vmax, img, state, adj, r, dvh, oterm, gterm, lterm, edge, part, total;
};
BwdLayout bwd_layout(int64_t rows, int64_t nseq, int64_t slots, int64_t heads, int64_t headdim, int64_t dstate) {
  const size_t cells = static_cast<size_t>(slots) * heads, tiles = headdim / 16;
  BwdLayout l = {};
  size_t at = kDeltaHeader;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~static_cast<size_t>(255);
    return here;
  };
  l.order = take(delta_order_bytes(nseq));
  l.amax = take(static_cast<size_t>(rows) * heads * 4);
  l.vscale = take(static_cast<size_t>(rows) * heads * 4);
  l.vmax = take(cells * 4);
  l.img = take(cells * kBwdImgBytes);
  l.state = take(cells * tiles * (dstate / 32) * 2 * kFrag);
  l.adj = take(cells * tiles * (dstate / 32) * kFrag);
  l.r = take(cells * tiles * 4 * kFrag);
  l.dvh = take(cells * tiles * 4 * kFrag);
  l.oterm = take(cells * tiles * kDeltaC * 4);
  l.gterm = take(cells * tiles * kDeltaC * 4);
  l.lterm = take(cells * tiles * kDeltaC * 4);
  l.edge = take(cells * tiles * kDeltaC * 4);
  l.part = take(cells * 2 * 4);
  l.total = at;
  return l;
}

template <int DK> hipError_t run_bwd(const DeltaBwdParams& bp, hipStream_t s) {
  constexpr int W = 4;
  const DeltaChunkParams& p = bp.c;
  const unsigned cells = static_cast<unsigned>(p.slots * p.H);
  const unsigned walks = static_cast<unsigned>(p.rows * p.H * ((bp.tiles + W - 1) / W));
  hipLaunchKernelGGL((delta_prep_kernel<DK, true>), dim3(cells), dim3(256), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Four wavefronts a workgroup always: eight would have 256 registers each, and spill (160 heads of 128 channels, dstate
  // 128, 64 chunks in two rounds of workgroups: 528 us; with eight, in one, 718 us).
  hipLaunchKernelGGL((delta_walk_kernel<DK, W, true>), dim3(walks), dim3(64 * W), 0, s, bp);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((delta_bwd_walk_kernel<DK, W>), dim3(walks), dim3(64 * W), 0, s, bp);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((delta_grad_kernel<DK>), dim3(static_cast<unsigned>(p.slots * p.G)), dim3(256), 0, s, bp);
  return hipGetLastError();
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" size_t ssm_delta_bwd_workspace_size(int64_t batch, int64_t L, int64_t heads, int64_t headdim,
                                               int64_t ngroups, int64_t dstate, int64_t nseq, ssm_dtype_t dt) {
  if (!delta_sizes_ok(batch, L, heads, headdim, ngroups, dstate) || (nseq > 0 && batch != 1) || nseq < 0) return 0;
  const int64_t rows = nseq > 0 ? nseq : batch;
  if (!delta_shape_supported(rows, L, heads, headdim, dstate) ||
      !bwd_supported(batch, L, heads, headdim, dstate, nseq, dt))
    return 0;
  return bwd_layout(rows, nseq, delta_slots(batch, L, nseq), heads, headdim, dstate).total;
}

extern "C" ssm_status_t ssm_delta_bwd(const void* q, const void* k, const void* v, const void* delta, const float* A,
                                      const void* beta, const float* delta_bias, int softplus_flag,
                                      int sigmoid_flag, float scale, const void* dy, const float* dfinal_state,
                                      const float* initial_state, const int64_t* cu_seqlens, int64_t nseq, void* dq,
                                      void* dk, void* dv, void* ddelta, float* dA, void* dbeta, float* ddelta_bias,
                                      float* dinitial_state, int64_t batch, int64_t L, int64_t heads,
                                      int64_t headdim, int64_t ngroups, int64_t dstate, ssm_dtype_t dt,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const DeltaArgs a = {q,     k, v,     delta,   A,       beta,   delta_bias, initial_state, cu_seqlens, nseq,
                       batch, L, heads, headdim, ngroups, dstate, softplus_flag ? 1 : 0, sigmoid_flag ? 1 : 0,
                       scale, dt};
  const ssm_status_t st = check_delta_args(a, dy, dinitial_state);
  if (st != SSM_OK) return st;
  if (!dq || !dk || !dv || !ddelta || !dA || !dbeta) return SSM_ERR_INVALID_ARG;
  // v, dy and the gradients of q, k and v pass in 8- and 16-byte pieces
  const void* wide[] = {v, dy, dq, dk, dv};
  for (const void* o : wide)
    if (!delta_aligned(o, 16)) return SSM_ERR_INVALID_ARG;
  if (!delta_aligned(ddelta, 2) || !delta_aligned(dbeta, 2)) return SSM_ERR_INVALID_ARG;
  if (!delta_aligned(dA, 4) || (ddelta_bias && !delta_aligned(ddelta_bias, 4)) ||
      (dfinal_state && !delta_aligned(dfinal_state, 16)))
    return SSM_ERR_INVALID_ARG;
  if (!bwd_supported(batch, L, heads, headdim, dstate, cu_seqlens ? nseq : 0, dt)) return SSM_ERR_UNSUPPORTED;
  const int64_t rows = cu_seqlens ? nseq : batch, slots = delta_slots(batch, L, cu_seqlens ? nseq : 0);
  const BwdLayout l = bwd_layout(rows, cu_seqlens ? nseq : 0, slots, heads, headdim, dstate);
  if (!workspace || workspace_bytes < l.total || !delta_aligned(workspace, 256)) return SSM_ERR_INVALID_ARG;
  char* ws = static_cast<char*>(workspace);
  DeltaBwdParams bp = {};
  DeltaChunkParams& p = bp.c;
  p.q = q;
  p.k = k;
  p.v = v;
  p.delta = delta;
  p.A = A;
  p.beta = beta;
  p.bias = delta_bias;
  p.h0 = initial_state;
  p.cu = cu_seqlens;
  p.order = reinterpret_cast<int*>(ws + l.order);
  p.img = ws + l.img;
  p.words = reinterpret_cast<unsigned*>(ws);
  p.amax = reinterpret_cast<unsigned*>(ws + l.amax);
  p.vscale = reinterpret_cast<float*>(ws + l.vscale);
  p.vmax = reinterpret_cast<unsigned*>(ws + l.vmax);
  p.rows = rows;
  p.L = L;
  p.H = heads;
  p.G = ngroups;
  p.P = headdim;
  p.chunks = (L + kDeltaC - 1) / kDeltaC;
  p.slots = slots;
  p.softplus = a.softplus;
  p.sigmoid = a.sigmoid;
  p.scale = scale;
  bp.dy = dy;
  bp.dfinal = dfinal_state;
  bp.dq = dq;
  bp.dk = dk;
  bp.dv = dv;
  bp.ddelta = ddelta;
  bp.dbeta = dbeta;
  bp.dh0 = dinitial_state;
  bp.state = ws + l.state;
  bp.adj = ws + l.adj;
  bp.r = ws + l.r;
  bp.dvh = ws + l.dvh;
  bp.oterm = reinterpret_cast<float*>(ws + l.oterm);
  bp.gterm = reinterpret_cast<float*>(ws + l.gterm);
  bp.lterm = reinterpret_cast<float*>(ws + l.lterm);
  bp.edge = reinterpret_cast<float*>(ws + l.edge);
  bp.part = reinterpret_cast<float*>(ws + l.part);
  bp.tiles = headdim / 16;
  if (cu_seqlens) {
    hipLaunchKernelGGL(packed_order_kernel, dim3(1), dim3(kOrderBins), 0, stream, p.cu, static_cast<int>(nseq), L,
                       p.order);
    if (hipGetLastError() != hipSuccess) return SSM_ERR_HIP;
  }
  hipError_t e = hipErrorInvalidValue;
  switch (dstate) {
    case 32: e = run_bwd<32>(bp, stream); break;
    case 64: e = run_bwd<64>(bp, stream); break;
    case 96: e = run_bwd<96>(bp, stream); break;
    case 128: e = run_bwd<128>(bp, stream); break;
  }
  if (e != hipSuccess) return SSM_ERR_HIP;
  hipLaunchKernelGGL(delta_gate_sum_kernel, dim3(static_cast<unsigned>(heads)), dim3(256), 0, stream,
                     static_cast<const float*>(bp.part), dA, ddelta_bias, slots, heads);
  return hipGetLastError() == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}
