// delta_host.hpp -- the arguments that the gated delta rule's entry points
// share, and their checks.
#pragma once

#include <stdint.h>

#include "ssm_scan.h"

namespace ssm {

struct DeltaArgs {
  const void *q, *k, *v, *delta;
  const float* A;
  const void* beta;
  const float *bias, *h0;
  const int64_t* cu;
  int64_t nseq, batch, L, heads, headdim, ngroups, dstate;
  int softplus, sigmoid;
  float scale;
  ssm_dtype_t dt;
};

inline bool delta_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool delta_sizes_ok(int64_t batch, int64_t L, int64_t heads, int64_t headdim, int64_t ngroups,
                           int64_t dstate) {
  return batch > 0 && L > 0 && heads > 0 && headdim > 0 && ngroups > 0 && dstate > 0 && heads % ngroups == 0;
}

// States of 32 .. 128 in steps of 32, and 192 and 256; sizes whose products stay far below 2^63.
inline bool delta_shape_supported(int64_t batch, int64_t L, int64_t heads, int64_t headdim, int64_t dstate) {
  if (dstate % 32 != 0 || dstate > 256 || dstate == 160 || dstate == 224) return false;
  if (batch > (1LL << 31) || L > 0x7fffffffLL || heads > (1 << 20) || headdim > (1 << 20)) return false;
  // one workgroup per 32 or more rows of a (row, head) unit: the grid stays below 2^31
  return batch * heads <= 0x7fffffffLL / ((headdim + 31) / 32);
}

// Chunks of 64 tokens: per batch row, or over packed sequences (delta_seq gives sequence s the slots from
// cu[s] / 64 + s on).
inline int64_t delta_slots(int64_t batch, int64_t L, int64_t nseq) {
  return nseq > 0 ? L / 64 + nseq : batch * ((L + 63) / 64);
}
// A workspace starts with a header; the order of packed sequences follows.
constexpr size_t kDeltaHeader = 256;
inline size_t delta_order_bytes(int64_t nseq) {
  return (static_cast<size_t>(nseq) * 4 + 255) & ~static_cast<size_t>(255);
}

inline ssm_status_t check_delta_args(const DeltaArgs& a, const void* y, const float* final_state) {
  if (!a.q || !a.k || !a.v || !a.delta || !a.A || !a.beta || !y) return SSM_ERR_INVALID_ARG;
  if (!delta_sizes_ok(a.batch, a.L, a.heads, a.headdim, a.ngroups, a.dstate)) return SSM_ERR_INVALID_ARG;
  if (a.dt != SSM_DTYPE_F32 && a.dt != SSM_DTYPE_BF16) return SSM_ERR_INVALID_ARG;
  const uintptr_t es = a.dt == SSM_DTYPE_F32 ? 4 : 2;
  // q, k and the states are read in 16-byte pieces
  if (!delta_aligned(a.q, 16) || !delta_aligned(a.k, 16)) return SSM_ERR_INVALID_ARG;
  if (!delta_aligned(a.v, es) || !delta_aligned(a.delta, es) || !delta_aligned(a.beta, es) || !delta_aligned(y, es))
    return SSM_ERR_INVALID_ARG;
  if (!delta_aligned(a.A, 4) || (a.bias && !delta_aligned(a.bias, 4))) return SSM_ERR_INVALID_ARG;
  if ((a.h0 && !delta_aligned(a.h0, 16)) || (final_state && !delta_aligned(final_state, 16)))
    return SSM_ERR_INVALID_ARG;
  if (a.cu && (!delta_aligned(a.cu, 8) || a.batch != 1 || a.nseq <= 0)) return SSM_ERR_INVALID_ARG;
  if (!a.cu && a.nseq > 0) return SSM_ERR_INVALID_ARG;
  if (!delta_shape_supported(a.cu ? a.nseq : a.batch, a.L, a.heads, a.headdim, a.dstate)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

}  // namespace ssm
