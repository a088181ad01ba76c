// C ABI of a draft model's operators (declared in include/q4.h): argument
// validation, then launches on the caller's stream.  No allocation, no
// synchronisation.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/q4.h"
#include "q4_kernels.h"
#include "q4_types.h"

using namespace q4;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool act_ok(int32_t act) { return act == Q4_ACT_SILU || act == Q4_ACT_GELU; }

bool ffn_shape_ok(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t most = int64_t(1) << 33;
  return M >= 1 && M <= (int64_t(1) << 20) && N >= 1 && N <= (int64_t(1) << 21) && K >= 32 &&
         K <= (int64_t(1) << 22) && K % 32 == 0 && M * N < most && M * K < most && N * K < most;
}

}  // namespace

extern "C" {

size_t q4_gated_ffn_workspace_bytes(int32_t type, int64_t M, int64_t N, int64_t K) {
  if (!type_ok(type) || !ffn_shape_ok(M, N, K)) return 0;
  return ffn_workspace_bytes(type, M, N, K, device_info().cu_count);
}

q4_status q4_gated_ffn(const void* w_gate, const void* w_up, const void* x, const void* r, void* h,
                       void* z, int32_t act, int32_t type, int64_t M, int64_t N, int64_t K,
                       void* workspace, size_t ws_bytes, void* stream) {
  if (!w_gate || !w_up || !x || !h) return Q4_ERR_NULL;
  if (!type_ok(type) || !act_ok(act)) return Q4_ERR_FORMAT;
  if (!ffn_shape_ok(M, N, K)) return Q4_ERR_SHAPE;
  if (!aligned16(w_gate) || !aligned16(w_up) || !aligned16(x) || !aligned16(r) || !aligned16(h) ||
      !aligned16(z) || !aligned16(workspace))
    return Q4_ERR_ALIGN;
  const int cus = device_info().cu_count;
  const size_t need = ffn_workspace_bytes(type, M, N, K, cus);
  if (need && (!workspace || ws_bytes < need)) return Q4_ERR_WORKSPACE;
  const FfnArgs a = {static_cast<const uint8_t*>(w_gate), static_cast<const uint8_t*>(w_up), x, r, h, z,
                     act, type, M, N, K, workspace, static_cast<hipStream_t>(stream)};
  return hip_status(launch_ffn(a, cus));
}

size_t q4_gated_ffn_grad_workspace_bytes(int32_t type, int64_t M, int64_t N, int64_t K) {
  if (!type_ok(type) || !ffn_shape_ok(M, N, K)) return 0;
  return ffn_grad_workspace_bytes(type, M, N, K, device_info().cu_count);
}

q4_status q4_gated_ffn_grad(const void* w_gate, const void* w_up, const void* z, const void* dh,
                            void* dx, void* dz, int32_t act, int32_t type, int64_t M, int64_t N,
                            int64_t K, void* workspace, size_t ws_bytes, void* stream) {
  if (!w_gate || !w_up || !z || !dh || (!dx && !dz)) return Q4_ERR_NULL;
  if (!type_ok(type) || !act_ok(act)) return Q4_ERR_FORMAT;
  if (!ffn_shape_ok(M, N, K)) return Q4_ERR_SHAPE;
  if (!aligned16(w_gate) || !aligned16(w_up) || !aligned16(z) || !aligned16(dh) || !aligned16(dx) ||
      !aligned16(dz) || !aligned16(workspace))
    return Q4_ERR_ALIGN;
  const int cus = device_info().cu_count;
  if (dx && (!workspace || ws_bytes < ffn_grad_workspace_bytes(type, M, N, K, cus)))
    return Q4_ERR_WORKSPACE;
  const FfnGradArgs a = {static_cast<const uint8_t*>(w_gate), static_cast<const uint8_t*>(w_up), z, dh,
                         dx, dz, act, type, M, N, K, workspace, static_cast<hipStream_t>(stream)};
  return hip_status(launch_ffn_grad(a, cus));
}

}  // extern "C"
