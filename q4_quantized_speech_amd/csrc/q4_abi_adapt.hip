// C ABI of the operators that adapt a frozen Q4_0 model (declared in
// include/q4.h): argument validation, then launches on the caller's stream.
// No allocation, no synchronisation.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/q4.h"
#include "q4_kernels.h"
#include "q4_types.h"

using namespace q4;

namespace {

constexpr int64_t MAX_M = int64_t(65535) * 128;
constexpr int64_t MAX_NK = int64_t(1) << 22;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool lora_shape_ok(int64_t M, int64_t N, int64_t K, int64_t R, int64_t adapters) {
  return M >= 1 && M <= MAX_M && N >= 1 && N <= MAX_NK && K >= 32 && K <= MAX_NK && K % 32 == 0 &&
         R >= 8 && R <= 128 && R % 8 == 0 && adapters >= 1 && adapters <= 65535 &&
         M * N < (int64_t(1) << 40) && M * K < (int64_t(1) << 40);
}

// The backward pass has a workgroup per adapter and 64 columns of A and B.
bool lora_grad_shape_ok(int64_t M, int64_t N, int64_t K, int64_t R, int64_t adapters) {
  return lora_shape_ok(M, N, K, R, adapters) &&
         adapters * ((K + 63) / 64 + (N + 63) / 64) <= (int64_t(1) << 21);
}

bool dx_shape_ok(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t most = int64_t(1) << 34;
  return M >= 1 && M <= (int64_t(1) << 20) && N >= 1 && N <= MAX_NK && K >= 32 && K <= MAX_NK &&
         K % 32 == 0 && M * N < most && M * K < most && N * K < most;
}

bool xent_shape_ok(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t most = int64_t(1) << 34;
  return M >= 1 && M <= 65536 && N >= 1 && N < (int64_t(1) << 31) && K >= 32 && K <= MAX_NK &&
         K % 32 == 0 && M * K < most && N * K < most;
}

}  // namespace

extern "C" {

size_t q4_matmul_dx_workspace_bytes(int32_t type, int64_t M, int64_t N, int64_t K) {
  if (!type_ok(type) || !dx_shape_ok(M, N, K)) return 0;
  return matmul_dx_workspace_bytes(type, M, N, K, device_info().cu_count);
}

q4_status q4_matmul_dx(const void* w_q4, const void* dy, void* dx, int32_t type, int64_t M,
                       int64_t N, int64_t K, void* workspace, size_t ws_bytes, void* stream) {
  if (!w_q4 || !dy || !dx) return Q4_ERR_NULL;
  if (!type_ok(type)) return Q4_ERR_FORMAT;
  if (!dx_shape_ok(M, N, K)) return Q4_ERR_SHAPE;
  if (!aligned16(w_q4) || !aligned16(dy) || !aligned16(dx) || !aligned16(workspace))
    return Q4_ERR_ALIGN;
  const int cus = device_info().cu_count;
  if (!workspace || ws_bytes < matmul_dx_workspace_bytes(type, M, N, K, cus))
    return Q4_ERR_WORKSPACE;
  return hip_status(launch_matmul_dx(static_cast<const uint8_t*>(w_q4), dy, dx, type, M, N, K,
                                     workspace, cus, static_cast<hipStream_t>(stream)));
}

size_t q4_lmhead_xent_workspace_bytes(int32_t type, int32_t grad, int64_t M, int64_t N,
                                      int64_t K) {
  if (!type_ok(type) || !xent_shape_ok(M, N, K)) return 0;
  return xent_workspace_bytes(type, grad != 0, M, N, K, 0, device_info().cu_count);
}

q4_status q4_lmhead_xent(const void* w_q4, const void* x, const int32_t* targets,
                         const float* dloss, float* loss, float* lse, void* dx, int32_t type,
                         int64_t M, int64_t N, int64_t K, void* workspace, size_t ws_bytes,
                         void* stream) {
  if (!w_q4 || !x || !targets || !loss || !lse) return Q4_ERR_NULL;
  if (!type_ok(type)) return Q4_ERR_FORMAT;
  if (!xent_shape_ok(M, N, K)) return Q4_ERR_SHAPE;
  if (!aligned16(w_q4) || !aligned16(x) || !aligned16(targets) || !aligned16(dloss) ||
      !aligned16(loss) || !aligned16(lse) || !aligned16(dx) || !aligned16(workspace))
    return Q4_ERR_ALIGN;
  const int cus = device_info().cu_count;
  if (!workspace || ws_bytes < xent_workspace_bytes(type, dx != nullptr, M, N, K, 0, cus))
    return Q4_ERR_WORKSPACE;
  return hip_status(launch_xent(static_cast<const uint8_t*>(w_q4), x, targets, nullptr, dloss, loss,
                                lse, dx, type, M, N, K, workspace, cus, static_cast<hipStream_t>(stream)));
}

size_t q4_lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R) {
  if (!lora_shape_ok(M, N, K, R, 1)) return 0;
  return lora_workspace_bytes(M, K, R, device_info().cu_count);
}

q4_status q4_lora(const void* x, const void* a, const void* b, const float* scale,
                  const int32_t* ids, const void* r, void* y, int32_t type, int32_t atype,
                  int64_t M, int64_t N, int64_t K, int64_t R, int64_t adapters, void* workspace,
                  size_t ws_bytes, void* stream) {
  if (!x || !a || !b || !ids || !y) return Q4_ERR_NULL;
  if (!lora_types_ok(type, atype)) return Q4_ERR_FORMAT;
  if (!lora_shape_ok(M, N, K, R, adapters)) return Q4_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(a) || !aligned16(b) || !aligned16(scale) || !aligned16(ids) ||
      !aligned16(r) || !aligned16(y) || !aligned16(workspace))
    return Q4_ERR_ALIGN;
  const int cus = device_info().cu_count;
  if (!workspace || ws_bytes < lora_workspace_bytes(M, K, R, cus)) return Q4_ERR_WORKSPACE;
  const LoraArgs p = {x,     nullptr, a,     b, r, scale, ids, y,        nullptr,   nullptr,
                      type,  atype,   false, M, N, K,     R,   adapters, workspace,
                      static_cast<hipStream_t>(stream)};
  return hip_status(launch_lora(p, cus));
}

size_t q4_lora_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R) {
  if (!lora_shape_ok(M, N, K, R, 1)) return 0;
  return lora_grad_workspace_bytes(M, N, K, R, device_info().cu_count);
}

q4_status q4_lora_grad(const void* x, const void* dy, const void* a, const void* b,
                       const float* scale, const int32_t* ids, const void* r, void* dx, float* da,
                       float* db, int32_t type, int32_t atype, int64_t M, int64_t N, int64_t K,
                       int64_t R, int64_t adapters, void* workspace, size_t ws_bytes,
                       void* stream) {
  if (!x || !dy || !a || !b || !ids || (!dx && !da && !db)) return Q4_ERR_NULL;
  if (!lora_types_ok(type, atype)) return Q4_ERR_FORMAT;
  if (!lora_grad_shape_ok(M, N, K, R, adapters)) return Q4_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(dy) || !aligned16(a) || !aligned16(b) || !aligned16(scale) ||
      !aligned16(ids) || !aligned16(r) || !aligned16(dx) || !aligned16(da) || !aligned16(db) ||
      !aligned16(workspace))
    return Q4_ERR_ALIGN;
  const int cus = device_info().cu_count;
  if (!workspace || ws_bytes < lora_grad_workspace_bytes(M, N, K, R, cus)) return Q4_ERR_WORKSPACE;
  const LoraArgs p = {x,     dy,    a,    b, r, scale, ids, dx,       da,        db,
                      type,  atype, true, M, N, K,     R,   adapters, workspace,
                      static_cast<hipStream_t>(stream)};
  return hip_status(launch_lora(p, cus));
}

}  // extern "C"
