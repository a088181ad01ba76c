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

// Ranges of q4_lmhead_xent, and a thread per teacher entry.
bool distill_shape_ok(int64_t M, int64_t N, int64_t K, int64_t top) {
  constexpr int64_t most = int64_t(1) << 34;
  return M >= 1 && M <= 65536 && N >= 1 && N < (int64_t(1) << 31) && K >= 32 &&
         K <= (int64_t(1) << 22) && K % 32 == 0 && M * K < most && N * K < most && top >= 1 && top <= 256;
}

// Its square and its inverse stay in float32's range.
bool temperature_ok(double t) { return t >= 0x1p-60 && t <= 0x1p60; }

bool verify_shape_ok(int64_t S, int64_t D, int64_t N) {
  return S >= 1 && S <= (int64_t(1) << 20) && D >= 0 && D <= 63 && N >= 1 &&
         N < (int64_t(1) << 31) && S * (D + 1) <= ((int64_t(1) << 40) - 1) / N;
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
  return ffn_grad_workspace_bytes(M, N, K, device_info().cu_count);
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
  if (dx && (!workspace || ws_bytes < ffn_grad_workspace_bytes(M, N, K, cus)))
    return Q4_ERR_WORKSPACE;
  const FfnGradArgs a = {static_cast<const uint8_t*>(w_gate), static_cast<const uint8_t*>(w_up), z, dh,
                         dx, dz, act, type, M, N, K, workspace, static_cast<hipStream_t>(stream)};
  return hip_status(launch_ffn_grad(a, cus));
}

size_t q4_lmhead_distill_workspace_bytes(int32_t type, int32_t grad, int64_t M, int64_t N,
                                         int64_t K, int64_t top) {
  if (!type_ok(type) || !distill_shape_ok(M, N, K, top)) return 0;
  return xent_workspace_bytes(type, grad != 0, M, N, K, top, device_info().cu_count);
}

q4_status q4_lmhead_distill(const void* w_q4, const void* x, const int32_t* top_ids,
                            const float* top_logits, double temperature, const float* dloss,
                            float* loss, float* lse, void* dx, int32_t type, int64_t M, int64_t N,
                            int64_t K, int64_t top, void* workspace, size_t ws_bytes,
                            void* stream) {
  if (!w_q4 || !x || !top_ids || !top_logits || !loss || !lse) return Q4_ERR_NULL;
  if (!type_ok(type)) return Q4_ERR_FORMAT;
  if (!distill_shape_ok(M, N, K, top) || !temperature_ok(temperature)) return Q4_ERR_SHAPE;
  if (!aligned16(w_q4) || !aligned16(x) || !aligned16(top_ids) || !aligned16(top_logits) ||
      !aligned16(dloss) || !aligned16(loss) || !aligned16(lse) || !aligned16(dx) ||
      !aligned16(workspace))
    return Q4_ERR_ALIGN;
  const int cus = device_info().cu_count;
  if (!workspace || ws_bytes < xent_workspace_bytes(type, dx != nullptr, M, N, K, top, cus))
    return Q4_ERR_WORKSPACE;
  const TeacherArgs t = {top_ids, top_logits, top, temperature};
  return hip_status(launch_xent(static_cast<const uint8_t*>(w_q4), x, nullptr, &t, dloss, loss, lse, dx,
                                type, M, N, K, workspace, cus, static_cast<hipStream_t>(stream)));
}

size_t q4_verify_draft_workspace_bytes(int64_t S, int64_t D, int64_t N) {
  return verify_shape_ok(S, D, N) ? verify_workspace_bytes(S, D, N) : 0;
}

q4_status q4_verify_draft(const void* logits, const int32_t* draft, const void* probs,
                          const float* u, const int32_t* lens, double temperature, int32_t* tokens,
                          int32_t* accepted, int32_t type, int64_t S, int64_t D, int64_t N,
                          void* workspace, size_t ws_bytes, void* stream) {
  if (!logits || (!draft && D != 0) || !u || !tokens || !accepted) return Q4_ERR_NULL;
  if (!type_ok(type)) return Q4_ERR_FORMAT;
  if (!verify_shape_ok(S, D, N) || !(temperature == 0.0 || temperature_ok(temperature)))
    return Q4_ERR_SHAPE;
  if (!aligned16(logits) || !aligned16(draft) || !aligned16(probs) || !aligned16(u) ||
      !aligned16(lens) || !aligned16(tokens) || !aligned16(accepted) || !aligned16(workspace))
    return Q4_ERR_ALIGN;
  if (!workspace || ws_bytes < verify_workspace_bytes(S, D, N)) return Q4_ERR_WORKSPACE;
  const VerifyArgs v = {logits, draft, probs, u, lens, temperature, tokens, accepted, type, S, D, N,
                        workspace, static_cast<hipStream_t>(stream)};
  return hip_status(launch_verify(v));
}

}  // extern "C"
