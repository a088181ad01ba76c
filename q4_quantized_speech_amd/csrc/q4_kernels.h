// Host-side launchers of the gfx950 kernels (internal to the library; the
// public surface is include/q4.h).  Each returns the hipError_t of its launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4 {

struct DeviceInfo {
  int cu_count;
};
DeviceInfo device_info();
// The q4_status of a HIP call; a failure is kept for q4_last_hip_error().
int hip_status(hipError_t e);

hipError_t launch_matvec(const uint8_t* w, const float* x, float* y, int64_t M, int64_t N,
                         int64_t K, hipStream_t s);

// out_embed (nullable): the decoded table row of each chosen index, [M, K].
hipError_t launch_lmhead_argmax(const uint8_t* w, const float* x, int32_t* out_idx, float* out_val,
                                float* out_embed, int64_t M, int64_t N, int64_t K, void* workspace,
                                hipStream_t s);
size_t lmhead_workspace_bytes(int64_t M);
// The argmax with the library's own per-device scratch (no allocation);
// 1 <= M <= lmhead_noalloc_max_m().
int64_t lmhead_noalloc_max_m();
hipError_t launch_lmhead_argmax_noalloc(const uint8_t* w, const float* x, int32_t* out_idx,
                                        float* out_val, int64_t M, int64_t N, int64_t K,
                                        hipStream_t s);
// Name of the matvec kernel variant launched for (N, K) (argmax or not).
const char* matvec_route(int64_t N, int64_t K, bool argmax);
// Name of the matmul kernel launched for the shape and workspace size, and
// its K split count.
const char* matmul_route(int64_t M, int64_t N, int64_t K, size_t ws_bytes, int cus, int* splits);

// r (nullable): y = r + the product (r is y or does not overlap it); an
// unfused route in place needs M*N floats of workspace for the product.
hipError_t launch_matmul(const uint8_t* w, const float* x, float* y, const float* r, int64_t M,
                         int64_t N, int64_t K, void* ws, size_t ws_bytes, int cus, hipStream_t s);
size_t matmul_workspace_bytes(int64_t M, int64_t N, int64_t K, int cus);
// Whether the residual add rides in a kernel of the product for this plan.
bool matmul_residual_fused(int64_t M, int64_t N, int64_t K, size_t ws_bytes, int cus);
size_t matmul_residual_workspace_bytes(int64_t M, int64_t N, int64_t K, int cus);
// M <= 4, K % 64 == 0: pps (pairs of blocks per K split) a multiple of 4
// when splits > 1; partials [splits][M][N] in P, folded by the caller.
int matmul_small_per_cu();
void launch_matmul_small(const uint8_t* w, const float* x, float* y, float* P, int64_t M,
                         int64_t N, int64_t K, int splits, int pps, hipStream_t s);

// 5 <= M <= 16: chunks of 256 K values per wave of the stream16 kernel
// (0 when it does not serve the shape), and its launch (no workspace).
int matmul_stream16_chunks(int64_t M, int64_t K);
hipError_t launch_matmul_stream16(const uint8_t* w, const float* x, float* y, int64_t M,
                                  int64_t N, int64_t K, int cus, hipStream_t s);

hipError_t launch_embed(const uint8_t* table, const int32_t* ids, float* out, int64_t M,
                        int64_t N, int64_t K, hipStream_t s);

hipError_t launch_quantize(const float* w, uint8_t* out, int64_t N, int64_t K, int32_t* flag,
                           hipStream_t s);

// Low-rank adapters (arguments as in q4_lora and q4_lora_grad; y is dx and n
// the output width in both).
struct LoraArgs {
  const void *x, *dy, *a, *b, *r;
  const float* scale;
  const int32_t* ids;
  void* y;
  float *da, *db;
  int type, atype;
  bool grad;
  int64_t M, N, K, R, adapters;
  void* ws;
  hipStream_t stream;
};
bool lora_types_ok(int type, int atype);
size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t R, int cus);
size_t lora_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int cus);
hipError_t launch_lora(const LoraArgs& p, int cus);

// dX = dY deq(W) (type: element type of dY and dX).
size_t matmul_dx_workspace_bytes(int type, int64_t M, int64_t N, int64_t K, int cus);
hipError_t launch_matmul_dx(const uint8_t* w, const void* dy, void* dx, int type, int64_t M,
                            int64_t N, int64_t K, void* ws, int cus, hipStream_t s);

// The gated feed-forward block (arguments as in q4_gated_ffn and
// q4_gated_ffn_grad).
constexpr int ACT_SILU = 0, ACT_GELU = 1;
struct FfnArgs {
  const uint8_t *gate, *up;
  const void *x, *r;
  void *h, *z;
  int act, type;
  int64_t M, N, K;
  void* ws;
  hipStream_t stream;
};
size_t ffn_workspace_bytes(int type, int64_t M, int64_t N, int64_t K, int cus);
hipError_t launch_ffn(const FfnArgs& a, int cus);
struct FfnGradArgs {
  const uint8_t *gate, *up;
  const void *z, *dh;
  void *dx, *dz;
  int act, type;
  int64_t M, N, K;
  void* ws;
  hipStream_t stream;
};
size_t ffn_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int cus);
hipError_t launch_ffn_grad(const FfnGradArgs& a, int cus);

// Cross entropy of the head against targets, or (teacher not null, targets
// null) against a teacher's softmax over `top` entries a row; dx null: the loss
// alone.
struct TeacherArgs {
  const int32_t* ids;
  const float* logits;
  int64_t top;
  double temperature;
};
size_t xent_workspace_bytes(int type, bool grad, int64_t M, int64_t N, int64_t K, int64_t top, int cus);
hipError_t launch_xent(const uint8_t* w, const void* x, const int32_t* targets,
                       const TeacherArgs* teacher, const float* dloss, float* loss, float* lse, void* dx,
                       int type, int64_t M, int64_t N, int64_t K, void* ws, int cus, hipStream_t s);

// Verification of drafted tokens (arguments as in q4_verify_draft).
struct VerifyArgs {
  const void* logits;
  const int32_t* draft;
  const void* probs;
  const float* u;
  const int32_t* lens;
  double temperature;
  int32_t *tokens, *accepted;
  int type;
  int64_t S, D, N;
  void* ws;
  hipStream_t stream;
};
size_t verify_workspace_bytes(int64_t S, int64_t D, int64_t N);
hipError_t launch_verify(const VerifyArgs& v);

}  // namespace q4
