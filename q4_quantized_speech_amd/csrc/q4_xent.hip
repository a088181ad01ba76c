// Softmax cross entropy of the Q4_0 LM head, in pieces of the vocabulary, and
// its gradient (section "Solutions techniques pour l'exécution dans le
// navigateur", item 3, of "Implémentation en Rust du modèle Voxtral Mini 4B
// Realtime de Mistral pour l'exécuter dans le navigateur": the 131072-row
// table kept in Q4).  With l[m, n] = x[m] . deq(T)[n] and t the row's target:
//
//   lse_m = log sum_n exp l[m, n]       loss_m = lse_m - l[m, t]
//   dx[m] = g_m (sum_{n != t} p_n T_n - (1 - p_t) T_t),  p_n = exp(l - lse)
//
// The logits of one piece exist at a time.  Per piece: the codes are unpacked
// into matrix-core operands (q4_gemm16.h), the logits computed with the exact
// codes, the running maximum and sum of the softmax updated, and, for the
// gradient, the piece's probabilities multiplied by the transposed piece into
// a float32 accumulator that is rescaled when the maximum grows.  1 - p_t is
// the sum of the other probabilities, and the gradient's probabilities are
// taken relative to the largest logit but the target's, brought to the row's
// scale once at the end: a row the model is sure of keeps its small gradient
// and loss, however far the target is above the others.
//
// Up to 64 rows read the table at its Q4_0 size instead, for the logits and for
// the gradient; a few rows without a gradient go through the matvec-accuracy
// kernels.

#include <algorithm>

#include "q4_gemm16.h"
#include "q4_kernels.h"

namespace q4 {
namespace {

constexpr float P_SCALE = 0x1p14f;  // probabilities relative to the largest but the target's, scaled into binary16

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
// exp(a - b) for a <= b; 1 where both are the same infinity.
__device__ __forceinline__ float exp_below(float a, float b) { return a == b ? 1.f : expf(a - b); }

// Over the four waves of a workgroup, in all threads.
__device__ __forceinline__ float group_max(float v, float* red) {
  v = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}
__device__ __forceinline__ float group_sum(float v, float* red) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return ((red[0] + red[1]) + red[2]) + red[3];
}

// loss and lse of a row from its maximum and its sum without the target (et:
// the target's term, 0 for a row without one).
__device__ __forceinline__ void row_loss(float top, float rest, float et, float target_logit,
                                         bool valid, float& loss, float& lse) {
  lse = top + logf(rest + et);
  loss = !valid ? 0.f : et >= rest ? log1pf(rest / et) : logf(rest + et) + (top - target_logit);
}

// Per row, one workgroup each.  GRAD: the new running maximum (of the logits
// but the target's, as tmax is), alpha = the factor that moves sums and gradients to it, and the running sum with the
// previous piece's partial sums (psum [chunks][M]).  Else: the piece's own
// (tmax, tsum) entries folded into the running pair, and after the last piece
// (loss not null) the results.
// Measured: 4.6 us (one row of 32 entries), 4.9 us (38 rows of 2048; 8.7 with the
// maxima read first and the sums after them): latency.
template <bool GRAD>
__global__ __launch_bounds__(256) void xent_rows_kernel(
    const float* __restrict__ tmax, const float* __restrict__ tsum, int64_t entries, int64_t tld,
    const float* __restrict__ psum, int chunks, float* __restrict__ run_max,
    float* __restrict__ run_sum, float* __restrict__ alpha, int64_t M, bool first,
    const float* __restrict__ tlogit, const int32_t* __restrict__ targets, int64_t N,
    float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float red[4];
  constexpr int U = 8;  // entries in flight per thread
  const int64_t m = blockIdx.x;
  float top = -__builtin_inff(), s = 0.f;  // this thread's entries' maximum and (no GRAD) sum
  for (int64_t e0 = threadIdx.x; e0 < entries; e0 += 256 * U) {
    float a[U], b[U], up = top;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t e = e0 + 256 * u;
      a[u] = e < entries ? tmax[m * tld + e] : -__builtin_inff();
      b[u] = !GRAD && e < entries ? tsum[m * tld + e] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) up = fmaxf(up, a[u]);
    if constexpr (!GRAD) {
      s *= exp_below(top, up);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (b[u] != 0.f) s += b[u] * exp_below(a[u], up);
    }
    top = up;
  }
  const float own = top;
  top = group_max(top, red);
  const float old = first ? -__builtin_inff() : run_max[m];
  top = fmaxf(top, old);
  const float al = first ? 0.f : exp_below(old, top);
  if constexpr (GRAD) {
    if (!first)
      for (int c = threadIdx.x; c < chunks; c += 256) s += psum[static_cast<int64_t>(c) * M + m];
    s = group_sum(s, red);
    if (threadIdx.x == 0) {
      run_sum[m] = first ? 0.f : (run_sum[m] + s) * al;
      alpha[m] = al;
      run_max[m] = top;
    }
  } else {
    if (s != 0.f) s *= exp_below(own, top);
    s = group_sum(s, red);
    if (threadIdx.x == 0) {
      const float sum = (first ? 0.f : run_sum[m] * al) + s;
      if (loss) {
        const int64_t t = targets[m];
        const bool valid = t >= 0 && t < N;
        row_loss(top, sum, valid ? exp_below(tlogit[m], top) : 0.f, tlogit[m], valid, loss[m], lse[m]);
      } else {
        run_sum[m] = sum;
        run_max[m] = top;
      }
    }
  }
}

// Probabilities of a piece relative to the running maximum of the logits but
// the target's, as operand fragments (NATURAL over the columns), 16 rows x
// `chunk` columns per workgroup; the target's is left out.  psum[chunk][m]
// their float32 sums.  Scaled by 2^14, a value is stored to 2^-11 (one part) or
// 2^-22 of it, and to 2^-39 of the largest of the others (binary16's smallest
// step is the same for both parts).
constexpr int PC_CHUNK = 2048;
// Measured per piece of 32768 columns: 375 rows in two parts 27 us (98 MB), 1500
// in one 62 us (295 MB, 4.8 TB/s); bound by bytes.
template <int PARTS>
__global__ __launch_bounds__(256) void xent_prob_kernel(const float* __restrict__ logits,
                                                        const float* __restrict__ run_max,
                                                        const int32_t* __restrict__ targets,
                                                        f16x8* __restrict__ out,
                                                        float* __restrict__ psum,
                                                        float* __restrict__ tlogit, int64_t M,
                                                        int64_t cols, int64_t ld, int64_t n0,
                                                        int64_t N) {
  __shared__ float red[4][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int64_t rt = blockIdx.x, m = rt * 16 + i, CB = cols / 32;
  const bool live = m < M;
  const float top = live ? run_max[m] : 0.f;
  const int64_t t = live ? static_cast<int64_t>(targets[m]) - n0 : -1;
  const int64_t b1 = min(CB, static_cast<int64_t>(blockIdx.y + 1) * (PC_CHUNK / 32));
  const int64_t part = static_cast<int64_t>(gridDim.x) * CB * 64;
  float sum = 0.f;
  for (int64_t b = static_cast<int64_t>(blockIdx.y) * (PC_CHUNK / 32) + wave; b < b1; b += 4) {
    const int64_t n = b * 32 + 8 * g;
    f16x8 hi = {}, lo = {};
    if (live) {
      float l[8];
      const f32x4 a = *reinterpret_cast<const f32x4*>(logits + m * ld + n);
      const f32x4 c = *reinterpret_cast<const f32x4*>(logits + m * ld + n + 4);
      l[0] = a.x; l[1] = a.y; l[2] = a.z; l[3] = a.w;
      l[4] = c.x; l[5] = c.y; l[6] = c.z; l[7] = c.w;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float p = 0.f;
        if (n0 + n + e < N) {
          if (t == n + e) {
            tlogit[m] = l[e];
          } else {
            p = exp_below(l[e], top);
          }
        }
        sum += p;
        p *= P_SCALE;
        hi[e] = static_cast<_Float16>(p);
        if constexpr (PARTS == 2) lo[e] = static_cast<_Float16>(p - static_cast<float>(hi[e]));
      }
    }
    const int64_t at = (rt * CB + b) * 64 + lane;
    out[at] = hi;
    if constexpr (PARTS == 2) out[part + at] = lo;
  }
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (lane < 16) red[wave][lane] = sum;
  __syncthreads();
  if (threadIdx.x < 16 && rt * 16 + threadIdx.x < M) {
    const int r = threadIdx.x;
    psum[static_cast<int64_t>(blockIdx.y) * M + rt * 16 + r] =
        ((red[0][r] + red[1][r]) + red[2][r]) + red[3][r];
  }
}

// loss, lse and the gradient: one workgroup per row.  With d the target's logit
// less the largest of the others, top, and rest = sum exp(l - top) without the
// target: p_n = f exp(l[n] - top), f = 1 / (rest + e^d) = e^-d / (rest e^-d + 1),
// the one whose exponential is at most 1.
// Measured: 375 x 3072 float32 20 us, 1500 bfloat16 28 us.
template <typename T>
__global__ __launch_bounds__(256) void xent_final_kernel(
    const float* __restrict__ run_max, const float* __restrict__ run_sum,
    const float* __restrict__ psum, int chunks, const float* __restrict__ tlogit,
    const int32_t* __restrict__ targets, const float* __restrict__ dloss,
    const float* __restrict__ part, int splits, const uint8_t* __restrict__ W,
    float* __restrict__ loss, float* __restrict__ lse, T* __restrict__ dx, int64_t M, int64_t N,
    int64_t K) {
  const int64_t m = blockIdx.x;
  const int64_t t = targets[m];
  const bool valid = t >= 0 && t < N;
  float rest = run_sum[m];
  for (int c = 0; c < chunks; ++c) rest += psum[static_cast<int64_t>(c) * M + m];
  const float top = run_max[m];  // -inf where the target is the only column: d is inf
  const float d = valid ? tlogit[m] - top : -__builtin_inff();
  const float ed = expf(-fabsf(d));
  const float f = d > 0.f ? ed / __builtin_fmaf(rest, ed, 1.f) : 1.f / (rest + ed);
  if (threadIdx.x == 0) {
    const float over = d > 0.f ? log1pf(rest * ed) : logf(rest + ed);  // of lse over the larger of the two
    lse[m] = (d > 0.f ? tlogit[m] : top) + over;
    loss[m] = !valid ? 0.f : d > 0.f ? over : over - d;
  }
  const float g = valid ? (dloss ? dloss[m] : 1.f) : 0.f;
  T* o = dx + m * K;
  for (int64_t k = 4 * threadIdx.x; k < K; k += 1024) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (valid) {
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
      for (int p = 0; p < splits; ++p)
        s += *reinterpret_cast<const f32x4*>(part + (static_cast<int64_t>(p) * M + m) * K + k);
      const uint8_t* blk = W + (t * (K / 32) + k / 32) * BLOCK_BYTES;
      const float ws = half_bits_to_float(*reinterpret_cast<const uint16_t*>(blk));
      const int j = static_cast<int>(k & 31);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t b = blk[2 + ((j + e) & 15)];
        const float w = (static_cast<float>(j < 16 ? b & 15u : b >> 4) - 8.f) * ws;
        v[e] = g * (f * (s[e] * (1.f / P_SCALE) - rest * w));
      }
    }
    store_f32<4>(o + k, v);
  }
}

// Maximum and sum (without the target) of a chunk of a row's logits.
constexpr int FEW_CHUNK = 4096;
// Measured: one row of 131072 4.9 us.
__global__ __launch_bounds__(256) void xent_chunk_kernel(const float* __restrict__ logits,
                                                         const int32_t* __restrict__ targets,
                                                         float* __restrict__ tmax,
                                                         float* __restrict__ tsum,
                                                         float* __restrict__ tlogit, int64_t N) {
  __shared__ float red[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = blockIdx.y;
  const float* l = logits + m * N;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * FEW_CHUNK, t = targets[m];
  float v[FEW_CHUNK / 256], top = -__builtin_inff();
#pragma unroll
  for (int u = 0; u < FEW_CHUNK / 256; ++u) {
    const int64_t n = n0 + u * 256 + threadIdx.x;
    v[u] = n < N ? l[n] : -__builtin_inff();
    top = fmaxf(top, v[u]);
  }
  top = wave_max(top);
  if (lane == 0) red[wave] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < FEW_CHUNK / 256; ++u) {
    const int64_t n = n0 + u * 256 + threadIdx.x;
    if (n < N) {
      if (n == t)
        tlogit[m] = v[u];
      else
        s += exp_below(v[u], top);
    }
  }
  s = wave_sum(s);
  if (lane == 0) red[wave] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    tmax[m * gridDim.x + blockIdx.x] = top;
    tsum[m * gridDim.x + blockIdx.x] = ((red[0] + red[1]) + red[2]) + red[3];
  }
}

template <typename T>
__global__ __launch_bounds__(256) void widen_kernel(const T* __restrict__ x, float* __restrict__ out,
                                                    int64_t quads) {
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < quads;
       e += static_cast<int64_t>(gridDim.x) * 256) {
    float v[4];
    load_f32<4>(x + 4 * e, v);
    store_f32<4>(out + 4 * e, v);
  }
}

constexpr int64_t LOGITS = int64_t(1) << 26;  // kept at a time (256 MiB)

// Losses alone (no gradient) that go through the matvec-accuracy kernels, four
// rows at a time, instead of the matrix cores.  K % 64 == 0: up to four rows
// (131072 x 3072, one row: 49 us against the direct kernel's 69, four 57
// against 71), and up to 16 of a table that gives few of the direct kernel's
// 512-row workgroups long rows to walk (16 rows of 8192 x 3072: 43 against 57;
// of 8192 x 1280 34 against 32).  Otherwise those kernels are slower, and only
// small products go there (1248 columns: one row of 16384 23 us against 36, of
// 65392 55 against 40, eight of 2000 24 against 37; of 160 columns 25 against
// 19).  They keep all logits, which the direct kernel takes in pieces: at most
// as many as one of its pieces.
bool few_rows(int64_t M, int64_t N, int64_t K) {
  if (M * N > LOGITS) return false;
  if (K % 64 == 0) return M <= (N <= 16384 && K >= 2048 ? 16 : 4);
  return K >= 1024 && M <= 16 && M * N * K <= int64_t(1) << 25;
}

struct XentPlan {
  bool few, direct;
  int pa, pp, pb, splits;      // parts of x, of the probabilities and of the transposed weights
  Tile t1, t2;
  int64_t piece, entries, chunks;
  size_t x, inv, run_max, run_sum, tlogit, alpha, tmax, tsum, psum, logits, codes, scale, wt, prob,
      part, total;
};

XentPlan xent_plan(int type, bool grad, int64_t M, int64_t N, int64_t K, int cus) {
  XentPlan p = {};
  Carver c;
  p.few = !grad && few_rows(M, N, K);
  p.direct = !p.few && M <= DIRECT_ROWS;
  p.run_max = c.take(M * 4);
  p.run_sum = c.take(M * 4);
  p.tlogit = c.take(M * 4);
  if (p.few) {
    p.entries = (N + FEW_CHUNK - 1) / FEW_CHUNK;
    if (type != TYPE_F32) p.x = c.take(static_cast<size_t>(M) * K * 4);
    p.logits = c.take(static_cast<size_t>(M) * N * 4);
    p.tmax = c.take(static_cast<size_t>(M) * p.entries * 4);
    p.tsum = c.take(static_cast<size_t>(M) * p.entries * 4);
    p.total = c.at;
    return p;
  }
  p.pa = type == TYPE_F32 ? 2 : 1;
  // the gradient of 16-bit types takes probabilities and weights with 11 bits: a
  // half step of float16 and an eighth of bfloat16's, each averaged over many
  // terms (131072 x 3072, bfloat16: the distance from the rounded exact dx is
  // 7.0e-5, that of float32 torch operations 1.6e-4); two parts of both would
  // take three products for one
  p.pp = p.pa;
  p.pb = p.pa;
  // pieces of equal size, of up to LOGITS logits in rows padded to 16 as the
  // probabilities' are (2048 columns for more than 32768 rows, 512 MiB at
  // 65536), 32768 columns where they are unpacked
  int64_t cap = std::max<int64_t>(2048, LOGITS / ((M + 15) / 16 * 16) / 256 * 256);
  if (!p.direct) cap = std::min<int64_t>(cap, 32768);
  const int64_t pieces = (N + cap - 1) / cap;
  p.piece = ((N + pieces - 1) / pieces + 255) / 256 * 256;
  p.piece = std::min<int64_t>(p.piece, (N + 63) / 64 * 64);
  p.entries = p.piece / 64;
  p.chunks = (p.piece + PC_CHUNK - 1) / PC_CHUNK;
  if (p.direct) {
    p.splits = transposed_plan(M, p.piece, K, p.pp + p.pb - 1, cus).splits;
  } else {
    double best1 = 1e30, best2 = 1e30;
    for (Tile t : {Tile::T256x256, Tile::T128x128}) {
      const double us = tile_time_us(t, M, p.piece, K, p.pa, 1, cus);
      if (us < best1) {
        best1 = us;
        p.t1 = t;
      }
      for (int s = 1; s <= 16 && (s == 1 || p.piece / s >= 128); ++s) {
        const double u2 = tile_time_us(t, M, K, p.piece, p.pp + p.pb - 1, s, cus);
        if (u2 < best2) {
          best2 = u2;
          p.t2 = t;
          p.splits = s;
        }
      }
    }
    p.splits = even_splits(p.piece / 32, p.splits);
  }
  p.x = c.take(static_cast<size_t>(frag_elems(M, K)) * 16 * p.pa);
  p.inv = c.take(M * 4);
  p.alpha = c.take(M * 4);
  p.tmax = c.take(static_cast<size_t>(M) * p.entries * 4);
  if (!p.direct) {
    p.codes = c.take(static_cast<size_t>(frag_elems(p.piece, K)) * 16);
    p.scale = c.take(static_cast<size_t>(p.piece) * blocks32(K) * 4);
  }
  if (grad) {
    p.psum = c.take(static_cast<size_t>(p.chunks) * M * 4);
    p.logits = c.take(static_cast<size_t>(M) * p.piece * 4);
    if (!p.direct) p.wt = c.take(static_cast<size_t>(K) * p.piece * 2 * p.pb);
    p.prob = c.take(static_cast<size_t>(frag_elems(M, p.piece)) * 16 * p.pp);
    p.part = c.take(static_cast<size_t>(p.splits) * M * K * 4);
  } else {
    p.tsum = c.take(static_cast<size_t>(M) * p.entries * 4);
  }
  p.total = c.at;
  return p;
}

#define Q4_TRY(expr)                          \
  do {                                        \
    const hipError_t e_ = (expr);             \
    if (e_ != hipSuccess) return e_;          \
  } while (0)

}  // namespace

size_t xent_workspace_bytes(int type, bool grad, int64_t M, int64_t N, int64_t K, int cus) {
  return xent_plan(type, grad, M, N, K, cus).total;
}

hipError_t launch_xent(const uint8_t* w, const void* x, const int32_t* targets, const float* dloss,
                       float* loss, float* lse, void* dx, int type, int64_t M, int64_t N, int64_t K,
                       void* ws, int cus, hipStream_t s) {
  const bool grad = dx != nullptr;
  const XentPlan p = xent_plan(type, grad, M, N, K, cus);
  char* base = static_cast<char*>(ws);
  auto f32 = [&](size_t at) { return reinterpret_cast<float*>(base + at); };
  float *run_max = f32(p.run_max), *run_sum = f32(p.run_sum), *tlogit = f32(p.tlogit);
  const dim3 rows(static_cast<unsigned>(M));
  int chunks = 0;

  if (p.few) {
    const float* xf = static_cast<const float*>(x);
    if (type != TYPE_F32) {
      const int64_t quads = M * K / 4;
      const unsigned grid = static_cast<unsigned>(std::min<int64_t>((quads + 255) / 256, 1024));
      if (type == TYPE_F16)
        hipLaunchKernelGGL(widen_kernel<_Float16>, dim3(grid), dim3(256), 0, s,
                           static_cast<const _Float16*>(x), f32(p.x), quads);
      else
        hipLaunchKernelGGL(widen_kernel<__bf16>, dim3(grid), dim3(256), 0, s,
                           static_cast<const __bf16*>(x), f32(p.x), quads);
      Q4_TRY(hipGetLastError());
      xf = f32(p.x);
    }
    for (int64_t m = 0; m < M; m += 4)
      Q4_TRY(launch_matmul(w, xf + m * K, f32(p.logits) + m * N, nullptr, std::min<int64_t>(4, M - m),
                           N, K, nullptr, 0, cus, s));
    hipLaunchKernelGGL(xent_chunk_kernel,
                       dim3(static_cast<unsigned>(p.entries), static_cast<unsigned>(M)), dim3(256), 0,
                       s, f32(p.logits), targets, f32(p.tmax), f32(p.tsum), tlogit, N);
    hipLaunchKernelGGL(xent_rows_kernel<false>, rows, dim3(256), 0, s, f32(p.tmax), f32(p.tsum),
                       p.entries, p.entries, nullptr, 0, run_max, run_sum, nullptr, M, true, tlogit,
                       targets, N, loss, lse);
    return hipGetLastError();
  }
  f16x8* xa = reinterpret_cast<f16x8*>(base + p.x);
  f16x8* codes = reinterpret_cast<f16x8*>(base + p.codes);
  f16x8* wt = grad ? reinterpret_cast<f16x8*>(base + p.wt) : nullptr;
  f16x8* prob = reinterpret_cast<f16x8*>(base + p.prob);
  Q4_TRY(prep_rows(x, type, Order::NIBBLE, xa, f32(p.inv), M, K, s));
  for (int64_t n0 = 0; n0 < N; n0 += p.piece) {
    const bool first = n0 == 0;
    const int64_t cols = std::min<int64_t>(p.piece, (N - n0 + 63) / 64 * 64);
    if (!p.direct) Q4_TRY(prep_weights(w, n0, cols, N, K, codes, f32(p.scale), wt, p.pb, s));
    LogitGemm lg = {};
    lg.a = xa;
    lg.q = codes;
    lg.pa = p.pa;
    lg.scale = f32(p.scale);
    lg.inv = f32(p.inv);
    lg.M = M;
    lg.cols = cols;
    lg.K = K;
    lg.CB = blocks32(K);
    lg.n0 = n0;
    lg.N = N;
    lg.targets = targets;
    lg.logits = grad ? f32(p.logits) : nullptr;
    lg.tmax = f32(p.tmax);
    lg.tsum = grad ? nullptr : f32(p.tsum);
    lg.tlogit = tlogit;
    lg.ld = p.piece;
    lg.tld = p.entries;
    Q4_TRY(p.direct ? launch_logits_direct(w, lg, s) : launch_gemm_logits(p.t1, lg, s));
    const int64_t entries = cols / 64;
    if (!grad) {
      const bool last = n0 + p.piece >= N;
      hipLaunchKernelGGL(xent_rows_kernel<false>, rows, dim3(256), 0, s, f32(p.tmax), f32(p.tsum),
                         entries, p.entries, nullptr, 0, run_max, run_sum, nullptr, M, first, tlogit,
                         targets, N, last ? loss : nullptr, lse);
      Q4_TRY(hipGetLastError());
      continue;
    }
    // `chunks` still is the previous piece's count
    hipLaunchKernelGGL(xent_rows_kernel<true>, rows, dim3(256), 0, s, f32(p.tmax), nullptr, entries,
                       p.entries, f32(p.psum), chunks, run_max, run_sum, f32(p.alpha), M, first,
                       nullptr, nullptr, N, nullptr, nullptr);
    chunks = static_cast<int>((cols + PC_CHUNK - 1) / PC_CHUNK);
    const dim3 pg(static_cast<unsigned>((M + 15) / 16), static_cast<unsigned>(chunks));
    if (p.pp == 2)
      hipLaunchKernelGGL(xent_prob_kernel<2>, pg, dim3(256), 0, s, f32(p.logits), run_max, targets,
                         prob, f32(p.psum), tlogit, M, cols, p.piece, n0, N);
    else
      hipLaunchKernelGGL(xent_prob_kernel<1>, pg, dim3(256), 0, s, f32(p.logits), run_max, targets,
                         prob, f32(p.psum), tlogit, M, cols, p.piece, n0, N);
    Q4_TRY(hipGetLastError());
    // a shorter last piece may fill fewer slices: the others keep their sums
    // but still have to move to the new maximum, so every piece uses p.splits
    if (p.direct) {
      TransposedGemm g = {};
      g.g = prob;
      g.pa = p.pp;
      g.pb = p.pb;
      g.type = type;
      g.w = w;
      g.n0 = n0;
      g.N = N;
      g.M = M;
      g.K = K;
      g.CB = cols / 32;
      g.splits = p.splits;
      g.part = f32(p.part);
      g.alpha = first ? nullptr : f32(p.alpha);
      Q4_TRY(launch_gemm_transposed(g, s));
      continue;
    }
    PlainGemm g = {};
    g.a = prob;
    g.b = wt;
    g.pa = p.pp;
    g.pb = p.pb;
    g.M = M;
    g.N = K;
    g.CB = cols / 32;
    g.splits = p.splits;
    g.out = f32(p.part);
    g.ld = K;
    g.alpha = first ? nullptr : f32(p.alpha);
    Q4_TRY(launch_gemm_plain(p.t2, g, s));
  }
  if (!grad) return hipSuccess;
  const float *psum = f32(p.psum), *part = f32(p.part);
  const dim3 grid(static_cast<unsigned>(M));
  const int splits = p.splits;
  if (type == TYPE_F32)
    hipLaunchKernelGGL(xent_final_kernel<float>, grid, dim3(256), 0, s, run_max, run_sum, psum,
                       chunks, tlogit, targets, dloss, part, splits, w, loss, lse,
                       static_cast<float*>(dx), M, N, K);
  else if (type == TYPE_F16)
    hipLaunchKernelGGL(xent_final_kernel<_Float16>, grid, dim3(256), 0, s, run_max, run_sum, psum,
                       chunks, tlogit, targets, dloss, part, splits, w, loss, lse,
                       static_cast<_Float16*>(dx), M, N, K);
  else
    hipLaunchKernelGGL(xent_final_kernel<__bf16>, grid, dim3(256), 0, s, run_max, run_sum, psum,
                       chunks, tlogit, targets, dloss, part, splits, w, loss, lse,
                       static_cast<__bf16*>(dx), M, N, K);
  return hipGetLastError();
}

}  // namespace q4
