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
//
// Distillation shares all of it.  With q the softmax of a row's teacher logits
// over temperature t and l, p the student's logits over t and their softmax:
//
//   loss_m = t^2 sum_j q_j (log q_j - log p_j)
//   dx[m]  = g_m t (sum_{n not the teacher's} p_n T_n + sum_j (p_j - q_j) T_j)
//
// The teacher's tokens are taken out of each piece's logits, as the target is
// above, and their part of the gradient, where p and q nearly cancel once the
// student is trained, is formed in float64 at the end.

#include <algorithm>

#include "q4_gemm16_tiles.h"
#include "q4_kernels.h"
#include "q4_wave.h"

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

// ---------------------------------------------------------------------------
// Distillation
// ---------------------------------------------------------------------------
constexpr int TOP_MAX = 256;  // teacher entries of a row: one thread each

// What the other kernels take of the teacher, [M][top]: q, the entry's token or -1
// (absent, or a repetition of an earlier entry, which has its sum).
struct Teacher {
  double* q;
  int32_t* at;
  float* logit;   // the student's at those tokens
  // M targets for the logits' kernels: the token with q above one half where the loss
  // alone is computed, -1 (none) else
  int32_t* target;
  int top;
  double temperature;
};

// A workgroup per row: q in float64 (loss and gradient are differences from it),
// and inv /= temperature, so that the products come out as l.
// Measured: 8 rows of 16 entries 4.2 us (latency), 1500 of 64 14.7.
__global__ __launch_bounds__(TOP_MAX) void distill_teacher_kernel(const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ logits,
                                                                  double temperature, int64_t N, bool alone,
                                                                  float* __restrict__ inv, Teacher t) {
  __shared__ int32_t id[TOP_MAX], target;
  __shared__ double e[TOP_MAX];
  const int64_t m = blockIdx.x;
  const int j = threadIdx.x;
  const double none = -__builtin_inf();
  double b = none;
  int32_t mine = -1;
  if (j < t.top) {
    mine = ids[m * t.top + j];
    if (mine < 0 || mine >= N) mine = -1;
    if (mine >= 0) b = static_cast<double>(logits[m * t.top + j]) / temperature;
  }
  id[j] = mine;
  e[j] = b;
  if (j == 0) target = -1;
  __syncthreads();
  double top = none;
  for (int i = 0; i < t.top; ++i) top = e[i] > top || e[i] != e[i] ? e[i] : top;
  // a NaN stays the maximum, +inf - +inf is one: either makes the row NaN
  const bool used = top != none;
  __syncthreads();
  const double v = mine >= 0 && used ? (b == none ? (top == top ? 0.0 : top) : exp(b - top)) : 0.0;
  e[j] = v;
  __syncthreads();
  double sum = 0.0, own = 0.0;
  bool first = mine >= 0 && used;
  for (int i = 0; i < t.top; ++i) {
    sum += e[i];
    if (id[i] == mine) {
      own += e[i];
      if (i < j) first = false;
    }
  }
  if (j < t.top) {
    const double q = first ? own / sum : 0.0;
    t.q[m * t.top + j] = q;
    t.at[m * t.top + j] = first ? mine : -1;
    if (alone && q > 0.5) target = mine;
  }
  __syncthreads();
  if (j == 0) {
    t.target[m] = target;
    inv[m] = static_cast<float>(inv[m] / temperature);
  }
}

// Takes the teacher's tokens of a piece out of a row's logits (they become
// -inf, their values are kept in t.logit) and of the 64-column maxima, then
// moves the running maximum and sum as xent_rows_kernel does.
// Measured per piece of 32768 columns, 1500 rows of 64 entries: 10.5 us.
__global__ __launch_bounds__(256) void distill_rows_kernel(
    float* __restrict__ logits, float* __restrict__ tmax, int64_t cols, int64_t ld, int64_t tld,
    int64_t n0, const float* __restrict__ psum, int chunks, float* __restrict__ run_max,
    float* __restrict__ run_sum, float* __restrict__ alpha, int64_t M, bool first, Teacher t) {
  __shared__ float red[4];
  __shared__ int touched[TOP_MAX];
  __shared__ int count;
  const int64_t m = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < t.top) {
    const int64_t n = static_cast<int64_t>(t.at[m * t.top + threadIdx.x]) - n0;
    if (n >= 0 && n < cols) {
      t.logit[m * t.top + threadIdx.x] = logits[m * ld + n];
      logits[m * ld + n] = -__builtin_inff();
      touched[atomicAdd(&count, 1)] = static_cast<int>(n >> 6);
    }
  }
  __syncthreads();
  // in any order: entries of one 64 write the same value
  for (int i = wave; i < count; i += 4) {
    const float top = wave_max(logits[m * ld + 64 * static_cast<int64_t>(touched[i]) + lane]);
    if (lane == 0) tmax[m * tld + touched[i]] = top;
  }
  __syncthreads();
  const int64_t entries = cols / 64;
  float top = -3.402823466e38f;  // with every column taken out: exp(-inf - top) is 0
  for (int64_t e = threadIdx.x; e < entries; e += 256) top = fmaxf(top, tmax[m * tld + e]);
  top = group_max(top, red);
  const float old = first ? top : run_max[m];
  top = fmaxf(top, old);
  const float al = first ? 0.f : exp_below(old, top);
  float s = 0.f;
  if (!first)
    for (int c = threadIdx.x; c < chunks; c += 256) s += psum[static_cast<int64_t>(c) * M + m];
  s = group_sum(s, red);
  if (threadIdx.x == 0) {
    run_sum[m] = first ? 0.f : (run_sum[m] + s) * al;
    alpha[m] = al;
    run_max[m] = top;
  }
}

// The eight weights of dword i of a block of a row of the table, columns
// 4 i .. and 16 + 4 i .. of the block.
__device__ __forceinline__ void weights8(const uint8_t* blk, int i, float (&w)[8]) {
  const float d = half_bits_to_float(*reinterpret_cast<const uint16_t*>(blk));
  const uint16_t* p = reinterpret_cast<const uint16_t*>(blk + 2 + 4 * i);
  const uint32_t q = p[0] | static_cast<uint32_t>(p[1]) << 16;
  const uint32_t lo = q & 0x0F0F0F0Fu, hi = (q >> 4) & 0x0F0F0F0Fu;
  w[0] = ubyte_f<0>(lo); w[1] = ubyte_f<1>(lo); w[2] = ubyte_f<2>(lo); w[3] = ubyte_f<3>(lo);
  w[4] = ubyte_f<0>(hi); w[5] = ubyte_f<1>(hi); w[6] = ubyte_f<2>(hi); w[7] = ubyte_f<3>(hi);
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = (w[e] - 8.f) * d;
}

// Compacts a row's entries (token >= 0) into LDS, their places and tokens in order,
// and returns their number.  All threads, at least 256; ends with a barrier.
__device__ __forceinline__ int row_entries(const Teacher& t, int64_t m, int (&slot)[TOP_MAX],
                                           int (&token)[TOP_MAX], int (&base)[4]) {
  const int j = threadIdx.x, lane = j & 63, wave = j >> 6;
  const int at = j < t.top ? t.at[m * t.top + j] : -1;
  const bool here = at >= 0;
  const uint64_t mask = __ballot(here);
  if (lane == 0 && wave < 4) base[wave] = __popcll(mask);  // (the others hold none)
  __syncthreads();
  int from = 0, all = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) from += base[w];
    all += base[w];
  }
  if (here) {
    const int n = from + __popcll(mask & ((uint64_t(1) << lane) - 1));
    slot[n] = j;
    token[n] = at;
  }
  __syncthreads();
  return all;
}

// Over the first four waves of a workgroup, in all threads (the others bring 0).
__device__ __forceinline__ double group_sum64(double v, double (&red)[4]) {
  v = wave64_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0 && threadIdx.x < TOP_MAX) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return ((red[0] + red[1]) + red[2]) + red[3];
}

// A row's softmax and divergence in float64, thread j its j-th entry.  A student that
// is sure of its teacher's likeliest token has a loss and a gradient far below 1: its
// 1 - p and the teacher's 1 - q are sums over the others, log p and log q those of 1
// less them, so that nothing is left to the rounding of a number next to 1.
struct Divergence {
  double over;  // log z, z = sum_n exp(l_n - base)
  double z, sum;
  double diff;  // p_j - q_j
  // entry j: q and the student's logit less base (q = 0 past the entries); rest: what
  // the tokens that are not the teacher's add to z, with ALL all but the likely one
  template <bool ALL>
  __device__ __forceinline__ Divergence(std::bool_constant<ALL>, bool mine, double q, double d, double rest,
                                        double (&red)[4]) {
    const bool likely = q > 0.5;  // one entry at most
    const double e = mine ? exp(d) : 0.0;
    const double own = group_sum64(likely ? e : 0.0, red);
    const double left = group_sum64(likely ? 0.0 : q, red);  // 1 - q of the likely one
    const double others = ALL ? rest : group_sum64(likely ? 0.0 : e, red) + rest;
    const double top = group_sum64(likely ? d : 0.0, red);
    z = own + others;
    // log z = d + log(1 + others / own) where own is the most of z
    over = own > others ? top + log1p(others / own) : log(z);
    const double logq = likely ? log1p(-left) : log(q);
    sum = group_sum64(mine && q != 0.0 ? q * (logq - d + over) : 0.0, red);
    diff = likely ? left - others / z : e / z - q;
  }
};

// loss, lse and the gradient: one workgroup per row.  Per teacher entry a row of
// the table is decoded, eight weights of a dword at a time.
// Measured: 375 rows of 32 entries, 1280 columns, float32 22 us; 1500 of 64, 3072
// columns, bfloat16 77 (166 MB of table rows: 2.2 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void distill_final_kernel(
    const float* __restrict__ run_max, const float* __restrict__ run_sum,
    const float* __restrict__ psum, int chunks, const float* __restrict__ dloss,
    const float* __restrict__ part, int splits, const uint8_t* __restrict__ W,
    float* __restrict__ loss, float* __restrict__ lse, T* __restrict__ dx, int64_t M, int64_t K,
    Teacher t) {
  __shared__ float red[4], c[TOP_MAX];
  __shared__ double red64[4];
  __shared__ int slot[TOP_MAX], token[TOP_MAX], base[4];
  __shared__ int64_t row[TOP_MAX];
  const int64_t m = blockIdx.x;
  const int count = row_entries(t, m, slot, token, base), j = threadIdx.x;
  const bool mine = j < count;
  const int64_t at = mine ? m * t.top + slot[j] : 0;
  const float l = mine ? t.logit[at] : -__builtin_inff();
  const double q = mine ? t.q[at] : 0.0;
  float rest = run_sum[m];
  for (int i = 0; i < chunks; ++i) rest += psum[static_cast<int64_t>(i) * M + m];
  const float most = run_max[m], top = group_max(fmaxf(l, most), red);
  const double er = exp(static_cast<double>(most) - top);
  const Divergence v(std::false_type{}, mine, q, static_cast<double>(l) - top, rest * er, red64);
  const double tt = t.temperature;
  if (j == 0) {
    lse[m] = static_cast<float>(top + v.over);
    loss[m] = count ? static_cast<float>(tt * tt * v.sum) : 0.f;
  }
  const float g = count ? (dloss ? dloss[m] : 1.f) * static_cast<float>(tt) : 0.f;
  if (mine) {
    c[j] = static_cast<float>(v.diff);
    row[j] = token[j] * (K / 32);
  }
  __syncthreads();
  const float f = static_cast<float>(er / v.z * (1.0 / P_SCALE));
  for (int64_t u = threadIdx.x; u < K / 8; u += 256) {
    const int64_t b = u >> 2;
    const int i = static_cast<int>(u & 3);
    const int64_t k = 32 * b + 4 * i;
    f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
    if (count) {
      for (int p = 0; p < splits; ++p) {
        const float* s = part + (static_cast<int64_t>(p) * M + m) * K + k;
        lo += *reinterpret_cast<const f32x4*>(s);
        hi += *reinterpret_cast<const f32x4*>(s + 16);
      }
      lo *= f;
      hi *= f;
#pragma unroll 4
      for (int n = 0; n < count; ++n) {
        float w[8];
        weights8(W + (row[n] + b) * BLOCK_BYTES, i, w);
        const float cn = c[n];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lo[e] = __builtin_fmaf(cn, w[e], lo[e]);
          hi[e] = __builtin_fmaf(cn, w[4 + e], hi[e]);
        }
      }
    }
    // a row without a teacher is zero whatever it holds: lo and hi are
    const float v0[4] = {g * lo.x, g * lo.y, g * lo.z, g * lo.w};
    const float v1[4] = {g * hi.x, g * hi.y, g * hi.z, g * hi.w};
    store_f32<4>(dx + m * K + k, v0);
    store_f32<4>(dx + m * K + k + 16, v1);
  }
}

// The loss alone.  The student's logits at the teacher's tokens come from the products,
// scales and order of the logits' kernels on the same operands: the same bits as in the
// sums, so a student at its teacher has no loss (a dot product of its own differed by
// up to 1e-6 of either sign).  The waves take the products of 16 tokens and one block
// each (of a tile's 16 rows one counts), then a thread per token adds them in order.
// A: prep_rows' operands.  tmax, tsum (nullable): the maxima and sums of a table in one
// piece, folded here; else run_max and run_sum are.
// Measured: 8 rows of 16 entries, 1280 columns float32, with the fold 10.3 us; latency (dot
// products took 7.1; products and sums by one wave per 16 tokens 22).
constexpr int LOSS_WAVES = 16;
constexpr int LOSS_ITEMS = 512;  // products kept at a time
template <int PA>
__global__ __launch_bounds__(64 * LOSS_WAVES) void distill_loss_kernel(
    const f16x8* __restrict__ A, const float* __restrict__ inv, const uint8_t* __restrict__ W,
    const float* __restrict__ tmax, const float* __restrict__ tsum, int64_t entries, int64_t tld,
    const float* __restrict__ run_max, const float* __restrict__ run_sum, float* __restrict__ lse,
    float* __restrict__ loss, int64_t M, int64_t K, int64_t CB, Teacher t) {
  __shared__ float red[LOSS_WAVES], product[LOSS_ITEMS][16], scale[LOSS_ITEMS][16];
  __shared__ double red64[4];
  __shared__ int slot[TOP_MAX], token[TOP_MAX], base[4];
  const int64_t m = blockIdx.x;
  const int j = threadIdx.x;
  // asked for first: two entries a thread are 131072 columns
  float em[2], es[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t e = j + u * 64 * LOSS_WAVES;
    em[u] = tmax && e < entries ? tmax[m * tld + e] : -__builtin_inff();
    es[u] = tmax && e < entries ? tsum[m * tld + e] : 0.f;
  }
  const int count = row_entries(t, m, slot, token, base);
  const int lane = j & 63, wave = j >> 6, i = lane & 15, g = lane >> 4;
  const bool mine = j < count;
  const int tiles = (count + 15) / 16, r = static_cast<int>(m & 15);
  const int64_t KB = K / 32, part = (M + 15) / 16 * CB * 64;
  const f16x8* a = A + (m >> 4) * CB * 64 + lane;
  float l = 0.f;  // entry j's logit
  for (int64_t b0 = 0; tiles && b0 < KB; b0 += LOSS_ITEMS / tiles) {
    const int blocks = static_cast<int>(min<int64_t>(LOSS_ITEMS / tiles, KB - b0));
#pragma unroll 4
    for (int item = wave; item < blocks * tiles; item += LOSS_WAVES) {
      const int64_t b = b0 + item / tiles;
      const int64_t row = token[min(item % tiles * 16 + i, count - 1)] * KB;
      const uint16_t* p = reinterpret_cast<const uint16_t*>(W + (row + b) * BLOCK_BYTES);
      const f16x8 q = codes8(p[1 + 2 * g] | static_cast<uint32_t>(p[2 + 2 * g]) << 16);
      f32x4 s = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[b * 64], q, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
      if constexpr (PA == 2) s = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[part + b * 64], q, s, 0, 0, 0);
      if (g == r >> 2) {  // row 4 g + v of the tile
        product[item][i] = r & 2 ? (r & 1 ? s.w : s.z) : (r & 1 ? s.y : s.x);
        scale[item][i] = half_bits_to_float(p[0]);
      }
    }
    __syncthreads();
    if (mine) {
#pragma unroll 8
      for (int b = 0; b < blocks; ++b) {
        const int item = b * tiles + (j >> 4);
        l = __builtin_fmaf(scale[item][j & 15], product[item][j & 15], l);
      }
    }
    __syncthreads();
  }
  auto all = [&](float v, auto fold) {  // over the waves, in all threads, in a fixed order
    __syncthreads();
    if (lane == 0) red[wave] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < LOSS_WAVES; ++w) v = fold(v, red[w]);
    return v;
  };
  float top, s = 0.f;
  if (tmax) {
    float own = fmaxf(em[0], em[1]);
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (es[u] != 0.f) s += es[u] * exp_below(em[u], own);
    for (int64_t e = j + 2 * 64 * LOSS_WAVES; e < entries; e += 64 * LOSS_WAVES) {
      const float v = tsum[m * tld + e], up = fmaxf(own, tmax[m * tld + e]);
      s *= exp_below(own, up);
      if (v != 0.f) s += v * exp_below(tmax[m * tld + e], up);
      own = up;
    }
    top = all(wave_max(own), [](float a, float b) { return fmaxf(a, b); });
    if (s != 0.f) s *= exp_below(own, top);
    s = all(wave_sum(s), [](float a, float b) { return a + b; });
  } else {
    top = run_max[m];
    s = run_sum[m];
  }
  const Divergence v(std::true_type{}, mine, mine ? t.q[m * t.top + slot[j]] : 0.0,
                     mine ? static_cast<double>(l * inv[m]) - top : 0.0, s, red64);
  if (j == 0) {
    lse[m] = static_cast<float>(top + v.over);
    loss[m] = count ? static_cast<float>(t.temperature * t.temperature * v.sum) : 0.f;
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
      part, q, at, student, target, total;
};

// top: teacher entries of a row (0: a loss against targets).
XentPlan xent_plan(int type, bool grad, int64_t M, int64_t N, int64_t K, int64_t top, int cus) {
  XentPlan p = {};
  Carver c;
  p.few = !grad && !top && few_rows(M, N, K);
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
  // terms (131072 x 3072, bfloat16: the distance from the rounded exact dx is 7.0
  // to 8.3e-5, that of float32 torch operations 1.6e-4; 20 rows of a table of 700,
  // few terms, up to 2.4e-4 against 5e-5, beside a rounding of 1.6e-3); two parts
  // of both would take three products for one
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
  if (top) {
    p.q = c.take(static_cast<size_t>(M) * top * 8);
    p.at = c.take(static_cast<size_t>(M) * top * 4);
    p.student = c.take(static_cast<size_t>(M) * top * 4);
    p.target = c.take(static_cast<size_t>(M) * 4);
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

size_t xent_workspace_bytes(int type, bool grad, int64_t M, int64_t N, int64_t K, int64_t top, int cus) {
  return xent_plan(type, grad, M, N, K, top, cus).total;
}

hipError_t launch_xent(const uint8_t* w, const void* x, const int32_t* targets,
                       const TeacherArgs* teacher, const float* dloss, float* loss, float* lse, void* dx,
                       int type, int64_t M, int64_t N, int64_t K, void* ws, int cus, hipStream_t s) {
  const bool grad = dx != nullptr;
  const XentPlan p = xent_plan(type, grad, M, N, K, teacher ? teacher->top : 0, cus);
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
  Teacher t = {};
  if (teacher) {
    t = {reinterpret_cast<double*>(base + p.q), reinterpret_cast<int32_t*>(base + p.at), f32(p.student),
         reinterpret_cast<int32_t*>(base + p.target), static_cast<int>(teacher->top), teacher->temperature};
    targets = t.target;
    hipLaunchKernelGGL(distill_teacher_kernel, rows, dim3(TOP_MAX), 0, s, teacher->ids, teacher->logits,
                       teacher->temperature, N, !grad, f32(p.inv), t);
    Q4_TRY(hipGetLastError());
  }
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
      if (teacher && first && last) break;  // folded with the loss
      hipLaunchKernelGGL(xent_rows_kernel<false>, rows, dim3(256), 0, s, f32(p.tmax), f32(p.tsum),
                         entries, p.entries, nullptr, 0, run_max, run_sum, nullptr, M, first, tlogit,
                         targets, N, last && !teacher ? loss : nullptr, lse);
      Q4_TRY(hipGetLastError());
      continue;
    }
    // `chunks` still is the previous piece's count
    if (teacher)
      hipLaunchKernelGGL(distill_rows_kernel, rows, dim3(256), 0, s, f32(p.logits), f32(p.tmax), cols,
                         p.piece, p.entries, n0, f32(p.psum), chunks, run_max, run_sum, f32(p.alpha), M,
                         first, t);
    else
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
  if (!grad) {
    if (teacher) {
      const bool one = p.piece >= N;
      auto* kernel = p.pa == 2 ? distill_loss_kernel<2> : distill_loss_kernel<1>;
      hipLaunchKernelGGL(kernel, rows, dim3(64 * LOSS_WAVES), 0, s, xa, f32(p.inv), w, one ? f32(p.tmax) : nullptr,
                         f32(p.tsum), (N + 63) / 64, p.entries, run_max, run_sum, lse, loss, M, K, blocks32(K), t);
    }
    return hipGetLastError();
  }
  if (teacher) {
    with_type(type, [&](auto v) {
      using T = decltype(v);
      hipLaunchKernelGGL(distill_final_kernel<T>, rows, dim3(256), 0, s, run_max, run_sum, f32(p.psum),
                         chunks, dloss, f32(p.part), p.splits, w, loss, lse, static_cast<T*>(dx), M, K, t);
    });
    return hipGetLastError();
  }
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
