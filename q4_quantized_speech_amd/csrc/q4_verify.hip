// Verification of drafted tokens against the large model's distribution
// (section "Architecture" of "Implémentation en Rust du modèle Voxtral Mini 4B
// Realtime de Mistral pour l'exécuter dans le navigateur": the decoder reads
// every weight once per pass, so a pass that settles several tokens saves as
// many).  With e_n = exp((l_n - max l) / T) and Z their sum over a row, p = e / Z:
//
//   token i stands if u_i q_i(t_i) Z < e(t_i), and the first that does not is
//   replaced by a draw from max(e - q Z, 0); after the last one a token is drawn
//   from e.
//
// A draw is the lowest n whose running sum passes v times the whole, so its
// outcome hangs on sums over a whole vocabulary: 64-bit exponentials and sums
// make it the same for any order of adding, but for one draw in 10^8.
//
// Three launches: maxima and sums of 4096 columns of every row; the decision
// per sequence (every workgroup of it takes it again from those) and the mass
// of each chunk of the distribution to draw from; the draw.  Bound by reading
// the logits once; the row that is drawn from is read again.

#include <algorithm>

#include "q4_kernels.h"
#include "q4_types.h"
#include "q4_wave.h"

namespace q4 {
namespace {

constexpr int CHUNK = 4096;         // columns of a workgroup
constexpr int PER = CHUNK / 256;    // per thread
constexpr int MAX_ROWS = 64;        // D + 1

// 2^t for -1010 < t <= 0: t = k + f, |f| <= 1/2, 2^f by the polynomial of degree 9
// through it at Chebyshev's nodes (computed in 60 digits; within 1.9e-14 of 2^f),
// k from the last bits of t + 1.5 * 2^52 and added to the exponent.
// (Conversions, ldexp and a Taylor series of 13 terms: verify_stats_kernel 58 us
// against 51 for 384 rows of 131072 float32.)
__device__ __forceinline__ double exp2_near(double t) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  constexpr double BIG = 0x1.8p52;
  const double sum = t + BIG, f = t - (sum - BIG);
  double p = 0x1.b6571de2f2351p-24;
  p = __builtin_fma(p, f, 0x1.63ef969a64d3cp-20);
  p = __builtin_fma(p, f, 0x1.ffcb76789860fp-17);
  p = __builtin_fma(p, f, 0x1.43088e257f341p-13);
  p = __builtin_fma(p, f, 0x1.5d87fe908f88ap-10);
  p = __builtin_fma(p, f, 0x1.3b2ab72b175eep-7);
  p = __builtin_fma(p, f, 0x1.c6b08d7044119p-5);
  p = __builtin_fma(p, f, 0x1.ebfbdff8149f2p-3);
  p = __builtin_fma(p, f, 0x1.62e42fefa39f7p-1);
  p = __builtin_fma(p, f, 0x1.000000000003dp+0);
  u32x2 bits = __builtin_bit_cast(u32x2, p);
  bits.y += __builtin_bit_cast(u32x2, sum).x << 20;
  return __builtin_bit_cast(double, bits);
}
// For any t <= 0, 0 below -1000.
__device__ __forceinline__ double exp2_64(double t) {
  const double r = exp2_near(fmax(t, -1001.0));
  return t > -1000.0 ? r : 0.0;
}

struct Stat {
  double sum;  // of exp((l - max) / T)
  float max;   // NaN if the chunk holds one
  int32_t at;  // lowest column of the maximum (greedy)
};
struct Decision {
  double z;        // the sum of the row that is drawn from
  float top;       // its maximum
  int32_t row;     // a: tokens that stand
  int32_t cut;     // whether drafted token a was refused
  int32_t none;    // no distribution there
  int32_t greedy;  // its best token
  int32_t pad;
};

struct Args {
  const void* logits;
  const int32_t* draft;
  const void* probs;
  const float* u;
  const int32_t* lens;
  int32_t *tokens, *accepted;
  int64_t S, N, chunks;
  int D, greedy;
  double scale;  // log2(e) / T
  Stat* stats;        // [S][D + 1][chunks]
  double* mass;       // [S][chunks]
  Decision* decision; // [S]
};

__device__ __forceinline__ int length(const Args& a, int64_t s) {
  return a.lens ? max(0, min(a.D, a.lens[s])) : a.D;
}

// The larger, NaN if either is.
__device__ __forceinline__ float larger(float a, float b) {
  return a != a || b != b ? __builtin_nanf("") : fmaxf(a, b);
}
__device__ __forceinline__ float wave_larger(float v) {
  return __any(v != v) ? __builtin_nanf("") : wave64_max(v);
}

// Columns n .. n + V - 1 of a row of N (those past it: `fill`).
template <int V, typename T>
__device__ __forceinline__ void load_columns(const T* row, int64_t n, int64_t N, float fill, float (&v)[V]) {
  if (n + V <= N) {
    load_any_f32<V>(row + n, v);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = n + e < N ? to_f32(row[n + e]) : fill;
  }
}

// Measured: 384 rows of 131072 float32 51 us (201 MB: 3.9 TB/s), bfloat16 of 48
// sequences with 0 to 7 drafts 26 us: bound by the float64 instructions of the
// exponentials (17 a column, at half the rate of float32's), not by the bytes.
template <typename T>
__global__ __launch_bounds__(256) void verify_stats_kernel(Args a, uint32_t first) {
  __shared__ float smax[4];
  __shared__ double ssum[4];
  __shared__ int32_t sat[4];
  constexpr int V = 16 / sizeof(T);
  const uint32_t chunks = static_cast<uint32_t>(a.chunks), rows = a.D + 1;
  const uint32_t item = first + blockIdx.x, r = item / chunks, c = item - r * chunks, s = r / rows;
  if (static_cast<int>(r - s * rows) > length(a, s)) return;
  const T* row = static_cast<const T*>(a.logits) + static_cast<int64_t>(r) * a.N;
  const int64_t n0 = static_cast<int64_t>(c) * CHUNK;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float l[PER];
  float top = -__builtin_inff();
#pragma unroll
  for (int u = 0; u < PER / V; ++u) {
    float v[V];
    load_columns<V>(row, n0 + V * (u * 256 + static_cast<int>(threadIdx.x)), a.N, -__builtin_inff(), v);
#pragma unroll
    for (int e = 0; e < V; ++e) l[u * V + e] = v[e];
  }
  float odd = 0.f;  // NaN once a NaN (or an infinity) is among them
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    top = fmaxf(top, l[e]);
    odd = __builtin_fmaf(l[e], 0.f, odd);
  }
  if (odd != odd) {
#pragma unroll
    for (int e = 0; e < PER; ++e) top = larger(top, l[e]);
  }
  top = wave_larger(top);
  if (lane == 0) smax[wave] = top;
  __syncthreads();
  top = larger(larger(smax[0], smax[1]), larger(smax[2], smax[3]));
  Stat out = {0.0, top, -1};
  if (a.greedy) {
    int64_t at = INT64_MAX;
#pragma unroll
    for (int u = PER / V - 1; u >= 0; --u)
#pragma unroll
      for (int e = V - 1; e >= 0; --e)
        if (l[u * V + e] == top) at = n0 + V * (u * 256 + static_cast<int>(threadIdx.x)) + e;
    int32_t best = at < a.N ? static_cast<int32_t>(at) : INT32_MAX;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) best = min(best, __shfl_xor(best, d));
    if (lane == 0) sat[wave] = best;
    __syncthreads();
    out.at = min(min(sat[0], sat[1]), min(sat[2], sat[3]));
  } else {
    double sum = 0.0;
    // a chunk of masked columns has no sum (nor has one that spoils its row)
    if (top > -__builtin_inff() && top < __builtin_inff()) {
      const double t = top;
      // a bound of 2^-900 of the largest, where float32 tells it from the largest
      // (not at temperatures near 0): masked columns, and what is below, count as
      // that much
      const float span = static_cast<float>(900.0 / a.scale);
      if (span > fabsf(top) * 0x1p-20f) {
        const float lowest = top - span;
#pragma unroll
        for (int e = 0; e < PER; ++e)
          sum += exp2_near((static_cast<double>(fmaxf(l[e], lowest)) - t) * a.scale);
      } else {
#pragma unroll 1
        for (int e = 0; e < PER; ++e) sum += exp2_64((static_cast<double>(l[e]) - t) * a.scale);
      }
    }
    sum = wave64_sum(sum);
    if (lane == 0) ssum[wave] = sum;
    __syncthreads();
    out.sum = ((ssum[0] + ssum[1]) + ssum[2]) + ssum[3];
  }
  if (threadIdx.x == 0) a.stats[item] = out;
}

// The decision for sequence s, in all 256 threads.
template <typename T>
__device__ __forceinline__ Decision decide(const Args& a, int64_t s) {
  __shared__ Decision rows[MAX_ROWS];
  __shared__ int stands[MAX_ROWS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, len = length(a, s);
  for (int i = wave; i <= len; i += 4) {
    const int64_t r = s * (a.D + 1) + i;
    const Stat* st = a.stats + r * a.chunks;
    // the token's logit and probability, on their way during the sums
    int64_t t = -1;
    float lt = 0.f;
    double q = 1.0;
    if (i < len) {
      t = a.draft[s * a.D + i];
      if (t < 0 || t >= a.N) t = -1;
      if (t >= 0) {
        lt = to_f32(static_cast<const T*>(a.logits)[r * a.N + t]);
        if (a.probs) q = to_f32(static_cast<const T*>(a.probs)[(s * a.D + i) * a.N + t]);
      }
    }
    float top = -__builtin_inff();
    for (int64_t c = lane; c < a.chunks; c += 64) top = larger(top, st[c].max);
    top = wave_larger(top);
    Decision d = {1.0, top, i, i < len, !(top > -__builtin_inff() && top < __builtin_inff()), -1, 0};
    double et = 0.0;
    if (!d.none) {
      if (a.greedy) {
        int32_t best = INT32_MAX;
        for (int64_t c = lane; c < a.chunks; c += 64)
          if (st[c].max == top) best = min(best, st[c].at);
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) best = min(best, __shfl_xor(best, k));
        d.greedy = best;
        et = t == best ? 1.0 : 0.0;
      } else {
        double z = 0.0;
        for (int64_t c = lane; c < a.chunks; c += 64)
          z += st[c].sum * exp2_64((static_cast<double>(st[c].max) - static_cast<double>(top)) * a.scale);
        d.z = wave64_sum(z);
        et = t < 0 ? 0.0 : exp2_64((static_cast<double>(lt) - static_cast<double>(top)) * a.scale);
      }
    }
    if (lane == 0) {
      rows[i] = d;
      stands[i] = i < len && static_cast<double>(a.u[s * (a.D + 1) + i]) * q * d.z < et;
    }
  }
  __syncthreads();
  int i = 0;
  while (i < len && stands[i]) ++i;
  return rows[i];
}

__device__ __forceinline__ void publish(const Args& a, int64_t s, const Decision& d) {
  for (int i = threadIdx.x; i <= a.D; i += 256)
    if (i != d.row) a.tokens[s * (a.D + 1) + i] = i < d.row ? a.draft[s * a.D + i] : -1;
  if (threadIdx.x == 0) {
    a.accepted[s] = d.row;
    if (d.none || a.greedy) a.tokens[s * (a.D + 1) + d.row] = d.none ? -1 : d.greedy;
  }
}

// What is drawn from, V columns from n: e, or what is left of it once the
// draft's share is gone (`left`).
template <int V, typename T>
__device__ __forceinline__ void entries(const Args& a, int64_t s, const Decision& d, bool left, int64_t n,
                                        double (&w)[V]) {
  float l[V], q[V];
  load_columns<V>(static_cast<const T*>(a.logits) + (s * (a.D + 1) + d.row) * a.N, n, a.N, -__builtin_inff(), l);
  const bool probs = left && a.probs;
  if (probs) load_columns<V>(static_cast<const T*>(a.probs) + (s * a.D + d.row) * a.N, n, a.N, 0.f, q);
  const int64_t t = left && !probs ? a.draft[s * a.D + d.row] : -1;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    w[e] = exp2_64((static_cast<double>(l[e]) - static_cast<double>(d.top)) * a.scale);
    if (probs) w[e] = fmax(__builtin_fma(-static_cast<double>(q[e]), d.z, w[e]), 0.0);
    if (t == n + e) w[e] = 0.0;
  }
}

// `per` workgroups a sequence, each every per-th chunk.
// Measured: one sequence of four drafts 7.4 us (the chain of loads of a decision and
// a chunk), 64 of five 19 to 20 us (67 MB).
template <typename T>
__global__ __launch_bounds__(256) void verify_mass_kernel(Args a, int per) {
  __shared__ double ssum[4];
  constexpr int V = 16 / sizeof(T);
  const uint32_t s = blockIdx.x / static_cast<uint32_t>(per), first = blockIdx.x - s * per;
  const Decision d = decide<T>(a, s);
  if (first == 0) {
    publish(a, s, d);
    if (threadIdx.x == 0) a.decision[s] = d;
  }
  // (what is not cut is known from the first launch)
  if (d.none || a.greedy || !d.cut) return;
  for (int64_t c = first; c < a.chunks; c += per) {
    double w[PER / V][V], sum = 0.0;
#pragma unroll
    for (int u = 0; u < PER / V; ++u)
      entries<V, T>(a, s, d, true, c * CHUNK + V * (u * 256 + static_cast<int>(threadIdx.x)), w[u]);
#pragma unroll
    for (int u = 0; u < PER / V; ++u)
#pragma unroll
      for (int e = 0; e < V; ++e) sum += w[u][e];
    sum = wave64_sum(sum);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) ssum[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) a.mass[s * a.chunks + c] = ((ssum[0] + ssum[1]) + ssum[2]) + ssum[3];
  }
}

// Sum of the earlier threads' values; `all` the whole.
__device__ __forceinline__ double sum_before(double v, double (&ws)[4], double& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double in = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(in, d);
    if (lane >= d) in += o;
  }
  __syncthreads();
  if (lane == 63) ws[wave] = in;
  __syncthreads();
  double before = 0.0;
  all = 0.0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) before += ws[w];
    all += ws[w];
  }
  // the neighbour's inclusive sum, not in - v: a sum over nothing is 0
  const double prev = __shfl_up(in, 1);
  return before + (lane ? prev : 0.0);
}
// The lowest and the highest of the threads' values.
__device__ __forceinline__ int64_t group_min(int64_t v, int64_t (&ws)[4]) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_xor(v, d);
    v = o < v ? o : v;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) ws[threadIdx.x >> 6] = v;
  __syncthreads();
  v = ws[0];
  for (int w = 1; w < 4; ++w) v = ws[w] < v ? ws[w] : v;
  return v;
}

// The draw: the chunk, then the column in it.  Measured: 7.1 us, 64 sequences 8.4:
// the latency of three dependent reads and of the scans.
template <typename T>
__global__ __launch_bounds__(256) void verify_draw_kernel(Args a) {
  __shared__ double ds[4];
  __shared__ int64_t is[4];
  __shared__ double chunk_base;
  const int64_t s = blockIdx.x;
  const Decision d = a.decision[s];
  if (d.none) return;
  const Stat* st = a.stats + (s * (a.D + 1) + d.row) * a.chunks;
  bool left = d.cut;
  auto mass = [&](int64_t c) {
    if (c >= a.chunks) return 0.0;
    if (left) return a.mass[s * a.chunks + c];
    return st[c].sum * exp2_64((static_cast<double>(st[c].max) - static_cast<double>(d.top)) * a.scale);
  };
  const double u = a.u[s * (a.D + 1) + a.D];
  double own = 0.0;  // this thread's chunk, where there are no more chunks than threads
  auto whole = [&]() {
    double v = 0.0, all;
    for (int64_t c = threadIdx.x; c < a.chunks; c += 256) v += own = mass(c);
    sum_before(v, ds, all);
    return all;
  };
  double total = whole();
  if (left && !(total > 0.0)) {  // nothing of p is above q
    left = false;
    own = 0.0;
    total = whole();
  }
  const double goal = u * total;
  // the first chunk whose running sum passes the goal; failing that (a number
  // of 1 or more, or a rounding), the last one that holds anything
  int64_t chunk = INT64_MAX, last = -1;
  double base = 0.0;
  for (int64_t c0 = 0; c0 < a.chunks; c0 += 256) {
    const int64_t c = c0 + threadIdx.x;
    const double v = a.chunks <= 256 ? own : mass(c);
    double all;
    const double before = base + sum_before(v, ds, all);
    const int64_t hit = group_min(v > 0.0 && before + v > goal ? c : INT64_MAX, is);
    const int64_t high = -group_min(v > 0.0 ? -c : INT64_MAX, is);
    if (high >= 0) last = high;
    const int64_t take = hit != INT64_MAX ? hit : high >= 0 ? high : -1;
    __syncthreads();
    if (c == take) chunk_base = before;
    __syncthreads();
    if (hit != INT64_MAX) {
      chunk = hit;
      break;
    }
    base += all;
  }
  if (chunk == INT64_MAX) chunk = last;
  if (chunk < 0) {  // cannot be: the largest logit's entry is 1
    if (threadIdx.x == 0) a.tokens[s * (a.D + 1) + d.row] = -1;
    return;
  }
  // sixteen neighbours per thread
  const int64_t n0 = chunk * CHUNK + PER * static_cast<int>(threadIdx.x);
  double w[PER], v = 0.0;
  entries<PER, T>(a, s, d, left, n0, w);
#pragma unroll
  for (int e = 0; e < PER; ++e) v += w[e];
  double all;
  double run = chunk_base + sum_before(v, ds, all);
  int64_t hit = INT64_MAX, high = -1;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    run += w[e];
    if (w[e] > 0.0) {
      high = n0 + e;
      if (hit == INT64_MAX && run > goal) hit = n0 + e;
    }
  }
  hit = group_min(hit, is);
  high = -group_min(high >= 0 ? -high : INT64_MAX, is);
  if (threadIdx.x == 0)
    a.tokens[s * (a.D + 1) + d.row] = static_cast<int32_t>(hit != INT64_MAX ? hit : high);
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

size_t verify_workspace_bytes(int64_t S, int64_t D, int64_t N) {
  const int64_t chunks = (N + CHUNK - 1) / CHUNK;
  return align256(S * (D + 1) * chunks * sizeof(Stat)) + align256(S * chunks * sizeof(double)) +
         align256(S * sizeof(Decision));
}

hipError_t launch_verify(const VerifyArgs& v) {
  Args a = {};
  a.logits = v.logits;
  a.draft = v.draft;
  a.probs = v.D ? v.probs : nullptr;
  a.u = v.u;
  a.lens = v.lens;
  a.tokens = v.tokens;
  a.accepted = v.accepted;
  a.S = v.S;
  a.N = v.N;
  a.chunks = (v.N + CHUNK - 1) / CHUNK;
  a.D = static_cast<int>(v.D);
  a.greedy = v.temperature == 0.0;
  a.scale = a.greedy ? 1.0 : 1.4426950408889634 / v.temperature;
  char* base = static_cast<char*>(v.ws);
  a.stats = reinterpret_cast<Stat*>(base);
  base += align256(v.S * (v.D + 1) * a.chunks * sizeof(Stat));
  a.mass = reinterpret_cast<double*>(base);
  base += align256(v.S * a.chunks * sizeof(double));
  a.decision = reinterpret_cast<Decision*>(base);
  // a dimension takes fewer than 2^32 threads: S (D + 1) ceil(N / CHUNK), which is below
  // 2^29, in launches of at most 2^23 workgroups
  const int64_t items = v.S * (v.D + 1) * a.chunks;
  constexpr int64_t MOST = int64_t(1) << 23;
  // every workgroup takes the decision: about as many as run at once
  const int per = a.greedy ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(a.chunks, 1024 / v.S)));
  hipError_t status = hipSuccess;
  // after a launch that fails there is none: it would read what was not written
  with_type(v.type, [&](auto t) {
    using T = decltype(t);
    for (int64_t first = 0; first < items; first += MOST) {
      hipLaunchKernelGGL(verify_stats_kernel<T>, dim3(static_cast<unsigned>(std::min(MOST, items - first))),
                         dim3(256), 0, v.stream, a, static_cast<uint32_t>(first));
      if ((status = hipGetLastError()) != hipSuccess) return;
    }
    hipLaunchKernelGGL(verify_mass_kernel<T>, dim3(static_cast<unsigned>(v.S * per)), dim3(256), 0, v.stream, a,
                       per);
    if ((status = hipGetLastError()) != hipSuccess || a.greedy) return;
    hipLaunchKernelGGL(verify_draw_kernel<T>, dim3(static_cast<unsigned>(v.S)), dim3(256), 0, v.stream, a);
    status = hipGetLastError();
  });
  return status;
}

}  // namespace q4
