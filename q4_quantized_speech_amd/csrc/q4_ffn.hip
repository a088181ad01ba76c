// The gated feed-forward block on Q4_0 weights and its gradient (section
// "Architecture" of "Implémentation en Rust du modèle Voxtral Mini 4B Realtime
// de Mistral pour l'exécuter dans le navigateur": the decoder's gate and up
// projections, which read the most weights of a layer):
//
//   g = r_g + x Wg^T    u = r_u + x Wu^T    h = act(g) u
//   dg = dh u act'(g)   du = dh act(g)      dx = dg Wg + du Wu
//
// A workgroup computes the same columns of both projections, so that the
// activation and the product are taken from its registers: g and u reach
// memory only where the caller keeps them.  Few rows read the Q4_0 bytes
// directly and are bound by them; more rows multiply unpacked codes on the
// matrix cores, gate and up interleaved.  The gradient goes through the
// transposed product on the bytes (q4_gemm16.h), dg and du as its operands.

#include <algorithm>

#include "q4_gemm16_tiles.h"
#include "q4_kernels.h"

namespace q4 {
namespace {

// ---------------------------------------------------------------------------
// Activations.  With s = sigmoid(a), 1 - s from the exponential as well: the
// derivative keeps its precision on both sides.
// ---------------------------------------------------------------------------
// EXACT: expf and a full division; else the hardware's exponential and
// reciprocal (a few units of 2^-24, far below a 16-bit result's rounding).
template <bool EXACT>
__device__ __forceinline__ void sigmoid(float a, float& s, float& rest) {
  const float t = EXACT ? expf(-fabsf(a)) : __expf(-fabsf(a));
  const float big = EXACT ? 1.f / (1.f + t) : __builtin_amdgcn_rcpf(1.f + t);
  const float small = t * big;
  s = a < 0.f ? small : big;
  rest = a < 0.f ? big : small;
}
constexpr float GELU_2A = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float GELU_B = 0.044715f;

// act(g); GRAD: slope = act'(g).
template <int ACT, bool EXACT, bool GRAD>
__device__ __forceinline__ float activate(float g, float& slope) {
  float s, rest;
  if constexpr (ACT == ACT_SILU) {
    sigmoid<EXACT>(g, s, rest);
    if constexpr (GRAD) slope = __builtin_fmaf(g * s, rest, s);
  } else {
    const float q = g * g;
    sigmoid<EXACT>(GELU_2A * g * __builtin_fmaf(GELU_B, q, 1.f), s, rest);
    if constexpr (GRAD) {
      const float p = s * rest;  // 0 for large |g|, where q may be infinite
      slope = p == 0.f ? s : __builtin_fmaf(g * p, GELU_2A * __builtin_fmaf(3.f * GELU_B, q, 1.f), s);
    }
  }
  return g * s;
}

// One element of the block from the two sums: h, and z where it is kept.
struct Out {
  const void* r;
  void *h, *z;
  int64_t M, N;
  int act;
};
template <typename T>
__device__ __forceinline__ void finish(const Out& o, int64_t m, int64_t n, float g, float u) {
  const int64_t at = m * 2 * o.N + n;
  if (o.r) {
    g += to_f32(static_cast<const T*>(o.r)[at]);
    u += to_f32(static_cast<const T*>(o.r)[at + o.N]);
  }
  if (o.z) {
    static_cast<T*>(o.z)[at] = from_f32<T>(g);
    static_cast<T*>(o.z)[at + o.N] = from_f32<T>(u);
  }
  constexpr bool EXACT = sizeof(T) == 4;
  float slope;
  const float a = o.act == ACT_SILU ? activate<ACT_SILU, EXACT, false>(g, slope)
                                    : activate<ACT_GELU, EXACT, false>(g, slope);
  static_cast<T*>(o.h)[m * o.N + n] = from_f32<T>(a * u);
}

// ---------------------------------------------------------------------------
// Few rows, straight from the Q4_0 bytes.  A workgroup owns 16 NT columns of
// each projection; its eight waves share them and take every eighth chunk of
// 128 k, and their sums are added in LDS at the end: all of a short matrix's
// bytes are requested at once, whatever its height.
//
// Lane (i, g) loads block g of the chunk of weight row i: a 16-bit scale and 16
// bytes of codes, at any even address.  A 4 x 4 transposition over the lane
// groups gives it dword g of each of the four blocks, the operand of the exact
// codes q - 8, and the scales of all four.
// ---------------------------------------------------------------------------
constexpr int FW = 8;            // waves
constexpr int64_t FEW_ROWS = 64; // rows of x this route takes

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Row g (lanes 16 g .. 16 g + 15) of r[t] holds X[g][t]; afterwards row g of
// r[p] holds X[p][g].
__device__ __forceinline__ void transpose4(uint32_t (&r)[4]) {
  const auto a = __builtin_amdgcn_permlane32_swap(r[0], r[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(r[1], r[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  r[0] = c[0];
  r[1] = c[1];
  r[2] = d[0];
  r[3] = d[1];
}

// The largest over the four lane groups, in all of them.
__device__ __forceinline__ float groups_max(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// This lane's blocks of a chunk, one of each of the workgroup's row tiles.
template <int TILES>
struct RawChunk {
  uint32_t q[TILES][4];
  int d[TILES];  // bits of the scale
  __device__ __forceinline__ void load(const uint8_t* const (&row)[TILES], int64_t c, int g, int64_t CB) {
    const int64_t off = min(4 * c + g, CB - 1) * BLOCK_BYTES;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const u32x4 v = *reinterpret_cast<const u32x4_any*>(row[t] + off + 2);
      d[t] = *reinterpret_cast<const uint16_t*>(row[t] + off);
      q[t][0] = v.x; q[t][1] = v.y; q[t][2] = v.z; q[t][3] = v.w;
    }
  }
};

// The activations of a chunk, up to 16 rows, read and split here: a row's chunk
// is scaled by a power of two into binary16 (float16 as it is).  Row a of the
// operand is row (a >> 2) + 4 (a & 3) of x, so that up to four rows lie in the
// first of a result's registers.  (More rows come as fragments from prep_rows.)
template <int PA, typename T>
struct Acts {
  typedef T vec __attribute__((ext_vector_type(4)));
  vec v[4][2];
  const T* row;
  __device__ __forceinline__ Acts(const void* x, int64_t M, int64_t K, int lane) {
    const int a = lane & 15;
    row = static_cast<const T*>(x) + min<int64_t>((a >> 2) + 4 * (a & 3), M - 1) * K + 4 * (lane >> 4);
  }
  __device__ __forceinline__ void load(int64_t c, int64_t CB) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const T* p = row + min(4 * c + b, CB - 1) * 32;
      v[b][0] = *reinterpret_cast<const vec*>(p);
      v[b][1] = *reinterpret_cast<const vec*>(p + 16);
    }
  }
  // The power of two that brings the chunk's largest magnitude to binary16's
  // range.
  __device__ __forceinline__ float scale() {
    if constexpr (__is_same(T, _Float16)) return 1.f;
    float top = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(to_f32(static_cast<T>(v[b][e >> 2][e & 3]))));
    top = row_scale(groups_max(top));
    // the values stay packed until their fragment is made
#pragma unroll
    for (int b = 0; b < 4; ++b) asm volatile("" : "+v"(v[b][0]), "+v"(v[b][1]));
    return top;
  }
  __device__ __forceinline__ void fragment(int b, float s, f16x8 (&a)[1][PA]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = to_f32(static_cast<T>(v[b][e >> 2][e & 3])) * s;
      a[0][0][e] = static_cast<_Float16>(x);
      if constexpr (PA == 2) a[0][1][e] = static_cast<_Float16>(x - static_cast<float>(a[0][0][e]));
    }
  }
};

template <int RT, int PA, int NT, int VR, typename T>
__global__ __launch_bounds__(64 * FW) __attribute__((amdgpu_waves_per_eu(RT == 1 ? 4 : 2)))
void ffn_few_kernel(const uint8_t* __restrict__ Wg, const uint8_t* __restrict__ Wu,
                    const void* __restrict__ X, const float* __restrict__ inv, int64_t K, Out o) {
  constexpr int TILES = 2 * NT;  // gate's, then up's
  __shared__ float red[FW][TILES][VR][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int64_t CB = K / 32, chunks = (CB + 3) / 4, AB = (CB + 1) / 2 * 2;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NT);
  const uint8_t* row[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t)
    row[t] = (t < NT ? Wg : Wu) + min(n0 + 16 * (t % NT) + i, o.N - 1) * CB * BLOCK_BYTES;

  f32x4 acc[RT][TILES];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  // A chunk: step 4-block-major, codes of block s / TILES of tile s % TILES
  // against a(b); a step's scaled sums are taken while the next one's products
  // run.  The empty volatile asm keeps that order: regrouped, all products
  // first, their results would spill.
  auto chunk = [&](RawChunk<TILES>& w, int64_t c, const float (&is)[VR], auto&& acts) {
    constexpr int STEPS = 4 * TILES;
    f16x8 a[2][RT][PA];
    f32x4 p[2][RT];
    int from = 4 * i;  // of the scale's lane, in bytes
    asm volatile("" : "+v"(from));
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      transpose4(w.q[t]);
      if (4 * c + g >= CB) w.d[t] = 0;  // blocks past the row have no weight
    }
    float d[2];
    auto products = [&](int s) {
      const int b = s / TILES, t = s % TILES;
      if (t == 0 && b + 1 < 4) acts(b + 1, a[(b + 1) & 1]);
      d[s & 1] = half_bits_to_float(static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(from + 64 * b, w.d[t])));
      const f16x8 q = codes8(w.q[t][b]);
#pragma unroll
      for (int r = 0; r < RT; ++r)
        p[s & 1][r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[b & 1][r][0], q, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
      if constexpr (PA == 2) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
          p[s & 1][r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[b & 1][r][1], q, p[s & 1][r], 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) asm volatile("" : "+v"(p[s & 1][r])::"memory");
    };
    acts(0, a[0]);
    products(0);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (s + 1 < STEPS) products(s + 1);
      const int t = s % TILES;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int v = 0; v < VR; ++v)
          acc[r][t][v] = __builtin_fmaf(RT == 1 ? d[s & 1] * is[v] : d[s & 1], p[s & 1][r][v], acc[r][t][v]);
        asm volatile("" : "+v"(acc[r][t]));
      }
    }
  };

  // one chunk is multiplied while the next one's bytes are in flight
  RawChunk<TILES> w0, w1;
  auto all = [&](auto&& one) {
    int64_t c = wave;
    if (c < chunks) w0.load(row, c, g, CB);
    for (; c < chunks; c += 2 * FW) {
      const bool two = c + FW < chunks;
      if (two) w1.load(row, c + FW, g, CB);
      one(w0, c);
      if (two) {
        if (c + 2 * FW < chunks) w0.load(row, c + 2 * FW, g, CB);
        one(w1, c + FW);
      }
    }
  };
  if constexpr (RT == 1) {
    Acts<PA, T> x(X, o.M, K, lane);
    all([&](RawChunk<TILES>& w, int64_t c) {
      x.load(c, CB);
      const float s = x.scale();
      float is[VR];
#pragma unroll
      for (int v = 0; v < VR; ++v) is[v] = __is_same(T, _Float16) ? 1.f : 1.f / __shfl(s, 4 * g + v);
      chunk(w, c, is, [&](int b, f16x8 (&a)[1][PA]) { x.fragment(b, s, a); });
    });
  } else {
    const f16x8* A = static_cast<const f16x8*>(X) + lane;
    const int64_t rta = (o.M + 15) / 16;
    const float one[VR] = {};
    all([&](RawChunk<TILES>& w, int64_t c) {
      chunk(w, c, one, [&](int b, f16x8 (&a)[RT][PA]) {
        const f16x8* at = A + min(4 * c + b, CB - 1) * 64;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int p = 0; p < PA; ++p) a[r][p] = at[(p * rta + min<int64_t>(r, rta - 1)) * AB * 64];
      });
    });
  }

  // the waves' sums in a fixed order; a thread takes one column of both
  // projections in one row
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (r) __syncthreads();
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int v = 0; v < VR; ++v) red[wave][t][v][lane] = acc[r][t][v];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < (NT * VR + FW - 1) / FW; ++u) {
      const int item = u * FW + wave;
      if (item >= NT * VR) break;  // wave-uniform
      const int t = item / VR, v = item % VR;
      const int64_t m = RT == 1 ? g + 4 * v : 16 * r + 4 * g + v, n = n0 + 16 * t + i;
      if (m >= o.M || n >= o.N) continue;
      float sg = red[0][t][v][lane], su = red[0][NT + t][v][lane];
#pragma unroll
      for (int w = 1; w < FW; ++w) {
        sg += red[w][t][v][lane];
        su += red[w][NT + t][v][lane];
      }
      const float f = RT == 1 ? 1.f : inv[m];
      finish<T>(o, m, n, f * sg, f * su);
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows: codes of both projections unpacked into operand fragments, 32 rows
// of the gate, the same 32 of up, and so on, so that the four column tiles of a
// wave are two of each at the same columns.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void ffn_codes_kernel(const uint8_t* __restrict__ Wg,
                                                        const uint8_t* __restrict__ Wu, int64_t N,
                                                        int64_t kblocks, int64_t KB,
                                                        f16x8* __restrict__ qfrag,
                                                        float* __restrict__ scale) {
  const int i = threadIdx.x & 15;
  const int64_t kb = static_cast<int64_t>(blockIdx.y) * 16 + (threadIdx.x >> 4);
  if (kb >= KB) return;
  const int64_t rt = blockIdx.x, n = rt / 4 * 32 + (rt & 1) * 16 + i;
  uint32_t d = 0, qs[4] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
  if (n < N && kb < kblocks) load_block_any(rt & 2 ? Wu : Wg, n * kblocks + kb, d, qs);
  const int64_t f = rt * KB + kb;
#pragma unroll
  for (int g = 0; g < 4; ++g) qfrag[f * 64 + i + 16 * g] = codes8(qs[g]);
  scale[f * 16 + i] = half_bits_to_float(d);
}

template <typename S, int PA, int KS, typename T>
__global__ __launch_bounds__(S::THREADS) __attribute__((amdgpu_waves_per_eu(2, 2)))
void ffn_gemm_kernel(const f16x8* __restrict__ A, const f16x8* __restrict__ Q,
                     const float* __restrict__ scale, const float* __restrict__ inv, int64_t cols,
                     int64_t CB, int tiles_m, Out o) {
  f32x4 acc[S::FM][S::FN];
  int64_t m0, c0;
  scaled_tile<S, PA, KS>(A, Q, scale, o.M, cols, CB, tiles_m, acc, m0, c0);
  if (c0 >= cols) return;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < S::FM; ++i) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t m = m0 + 16 * i + 4 * (lane >> 4) + v;
      if (m >= o.M) continue;
      const float f = inv[m];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t n = c0 / 2 + 16 * j + (lane & 15);
        if (n < o.N) finish<T>(o, m, n, f * acc[i][j][v], f * acc[i][2 + j][v]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------
// Per row, the power of two that brings dg and du into binary16: their
// magnitudes are below 1.13 max|dh| max|z| (act' of either activation is below
// 1.13, |act(g)| at most |g|).  A bound that is too high by 2^b only costs values
// 2^-(39 - b) times it.
template <typename T>
__global__ __launch_bounds__(256) void ffn_bound_kernel(const T* __restrict__ z,
                                                        const T* __restrict__ dh,
                                                        float* __restrict__ inv, int64_t N) {
  __shared__ float red[4][2];
  const int64_t m = blockIdx.x;
  float tz = 0.f, td = 0.f;
  const T *zr = z + m * 2 * N, *dr = dh + m * N;
  auto top = [](const T* p, int64_t n, float& t) {
    constexpr int V = 16 / sizeof(T);
    for (int64_t c = V * static_cast<int64_t>(threadIdx.x); c < n; c += V * 256) {
      if (c + V <= n) {
        float v[V];
        load_any_f32<V>(p + c, v);
#pragma unroll
        for (int e = 0; e < V; ++e) t = fmaxf(t, fabsf(v[e]));
      } else {
        for (int64_t e = c; e < n; ++e) t = fmaxf(t, fabsf(to_f32(p[e])));
      }
    }
  };
  top(zr, 2 * N, tz);
  top(dr, N, td);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    tz = fmaxf(tz, __shfl_xor(tz, d));
    td = fmaxf(td, __shfl_xor(td, d));
  }
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6][0] = tz;
    red[threadIdx.x >> 6][1] = td;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  tz = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
  td = fmaxf(fmaxf(red[0][1], red[1][1]), fmaxf(red[2][1], red[3][1]));
  float is = 1.f;
  if (tz > 0.f && td > 0.f && tz < __builtin_inff() && td < __builtin_inff()) {
    int ez, ed;
    frexpf(tz, &ez);
    frexpf(td, &ed);  // the bound lies below 2^(ez + ed + 1)
    is = ldexpf(1.f, max(-126, min(126, ez + ed + 1 - 15)));
  }
  inv[m] = is;
}

// dg and du as operand fragments (NATURAL over the columns), and where the
// caller wants them in dz.  A wave takes 16 rows of 32 columns.
template <int ACT, int PARTS, typename T>
__global__ __launch_bounds__(256) void ffn_dz_kernel(const T* z, const T* __restrict__ dh, T* dz,
                                                     const float* __restrict__ inv,
                                                     f16x8* __restrict__ fg, f16x8* __restrict__ fu,
                                                     int64_t M, int64_t N, int64_t CB) {
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int64_t nb = static_cast<int64_t>(blockIdx.y) * 4 + (threadIdx.x >> 6);
  if (nb >= CB) return;
  const int64_t rt = blockIdx.x, m = rt * 16 + i, n = nb * 32 + 8 * g;
  float zg[8], zu[8], d[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) zg[e] = zu[e] = d[e] = 0.f;
  const bool live = m < M && n < N;
  if (live) {
    const T *pz = z + m * 2 * N + n, *pd = dh + m * N + n;
    if (n + 8 <= N) {
      load_any_f32<8>(pz, zg);
      load_any_f32<8>(pz + N, zu);
      load_any_f32<8>(pd, d);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < N) {
          zg[e] = to_f32(pz[e]);
          zu[e] = to_f32(pz[N + e]);
          d[e] = to_f32(pd[e]);
        }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float slope;
    const float a = activate<ACT, sizeof(T) == 4, true>(zg[e], slope);
    zg[e] = d[e] * zu[e] * slope;
    zu[e] = d[e] * a;
  }
  if (dz && live) {
    T* p = dz + m * 2 * N + n;
    if (n + 8 <= N) {
      store_any_f32<8>(p, zg);
      store_any_f32<8>(p + N, zu);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < N) {
          p[e] = from_f32<T>(zg[e]);
          p[N + e] = from_f32<T>(zu[e]);
        }
    }
  }
  if (!fg) return;
  const float s = m < M ? 1.f / inv[m] : 1.f;
  const int64_t at = (rt * CB + nb) * 64 + lane, part = static_cast<int64_t>(gridDim.x) * CB * 64;
  auto put = [&](f16x8* f, const float (&v)[8]) {
    f16x8 hi, lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = v[e] * s;
      hi[e] = static_cast<_Float16>(x);
      if constexpr (PARTS == 2) lo[e] = static_cast<_Float16>(x - static_cast<float>(hi[e]));
    }
    f[at] = hi;
    if constexpr (PARTS == 2) f[part + at] = lo;
  };
  put(fg, zg);
  put(fu, zu);
}

struct FfnPlan {
  bool few;
  int rt, nt, pa;
  Tile tile;
  int64_t cols;  // rows of both projections, padded
  size_t x, inv, codes, scale, total;
};

FfnPlan ffn_plan(int type, int64_t M, int64_t N, int64_t K, int cus) {
  FfnPlan p = {};
  Carver c;
  p.pa = type == TYPE_F32 ? 2 : 1;
  p.few = M <= FEW_ROWS;
  p.rt = static_cast<int>((M + 15) / 16);
  if (p.few) {
    // the tile that keeps the busiest CU's columns fewest; a workgroup's x is
    // read whatever its columns, so the wider of equals
    int64_t best = INT64_MAX;
    for (int nt = p.rt == 1 || p.rt > 3 ? 2 : 3; nt >= 1; --nt) {
      const int64_t groups = (N + 16 * nt - 1) / (16 * nt);
      const int64_t most = (groups + cus - 1) / cus * nt;
      if (most < best) {
        best = most;
        p.nt = nt;
      }
    }
    if (p.rt == 1) return p;
  }
  p.x = c.take(static_cast<size_t>(frag_elems(M, K)) * 16 * p.pa);
  p.inv = c.take(static_cast<size_t>(M) * 4);
  if (!p.few) {
    p.cols = (N + 31) / 32 * 64;
    double best = 1e30;
    for (Tile t : {Tile::T256x256, Tile::T128x128}) {
      const double us = tile_time_us(t, M, p.cols, K, p.pa, 1, cus);
      if (us < best) {
        best = us;
        p.tile = t;
      }
    }
    p.codes = c.take(static_cast<size_t>(frag_elems(p.cols, K)) * 16);
    p.scale = c.take(static_cast<size_t>(p.cols) * blocks32(K) * 4);
  }
  p.total = c.at;
  return p;
}

struct GradPlan {
  int pa, splits;  // of each projection
  int64_t rows;    // of a projection, padded
  size_t inv, fg, fu, part, total;
};

GradPlan grad_plan(int type, int64_t M, int64_t N, int64_t K, int cus) {
  GradPlan p = {};
  Carver c;
  p.pa = type == TYPE_F32 ? 2 : 1;
  p.rows = (N + 63) / 64 * 64;
  p.splits = (transposed_plan(M, 2 * p.rows, K, p.pa + 1, cus).splits + 1) / 2;
  p.inv = c.take(static_cast<size_t>(M) * 4);
  p.fg = c.take(static_cast<size_t>(frag_elems(M, p.rows)) * 16 * p.pa);
  p.fu = c.take(static_cast<size_t>(frag_elems(M, p.rows)) * 16 * p.pa);
  p.part = c.take(static_cast<size_t>(2 * p.splits) * M * K * 4);
  p.total = c.at;
  return p;
}

using std::integral_constant;
template <int V>
using Int = integral_constant<int, V>;


#define Q4_TRY(expr)                          \
  do {                                        \
    const hipError_t e_ = (expr);             \
    if (e_ != hipSuccess) return e_;          \
  } while (0)

}  // namespace

size_t ffn_workspace_bytes(int type, int64_t M, int64_t N, int64_t K, int cus) {
  return ffn_plan(type, M, N, K, cus).total;
}

hipError_t launch_ffn(const FfnArgs& a, int cus) {
  const FfnPlan p = ffn_plan(a.type, a.M, a.N, a.K, cus);
  char* base = static_cast<char*>(a.ws);
  f16x8* xa = reinterpret_cast<f16x8*>(base + p.x);
  float* inv = reinterpret_cast<float*>(base + p.inv);
  const Out o = {a.r, a.h, a.z, a.M, a.N, a.act};
  if (!p.few || p.rt > 1) Q4_TRY(prep_rows(a.x, a.type, Order::NIBBLE, xa, inv, a.M, a.K, a.stream));
  if (p.few) {
    with_type(a.type, [&](auto type) {
      using T = decltype(type);
      constexpr int PA = sizeof(T) == 4 ? 2 : 1;
      auto launch = [&](auto rt, auto nt, auto vr) {
        constexpr int RT = decltype(rt)::value, NT = decltype(nt)::value, VR = decltype(vr)::value;
        const unsigned grid = static_cast<unsigned>((a.N + 16 * NT - 1) / (16 * NT));
        hipLaunchKernelGGL((ffn_few_kernel<RT, PA, NT, VR, T>), dim3(grid), dim3(64 * FW), 0, a.stream,
                           a.gate, a.up, RT == 1 ? a.x : static_cast<const void*>(xa), inv, a.K, o);
      };
      auto cols = [&](auto rt, auto vr) {
        if (p.nt == 1) launch(rt, Int<1>{}, vr);
        else if (p.nt == 2) launch(rt, Int<2>{}, vr);
        else launch(rt, Int<(decltype(rt)::value == 1 || decltype(rt)::value > 3) ? 2 : 3>{}, vr);
      };
      if (a.M <= 4) cols(Int<1>{}, Int<1>{});
      else if (a.M <= 8) cols(Int<1>{}, Int<2>{});
      else if (a.M <= 16) cols(Int<1>{}, Int<4>{});
      else if (a.M <= 32) cols(Int<2>{}, Int<4>{});
      else if (a.M <= 48) cols(Int<3>{}, Int<4>{});
      else cols(Int<4>{}, Int<4>{});
    });
    return hipGetLastError();
  }
  f16x8* codes = reinterpret_cast<f16x8*>(base + p.codes);
  float* scale = reinterpret_cast<float*>(base + p.scale);
  const int64_t KB = blocks32(a.K);
  hipLaunchKernelGGL(ffn_codes_kernel,
                     dim3(static_cast<unsigned>(p.cols / 16), static_cast<unsigned>((KB + 15) / 16)),
                     dim3(256), 0, a.stream, a.gate, a.up, a.N, a.K / 32, KB, codes, scale);
  Q4_TRY(hipGetLastError());
  const TileDim d = tile_dim(p.tile);
  const int tm = static_cast<int>((a.M + d.m - 1) / d.m), tn = static_cast<int>((p.cols + d.n - 1) / d.n);
  with_type(a.type, [&](auto type) {
    using T = decltype(type);
    constexpr int PA = sizeof(T) == 4 ? 2 : 1, KS = PA == 1 ? 2 : 1;
    auto go = [&](auto shape) {
      using S = decltype(shape);
      hipLaunchKernelGGL((ffn_gemm_kernel<S, PA, KS, T>),
                         dim3(static_cast<unsigned>(static_cast<int64_t>(tm) * tn)), dim3(S::THREADS), 0,
                         a.stream, xa, codes, scale, inv, p.cols, KB, tm, o);
    };
    if (p.tile == Tile::T256x256) go(S256{});
    else go(S128{});
  });
  return hipGetLastError();
}

size_t ffn_grad_workspace_bytes(int type, int64_t M, int64_t N, int64_t K, int cus) {
  return grad_plan(type, M, N, K, cus).total;
}

hipError_t launch_ffn_grad(const FfnGradArgs& a, int cus) {
  const GradPlan p = grad_plan(a.type, a.M, a.N, a.K, cus);
  char* base = static_cast<char*>(a.ws);
  f16x8* fg = a.dx ? reinterpret_cast<f16x8*>(base + p.fg) : nullptr;
  f16x8* fu = a.dx ? reinterpret_cast<f16x8*>(base + p.fu) : nullptr;
  float* inv = reinterpret_cast<float*>(base + p.inv);
  const int64_t CB = p.rows / 32;
  with_type(a.type, [&](auto type) {
    using T = decltype(type);
    constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
    const T *z = static_cast<const T*>(a.z), *dh = static_cast<const T*>(a.dh);
    if (a.dx)
      hipLaunchKernelGGL(ffn_bound_kernel<T>, dim3(static_cast<unsigned>(a.M)), dim3(256), 0, a.stream, z,
                         dh, inv, a.N);
    const dim3 grid(static_cast<unsigned>((a.M + 15) / 16), static_cast<unsigned>((CB + 3) / 4));
    auto* kernel = a.act == ACT_SILU ? ffn_dz_kernel<ACT_SILU, PARTS, T> : ffn_dz_kernel<ACT_GELU, PARTS, T>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, a.stream, z, dh,
                       static_cast<T*>(a.dz), inv, fg, fu, a.M, a.N, CB);
  });
  Q4_TRY(hipGetLastError());
  if (!a.dx) return hipSuccess;
  TransposedGemm g = {};
  g.g = fg;
  g.g2 = fu;
  g.pa = p.pa;
  g.pb = 2;
  g.type = a.type;
  g.w = a.gate;
  g.w2 = a.up;
  g.N = a.N;
  g.M = a.M;
  g.K = a.K;
  g.CB = CB;
  g.splits = p.splits;
  g.part = reinterpret_cast<float*>(base + p.part);
  Q4_TRY(launch_gemm_transposed(g, a.stream));
  return launch_fold(g.part, 2 * p.splits, inv, a.dx, a.type, a.M, a.K, a.stream);
}

}  // namespace q4
