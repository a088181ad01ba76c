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
#include "q4_wave.h"

namespace q4 {
namespace {

template <int V>
using Int = std::integral_constant<int, V>;

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
// each projection; its waves share them and take every nw-th chunk of 256 k,
// and their sums are added in LDS at the end: most of a matrix's bytes are
// requested at once, whatever its height.
//
// Lane (i, g) loads the block pair g of the chunk of weight row i: 36 bytes.
// 4 x 4 transpositions over the lane groups give it dword g of each of the
// eight blocks, the operand of the exact codes q - 8.
// ---------------------------------------------------------------------------
constexpr int FW = 8;  // waves at most
// Rows of x this route takes: four tiles of 16, whose sums fill the registers.  Above,
// unpacking the codes of both projections costs 35 us (2 x 9216 x 3072) whatever the
// number of rows.  This route and the unpacked one, weights from memory, us:
// 2 x 9216 x 3072 float32 32 rows 31.4 and 91.0, 64 41.3 and 95.1; bfloat16 64 33.8
// and 84.0; 2 x 5120 x 1280 float32 64 18.9 and 50.3.  So 65 rows (94.7, 83.0 and 49.8)
// take more than two calls of half of them would, up to about 128.
constexpr int64_t FEW_ROWS = 64;

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

// The power of two that brings `top` to [2^14, 2^15) (at most 2^126: for zero and
// the smallest numbers), and its inverse.
struct PowerOfTwo {
  float s, inv;
  __device__ __forceinline__ explicit PowerOfTwo(float top) {
    const int e = min(268 - static_cast<int>(__float_as_uint(top) >> 23), 253);
    s = __uint_as_float(static_cast<uint32_t>(e) << 23);
    inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  }
};

// The largest over the four lane groups, in all of them.
__device__ __forceinline__ float groups_max(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// The largest over LANES (32 or 64) neighbours, in all of them.
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (LANES == 64) return wave64_max(v);
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  v = fmaxf(v, dpp_f32<0x140>(v));
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// This lane's block pairs of a chunk, one of each of the workgroup's row tiles.
// ODD: K is an odd multiple of 32; rows start at any even address and end with
// half a pair, the other half of which may lie outside the matrix.
typedef uint32_t u32x4_at __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_at __attribute__((aligned(2)));
template <int TILES, bool ODD>
struct RawChunk {
  uint32_t w[TILES][9];
  // row: this lane's pair of each tile; half: it is half a pair
  __device__ __forceinline__ void load_pair(const uint8_t* const (&row)[TILES], bool half) {
    if (ODD && half) {
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(row[t]);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[t][e] = h[2 * e] | static_cast<uint32_t>(h[2 * e + 1]) << 16;
        w[t][4] = h[8];  // the second block's scale: 0
#pragma unroll
        for (int e = 5; e < 9; ++e) w[t][e] = 0;
      }
      return;
    }
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const u32x4 a = *reinterpret_cast<const u32x4_at*>(row[t]);
      const u32x4 b = *reinterpret_cast<const u32x4_at*>(row[t] + 16);
      w[t][8] = *reinterpret_cast<const u32_at*>(row[t] + 32);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[t][e] = a[e];
        w[t][4 + e] = b[e];
      }
    }
  }
  __device__ __forceinline__ void load(const uint8_t* const (&row)[TILES], int64_t c, int g, int64_t K) {
    const int64_t pairs = (K + 32) / 64, p = min(4 * c + g, pairs - 1);
    const uint8_t* at[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) at[t] = row[t] + p * PAIR_BYTES;
    load_pair(at, ODD && p == pairs - 1);
  }
};

// Up to 16 rows of x: a wave reads its chunk of each of them once, scales the
// row's XB blocks by a power of two into binary16 (float16 as it is), splits
// them and puts them into LDS in operand order, so the split costs by the rows
// there are.  Row a of the operand is row (a >> 2) + 4 (a & 3) of x: up to 4 VR
// rows lie in the first VR of a result's registers.
template <int PA, int VR, typename T>
struct Acts {
  static constexpr int ROWS = 4 * VR;
  static constexpr int XB = VR == 4 ? 4 : 8;      // blocks staged at a time
  static constexpr int LANES = 8 * XB;            // per row
  static constexpr int LOADS = ROWS * LANES / 64; // per stage
  static constexpr int BLOCK = ROWS * 64 + 64;    // bytes; the padding spreads a store over the banks
  static constexpr int BYTES = PA * XB * BLOCK + ROWS * 4;  // of a wave
  typedef T vec __attribute__((ext_vector_type(4)));
  vec v[LOADS];

  // stage s: blocks XB s .. of the operand's blocks
  __device__ __forceinline__ void load(const T* x, int64_t M, int64_t K, int64_t s, int lane) {
    const int64_t k = s * XB * 32 + 4 * (lane % LANES);
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int r = u * (64 / LANES) + lane / LANES;
      v[u] = vec{};
      if (LANES == 64 ? u < M : u * (64 / LANES) < M)  // uniform
        if (k < K) v[u] = *reinterpret_cast<const vec*>(x + min<int64_t>(r, M - 1) * K + k);
    }
  }
  __device__ __forceinline__ void store(char* lds, int64_t M, int lane) const {
    const int l = lane % LANES;
    char* to = lds + (l >> 3) * BLOCK + (l & 3) * 16 + (l & 4) * 2;
    float* scales = reinterpret_cast<float*>(lds + PA * XB * BLOCK);
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      if (!(LANES == 64 ? u < M : u * (64 / LANES) < M)) continue;  // uniform
      const int r = u * (64 / LANES) + lane / LANES;
      float f[4], s = 1.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = to_f32(static_cast<T>(v[u][e]));
      if constexpr (!__is_same(T, _Float16)) {
        const PowerOfTwo p(
            lanes_max<LANES>(fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])))));
        s = p.s;
        if (l == 0) scales[r] = p.inv;
      }
      typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
      f16x4 hi, lo;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float y = f[e] * s;
        hi[e] = static_cast<_Float16>(y);
        if constexpr (PA == 2) lo[e] = static_cast<_Float16>(y - static_cast<float>(hi[e]));
      }
      *reinterpret_cast<f16x4*>(to + r * 64) = hi;
      if constexpr (PA == 2) *reinterpret_cast<f16x4*>(to + XB * BLOCK + r * 64) = lo;
    }
  }
  static __device__ __forceinline__ f16x8 fragment(const char* lds, int b, int part, int64_t M, int lane) {
    const int a = lane & 15, r = static_cast<int>(min<int64_t>((a >> 2) + 4 * (a & 3), M - 1));
    return *reinterpret_cast<const f16x8*>(lds + (part * XB + b) * BLOCK + r * 64 + (lane >> 4) * 16);
  }
  // of the row in register v of a result
  static __device__ __forceinline__ float inverse(const char* lds, int v, int64_t M, int lane) {
    if constexpr (__is_same(T, _Float16)) return 1.f;
    return reinterpret_cast<const float*>(lds + PA * XB * BLOCK)[min<int64_t>((lane >> 4) + 4 * v, M - 1)];
  }
};

// Measured, 9216 x 3072: 32 rows float32 27.6 us with prep_rows, 38 rows 32.4 (of
// them 6.6), 64 rows bfloat16 31; bound by the latency of x's operands, which
// every workgroup reads from the L2 (340 MB in all at 38 rows), beside the 32 MB
// of weights.
template <int RT, int PA, int NT, int VR, typename T, bool ODD>
__global__ __launch_bounds__(64 * FW) __attribute__((amdgpu_waves_per_eu(RT > 1 || NT > 1 ? 2 : VR > 2 ? 3 : 4)))
void ffn_few_kernel(const uint8_t* __restrict__ Wg, const uint8_t* __restrict__ Wu,
                    const void* __restrict__ X, const float* __restrict__ inv, int64_t K, Out o) {
  constexpr int TILES = 2 * NT;  // gate's, then up's
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = static_cast<int>(blockDim.x) >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int64_t pairs = (K + 32) / 64, chunks = (pairs + 3) / 4, AB = 2 * pairs, M = o.M;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NT);
  const uint8_t* row[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t)
    row[t] = (t < NT ? Wg : Wu) + min(n0 + 16 * (t % NT) + i, o.N - 1) * (K / 32) * BLOCK_BYTES;

  f32x4 acc[RT][TILES];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TILES; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  // codes in place of the loaded bytes: q[t][o][p] is this lane's dword of block
  // 2 p + o of the chunk, dd[t] the two scales of its own pair
  struct Codes {
    uint32_t q[TILES][2][4], dd[TILES];
  };
  auto decode = [&](const RawChunk<TILES, ODD>& w, int64_t c) {
    Codes k;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const uint32_t* r = w.w[t];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        k.q[t][0][e] = shift16(r[e + 1], r[e]);
        k.q[t][1][e] = r[5 + e];
      }
      // pairs past the row have no weight
      k.dd[t] = 4 * c + g < pairs ? __builtin_amdgcn_perm(r[4], r[0], 0x07060100u) : 0u;
      transpose4(k.q[t][0]);
      transpose4(k.q[t][1]);
    }
    return k;
  };
  // blocks B0 .. B0 + NB - 1 of a chunk: step s is block s / TILES against tile
  // s % TILES; a step's scaled sums are taken while the next one's products run.
  // Operands of x are asked for AD - 1 blocks ahead (acts of a block past the
  // chunk are the next chunk's).  The empty volatile asm keeps that order:
  // regrouped, all products first, their results would spill.
  constexpr int AD = RT == 1 || RT * PA > 6 ? 2 : 4;
  f16x8 a[AD][RT][PA];
  auto blocks = [&](const Codes& k, auto b0, auto nb, const float (&is)[VR], auto&& acts) __attribute__((always_inline)) {
    constexpr int B0 = decltype(b0)::value, NB = decltype(nb)::value, STEPS = NB * TILES;
    f32x4 p[2][RT];
    uint32_t d[2][TILES];
    int from = 4 * i;  // of the scale's lane, in bytes
    asm volatile("" : "+v"(from));
    auto products = [&](int s) __attribute__((always_inline)) {
      const int b = B0 + s / TILES, t = s % TILES;
      if (t == 0 && (RT > 1 || s + TILES < STEPS)) acts(b + AD - 1, a[(b + AD - 1) % AD]);
      if ((b & 1) == 0)
        d[(b >> 1) & 1][t] = __builtin_amdgcn_ds_bpermute(from + 64 * (b >> 1), k.dd[t]);
      const f16x8 q = codes8(k.q[t][b & 1][b >> 1]);
#pragma unroll
      for (int r = 0; r < RT; ++r)
        p[s & 1][r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[b % AD][r][0], q, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
      if constexpr (PA == 2) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
          p[s & 1][r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[b % AD][r][1], q, p[s & 1][r], 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) asm volatile("" : "+v"(p[s & 1][r])::"memory");
    };
    if constexpr (RT == 1) acts(B0, a[B0 % AD]);
    products(0);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (s + 1 < STEPS) products(s + 1);
      const int b = B0 + s / TILES, t = s % TILES;
      const uint32_t pair = d[(b >> 1) & 1][t];
      const float ds = half_bits_to_float(b & 1 ? pair >> 16 : pair & 0xFFFFu);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int v = 0; v < VR; ++v)
          acc[r][t][v] = __builtin_fmaf(RT == 1 && !__is_same(T, _Float16) ? ds * is[v] : ds, p[s & 1][r][v], acc[r][t][v]);
        asm volatile("" : "+v"(acc[r][t]));
      }
    }
  };

  // one chunk is multiplied while the next one's bytes are in flight
  RawChunk<TILES, ODD> w;
  int64_t c = wave;
  if constexpr (RT == 1) {
    using X1 = Acts<PA, VR, T>;
    const T* x = static_cast<const T*>(X);
    char* mine = lds + wave * X1::BYTES;
    X1 xa;
    if (c < chunks) {
      xa.load(x, M, K, c * (8 / X1::XB), lane);
      w.load(row, c, g, K);
    }
    for (; c < chunks; c += waves) {
      const int64_t next = c + waves;
      auto stage = [&](int64_t following) {
        xa.store(mine, M, lane);
        issued();
        if (following >= 0) xa.load(x, M, K, following, lane);
      };
      stage(X1::XB == 4 ? 2 * c + 1 : next < chunks ? next : -1);
      const Codes k = decode(w, c);
      if (next < chunks) w.load(row, next, g, K);
      float is[VR];
      auto acts = [&](int b, f16x8 (&a)[1][PA]) {
#pragma unroll
        for (int p = 0; p < PA; ++p) a[0][p] = X1::fragment(mine, b % X1::XB, p, M, lane);
      };
#pragma unroll
      for (int v = 0; v < VR; ++v) is[v] = X1::inverse(mine, v, M, lane);
      blocks(k, Int<0>{}, Int<X1::XB>{}, is, acts);
      if constexpr (X1::XB == 4) {
        issued();
        stage(next < chunks ? 2 * next : -1);
#pragma unroll
        for (int v = 0; v < VR; ++v) is[v] = X1::inverse(mine, v, M, lane);
        blocks(k, Int<4>{}, Int<4>{}, is, acts);
      }
      issued();
    }
  } else {
    const f16x8* A = static_cast<const f16x8*>(X) + lane;
    const int64_t rta = (M + 15) / 16;
    const float none[VR] = {};
    auto acts = [&](int64_t block, f16x8 (&to)[RT][PA]) {
      const f16x8* at = A + min(block, AB - 1) * 64;
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int p = 0; p < PA; ++p) to[r][p] = at[(p * rta + min<int64_t>(r, rta - 1)) * AB * 64];
    };
    if (c < chunks) {
      w.load(row, c, g, K);
#pragma unroll
      for (int b = 0; b < AD - 1; ++b) acts(8 * c + b, a[b]);
    }
    for (; c < chunks; c += waves) {
      const Codes k = decode(w, c);
      if (c + waves < chunks) w.load(row, c + waves, g, K);
      blocks(k, Int<0>{}, Int<8>{}, none, [&](int b, f16x8 (&to)[RT][PA]) {
        acts(b < 8 ? 8 * c + b : 8 * (c + waves) + b - 8, to);
      });
    }
  }

  // the waves' sums in a fixed order; a thread takes one column of both
  // projections in one row
  float(*red)[TILES][VR][64] = reinterpret_cast<float(*)[TILES][VR][64]>(lds);
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int v = 0; v < VR; ++v) red[wave][t][v][lane] = acc[r][t][v];
    __syncthreads();
    for (int item = wave; item < NT * VR; item += waves) {
      const int t = item / VR, v = item % VR;
      const int64_t m = RT == 1 ? g + 4 * v : 16 * r + 4 * g + v, n = n0 + 16 * t + i;
      if (m >= M || n >= o.N) continue;
      float sg = red[0][t][v][lane], su = red[0][NT + t][v][lane];
      for (int u = 1; u < waves; ++u) {
        sg += red[u][t][v][lane];
        su += red[u][NT + t][v][lane];
      }
      const float f = RT == 1 ? 1.f : inv[m];
      finish<T>(o, m, n, f * sg, f * su);
    }
  }
}

// ---------------------------------------------------------------------------
// Up to 16 rows of up to 4096 columns: persistent workgroups, a wave per chunk of
// 256 k, which it keeps of every row of x in registers, as matrix-core operands.
// A pass is eight columns of each projection, gate's in the low half of the
// operand's sixteen; two passes' bytes are in flight.
// ---------------------------------------------------------------------------
// Measured, 9216 x 3072 (32 MB of weights, 6.2 us at the rate of a large copy): one
// row float32 10.3 us, bfloat16 9.4, four 11.6, seven bfloat16 12.5, sixteen
// float32 19; the first version, without persistence, 19.5 and 23.6 for one and
// seven.  Bound by the start (x, then two passes of weights) and by five passes
// of about 1 us, each with a barrier, at 4.5 passes of work.
constexpr int STREAM_K = 4096;

template <int PA, int VR, typename T, bool ODD>
__global__ __launch_bounds__(1024) void ffn_stream_kernel(const uint8_t* __restrict__ Wg,
                                                          const uint8_t* __restrict__ Wu,
                                                          const T* __restrict__ X, int K, int passes,
                                                          Out o) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = static_cast<int>(blockDim.x) >> 6;
  float(*red)[VR][64] = reinterpret_cast<float(*)[VR][64]>(lds);  // [2 waves][VR][64]
  const int i = lane & 15, g = lane >> 4;
  const int pairs = (K + 32) / 64, pair = 4 * wave + g;
  const int64_t rb = static_cast<int64_t>(K / 32) * BLOCK_BYTES;
  const uint8_t* base = (i < 8 ? Wg : Wu) + min(pair, pairs - 1) * PAIR_BYTES;
  RawChunk<1, ODD> w0, w1;
  auto load = [&](int u, RawChunk<1, ODD>& w) {
    w.load_pair({base + min<int64_t>(8 * static_cast<int64_t>(u) + (i & 7), o.N - 1) * rb},
                ODD && pair >= pairs - 1);
  };

  // x, its rows as Acts has them.  Up to four are split once and reach the
  // operands through LDS (one row straight into operands, each of its values
  // split by sixteen lanes: 12.9 us against 10.8); more are read as operands.
  f16x8 a[8][PA];
  float is[VR];
  auto start = [&]() {
    load(blockIdx.x, w0);
    if (static_cast<int>(blockIdx.x + gridDim.x) < passes) load(blockIdx.x + gridDim.x, w1);
  };
  if constexpr (VR <= 2) {
    using X1 = Acts<PA, VR, T>;
    char* mine = lds + 2 * waves * VR * 256 + wave * X1::BYTES;
    X1 x;
    x.load(X, o.M, K, wave, lane);
    start();
    x.store(mine, o.M, lane);
    issued();
#pragma unroll
    for (int b = 0; b < 8; ++b)
#pragma unroll
      for (int p = 0; p < PA; ++p) a[b][p] = X1::fragment(mine, b, p, o.M, lane);
#pragma unroll
    for (int v = 0; v < VR; ++v) is[v] = X1::inverse(mine, v, o.M, lane);
  } else {
    typedef T vec __attribute__((ext_vector_type(4)));
    vec v[8][2];
    const int row = (i >> 2) + 4 * (i & 3);
    const T* x = X + static_cast<int64_t>(min<int64_t>(row, o.M - 1)) * K + 4 * g;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const int k = 256 * wave + 32 * b;
      const T* p = x + min(k, K - 32);
      v[b][0] = *reinterpret_cast<const vec*>(p);
      v[b][1] = *reinterpret_cast<const vec*>(p + 16);
      if (k >= K) v[b][0] = v[b][1] = vec{};
    }
    start();
    float s = 1.f, back = 1.f;
    if constexpr (!__is_same(T, _Float16)) {
      float top = 0.f;
#pragma unroll
      for (int b = 0; b < 8; ++b)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(to_f32(static_cast<T>(v[b][e >> 2][e & 3]))));
      const PowerOfTwo p(groups_max(top));
      s = p.s;
      back = p.inv;
    }
#pragma unroll
    for (int b = 0; b < 8; ++b) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = to_f32(static_cast<T>(v[b][e >> 2][e & 3])) * s;
        a[b][0][e] = static_cast<_Float16>(y);
        if constexpr (PA == 2) a[b][1][e] = static_cast<_Float16>(y - static_cast<float>(a[b][0][e]));
      }
    }
#pragma unroll
    for (int v = 0; v < VR; ++v) is[v] = __is_same(T, _Float16) ? 1.f : __shfl(back, 4 * g + v);
  }

  auto compute = [&](const RawChunk<1, ODD>& w, f32x4& acc) {
    uint32_t q[2][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[0][e] = shift16(w.w[0][e + 1], w.w[0][e]);
      q[1][e] = w.w[0][5 + e];
    }
    const uint32_t dd = pair < pairs ? __builtin_amdgcn_perm(w.w[0][4], w.w[0][0], 0x07060100u) : 0u;
    transpose4(q[0]);
    transpose4(q[1]);
    uint32_t d[4];
    int from = 4 * i;
    asm volatile("" : "+v"(from));
#pragma unroll
    for (int p = 0; p < 4; ++p) d[p] = __builtin_amdgcn_ds_bpermute(from + 64 * p, dd);
    f32x4 t[2];
    auto products = [&](int b) {
      const f16x8 c = codes8(q[b & 1][b >> 1]);
      t[b & 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[b][0], c, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
      if constexpr (PA == 2) t[b & 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[b][1], c, t[b & 1], 0, 0, 0);
      asm volatile("" : "+v"(t[b & 1])::"memory");
    };
    acc = f32x4{0.f, 0.f, 0.f, 0.f};
    products(0);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      if (b + 1 < 8) products(b + 1);
      const float s = half_bits_to_float(b & 1 ? d[b >> 1] >> 16 : d[b >> 1] & 0xFFFFu);
#pragma unroll
      for (int v = 0; v < VR; ++v) acc[v] = __builtin_fmaf(s, t[b & 1][v], acc[v]);
      asm volatile("" : "+v"(acc));
    }
  };
  // the waves' sums in a fixed order, by the waves in turn
  int turn = wave;
  auto put = [&](int u, const f32x4& acc, int q) {
#pragma unroll
    for (int v = 0; v < VR; ++v) red[q * waves + wave][v][lane] = acc[v] * is[v];
    __syncthreads();
#pragma unroll
    for (int v = 0; v < VR; ++v) {
      if (turn != v % waves) continue;  // (wave-uniform)
      const int64_t m = g + 4 * v, n = 8 * static_cast<int64_t>(u) + (i & 7);
      float s = 0.f;
#pragma unroll 1
      for (int k = 0; k < waves; k += 4) {  // four in flight
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = k + e < waves ? red[q * waves + k + e][v][lane] : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) s += p[e];
      }
      const float up = dpp_f32<0x128>(s);  // row_ror:8
      if (i < 8 && m < o.M && n < o.N) finish<T>(o, m, n, s, up);
    }
    if (VR < waves) turn = turn + VR < waves ? turn + VR : turn + VR - waves;
  };
  const int step = gridDim.x;
  for (int u = blockIdx.x; u < passes; u += 2 * step) {
    f32x4 acc;
    compute(w0, acc);
    if (u + 2 * step < passes) load(u + 2 * step, w0);
    __builtin_amdgcn_sched_barrier(0);
    put(u, acc, 0);
    if (u + step >= passes) break;
    compute(w1, acc);
    if (u + 3 * step < passes) load(u + 3 * step, w1);
    __builtin_amdgcn_sched_barrier(0);
    put(u + step, acc, 1);
  }
}

// Bytes of LDS per wave.
template <int RT, int PA, int NT, int VR, typename T>
constexpr int few_lds() {
  const int sums = 2 * NT * VR * 256;
  return RT == 1 && Acts<PA, VR, T>::BYTES > sums ? Acts<PA, VR, T>::BYTES : sums;
}

// ---------------------------------------------------------------------------
// Many rows: codes of both projections unpacked into operand fragments, 32 rows
// of the gate, the same 32 of up, and so on, so that the four column tiles of a
// wave are two of each at the same columns.
// ---------------------------------------------------------------------------
// Measured: 2 x 9216 x 3072 34.6 us (32 MB read, 121 written: 4.4 TB/s), bound by
// the writes.
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

// Measured: 1500 x 2 x 9216 x 3072 bfloat16, with g and u kept, 237 to 248 us in a
// trace from a cold start; the call with prep_rows and ffn_codes 253.  A block's
// scale costs as many vector cycles (four FMAs) as its product costs the matrix
// cores, and the two hardly overlap: that call without three of the four FMAs took
// 210 us, with the loads always of one block 244, against 253.  432 tiles on 256
// CUs are two rounds, 84 % full.
template <typename S, int PA, typename T>
__global__ __launch_bounds__(S::THREADS) __attribute__((amdgpu_waves_per_eu(2, 2)))
void ffn_gemm_kernel(const f16x8* __restrict__ A, const f16x8* __restrict__ Q,
                     const float* __restrict__ scale, const float* __restrict__ inv, int64_t cols,
                     int64_t CB, int tiles_m, Out o) {
  f32x4 acc[S::FM][S::FN];
  int64_t m0, c0;
  scaled_tile<S, PA>(A, Q, scale, o.M, cols, CB, tiles_m, acc, m0, c0);
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
// Measured: 76 rows of 9216 float32 4.9 us, 1500 of 5120 bfloat16 9.7.
constexpr int BOUND_WAVES = 16;
template <typename T>
__global__ __launch_bounds__(64 * BOUND_WAVES) void ffn_bound_kernel(const T* __restrict__ z,
                                                        const T* __restrict__ dh,
                                                        float* __restrict__ inv, int64_t N) {
  __shared__ float red[BOUND_WAVES][2];
  const int64_t m = blockIdx.x;
  float tz = 0.f, td = 0.f;
  const T *zr = z + m * 2 * N, *dr = dh + m * N;
  auto top = [](const T* p, int64_t n, float& t) {
    constexpr int V = 16 / sizeof(T);
    for (int64_t c = V * static_cast<int64_t>(threadIdx.x); c < n; c += V * 64 * BOUND_WAVES) {
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
  tz = wave64_max(tz);
  td = wave64_max(td);
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6][0] = tz;
    red[threadIdx.x >> 6][1] = td;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < BOUND_WAVES; ++w) {
    tz = fmaxf(tz, red[w][0]);
    td = fmaxf(td, red[w][1]);
  }
  float is = 1.f;
  if (tz > 0.f && td > 0.f && tz < __builtin_inff() && td < __builtin_inff()) {
    int ez, ed;
    frexpf(tz, &ez);
    frexpf(td, &ed);  // the bound lies below 2^(ez + ed + 1)
    is = ldexpf(1.f, max(-126, min(126, ez + ed + 1 - 15)));
  }
  inv[m] = is;
}

// dg and du as operand fragments (NATURAL over the columns) of two parts whatever
// the type, and where the caller wants them in dz: one part, 11 bits, would be
// below bfloat16's own rounding for a term but not for a sum whose terms cancel
// (random terms: dx 8.6e-4 from the exact one rounded, two parts 3e-5).  A wave
// takes 16 rows of 32 columns.
// Measured: 76 x 9216 float32 7.3 us, 1500 x 5120 bfloat16 18 (107 MB: 5.8 TB/s).
template <int ACT, typename T>
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
      lo[e] = static_cast<_Float16>(x - static_cast<float>(hi[e]));
    }
    f[at] = hi;
    f[part + at] = lo;
  };
  put(fg, zg);
  put(fu, zu);
}

struct FfnPlan {
  bool stream, few;
  int rt, nt, pa, waves, grid;
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
  // (five to eight rows of float32: the staged rows of sixteen waves are past the
  // LDS)
  if (p.rt == 1 && K <= (p.pa == 2 && M > 4 && M <= 8 ? STREAM_K - 256 : STREAM_K)) {
    p.stream = true;
    p.waves = static_cast<int>((K + 255) / 256);
    // a workgroup per CU, more of fewer waves
    p.grid = static_cast<int>(std::min<int64_t>((N + 7) / 8, static_cast<int64_t>(cus) * std::max(1, 8 / p.waves)));
    return p;
  }
  if (p.few) {
    // Up to 16 rows here have long rows (more than STREAM_K columns): eight waves.
    // Nine to sixteen take the wider tile once a CU has more than one of the narrow,
    // which then read x again (16 float32 rows, narrow and wide, us: 9216 x 5120 54.3
    // and 46.2, 4112 x 8192 57.2 and 38.6, but 4096 x 8192 32.0 and 38.4; 8 rows 30.9
    // and 35.8, 31.5 and 29.3, 21.4 and 29.3; one row 19.4 and 27.4, 19.5 and 22.0).
    // Above, four waves of one tile, whose registers let two workgroups share a CU
    // with four blocks of x in flight (38 rows of 9216 x 3072: 32.4 us; six waves
    // 41.7, two tiles 39.8, two blocks in flight 38.5 and 34.6).
    const int64_t chunks = (K + 255) / 256;
    p.nt = p.rt == 1 && M > 8 && (N + 15) / 16 > cus ? 2 : 1;
    p.waves = static_cast<int>(std::min<int64_t>(chunks, p.rt == 1 ? FW : 4));
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

constexpr int GRAD_UNITS = 3;  // products of a pair of fragments: two parts of each
struct GradPlan {
  int rt, splits;  // splits of each projection
  int64_t rows;    // of a projection, padded
  size_t inv, fg, fu, part, total;
};

GradPlan grad_plan(int64_t M, int64_t N, int64_t K, int cus) {
  GradPlan p = {};
  Carver c;
  p.rows = (N + 63) / 64 * 64;
  // tiles of as many rows as leave the fewest products, and of equals the tallest
  // (76 rows: two of 48, not of 64)
  int64_t least = INT64_MAX;
  for (int rt = 4; rt >= 1; --rt) {
    const int64_t clk = (M + 16 * rt - 1) / (16 * rt) * std::max(8 * rt * GRAD_UNITS * 16, 800);
    if (clk < least) {
      least = clk;
      p.rt = rt;
    }
  }
  p.splits = (transposed_plan(M, 2 * p.rows, K, GRAD_UNITS, cus, p.rt).splits + 1) / 2;
  p.inv = c.take(static_cast<size_t>(M) * 4);
  p.fg = c.take(static_cast<size_t>(frag_elems(M, p.rows)) * 16 * 2);
  p.fu = c.take(static_cast<size_t>(frag_elems(M, p.rows)) * 16 * 2);
  p.part = c.take(static_cast<size_t>(2 * p.splits) * M * K * 4);
  p.total = c.at;
  return p;
}


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
  if (p.stream) {
    with_type(a.type, [&](auto type) {
      using T = decltype(type);
      constexpr int PA = sizeof(T) == 4 ? 2 : 1;
      auto go = [&](auto vr) {
        constexpr int VR = decltype(vr)::value;
        auto* kernel = a.K % 64 == 0 ? ffn_stream_kernel<PA, VR, T, false> : ffn_stream_kernel<PA, VR, T, true>;
        const unsigned lds = p.waves * (2 * VR * 256 + (VR <= 2 ? Acts<PA, VR, T>::BYTES : 0));
        hipLaunchKernelGGL(kernel, dim3(p.grid), dim3(64 * p.waves), lds, a.stream, a.gate, a.up,
                           static_cast<const T*>(a.x), static_cast<int>(a.K),
                           static_cast<int>((a.N + 7) / 8), o);
      };
      if (a.M <= 4) go(Int<1>{});
      else if (a.M <= 8) go(Int<2>{});
      else go(Int<4>{});
    });
    return hipGetLastError();
  }
  if (p.few) {
    with_type(a.type, [&](auto type) {
      using T = decltype(type);
      constexpr int PA = sizeof(T) == 4 ? 2 : 1;
      auto launch = [&](auto rt, auto nt, auto vr) {
        constexpr int RT = decltype(rt)::value, NT = decltype(nt)::value, VR = decltype(vr)::value;
        const unsigned grid = static_cast<unsigned>((a.N + 16 * NT - 1) / (16 * NT));
        auto* kernel = a.K % 64 == 0 ? ffn_few_kernel<RT, PA, NT, VR, T, false> : ffn_few_kernel<RT, PA, NT, VR, T, true>;
        const unsigned lds = p.waves * few_lds<RT, PA, NT, VR, T>();
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * p.waves), lds, a.stream, a.gate, a.up,
                           RT == 1 ? a.x : static_cast<const void*>(xa), inv, a.K, o);
      };
      const Int<1> one;
      const Int<4> four;
      if (a.M <= 4) launch(one, one, one);
      else if (a.M <= 8) launch(one, one, Int<2>{});
      else if (a.M <= 16 && p.nt == 1) launch(one, one, four);
      else if (a.M <= 16) launch(one, Int<2>{}, four);
      else if (a.M <= 32) launch(Int<2>{}, one, four);
      else if (a.M <= 48) launch(Int<3>{}, one, four);
      else launch(four, one, four);
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
    constexpr int PA = sizeof(T) == 4 ? 2 : 1;
    auto go = [&](auto shape) {
      using S = decltype(shape);
      hipLaunchKernelGGL((ffn_gemm_kernel<S, PA, T>),
                         dim3(static_cast<unsigned>(static_cast<int64_t>(tm) * tn)), dim3(S::THREADS), 0,
                         a.stream, xa, codes, scale, inv, p.cols, KB, tm, o);
    };
    if (p.tile == Tile::T256x256) go(S256{});
    else go(S128{});
  });
  return hipGetLastError();
}

size_t ffn_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int cus) {
  return grad_plan(M, N, K, cus).total;
}

hipError_t launch_ffn_grad(const FfnGradArgs& a, int cus) {
  const GradPlan p = grad_plan(a.M, a.N, a.K, cus);
  char* base = static_cast<char*>(a.ws);
  f16x8* fg = a.dx ? reinterpret_cast<f16x8*>(base + p.fg) : nullptr;
  f16x8* fu = a.dx ? reinterpret_cast<f16x8*>(base + p.fu) : nullptr;
  float* inv = reinterpret_cast<float*>(base + p.inv);
  const int64_t CB = p.rows / 32;
  with_type(a.type, [&](auto type) {
    using T = decltype(type);
    const T *z = static_cast<const T*>(a.z), *dh = static_cast<const T*>(a.dh);
    if (a.dx)
      hipLaunchKernelGGL(ffn_bound_kernel<T>, dim3(static_cast<unsigned>(a.M)), dim3(64 * BOUND_WAVES), 0, a.stream, z,
                         dh, inv, a.N);
    const dim3 grid(static_cast<unsigned>((a.M + 15) / 16), static_cast<unsigned>((CB + 3) / 4));
    auto* kernel = a.act == ACT_SILU ? ffn_dz_kernel<ACT_SILU, T> : ffn_dz_kernel<ACT_GELU, T>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, a.stream, z, dh,
                       static_cast<T*>(a.dz), inv, fg, fu, a.M, a.N, CB);
  });
  Q4_TRY(hipGetLastError());
  if (!a.dx) return hipSuccess;
  TransposedGemm g = {};
  g.g = fg;
  g.g2 = fu;
  g.pa = 2;
  g.pb = 2;
  g.type = a.type;
  g.w = a.gate;
  g.w2 = a.up;
  g.N = a.N;
  g.M = a.M;
  g.K = a.K;
  g.CB = CB;
  g.rt = p.rt;
  g.splits = p.splits;
  g.part = reinterpret_cast<float*>(base + p.part);
  Q4_TRY(launch_gemm_transposed(g, a.stream));
  return launch_fold(g.part, 2 * p.splits, inv, a.dx, a.type, a.M, a.K, a.stream);
}

}  // namespace q4
