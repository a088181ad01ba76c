// Low-rank adapters of many requests beside a shared projection, forward and
// backward.  With a = ids[m] the adapter of row m (none if outside
// [0, adapters)), A_a [R, K], B_a [N, R] and the adapter's scale s_a:
//
//   forward   y[m] = r[m] + s_a B_a (A_a x[m])
//   backward  h[m] = s_a A_a x[m]         g[m] = s_a B_a^T dy[m]
//             dx[m] = r[m] + A_a^T g[m]
//             dA_a = sum_{m of a} g[m] x[m]^T     dB_a = sum_{m of a} dy[m] h[m]^T
//
// The rank is small (8 to 128), so every product streams a long operand (x,
// dy, A, B, y) past a small one; what bounds them is bytes, and for a decode
// step the two dependent launches.  All sums are float32 on the matrix cores
// (v_mfma_f32_16x16x4_f32 takes float32 operands, so values of every type
// enter exactly), in a fixed order.
//
// A first launch contracts the long axis ("down": rank vectors h and g),
// split over workgroups into slices that the second launch adds while it
// loads them.  Rows are taken 16 at a time; within a tile the rows that share
// an adapter (not necessarily adjacent) form a group, and the groups of a
// tile are dealt to gridDim.y workgroups, so a decode batch whose rows all
// use different adapters reads those adapters in parallel.
//
// MFMA operand layout: lane l = i + 16 g (i < 16, g < 4) carries row / column
// i and one reduction index of group g; any permutation of the reduction axis
// may be used if both operands agree.  Result: column l % 16, rows 4 g + v.

#include <algorithm>

#include "q4_kernels.h"
#include "q4_types.h"

namespace q4 {
namespace {

constexpr int LT = 16;          // rows per tile
constexpr int DOWN_WAVES = 8;   // waves of a "down" workgroup, each its part of the long axis
constexpr int DOWN_STEP = 32;   // reduction indices per wave and step

__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// The adapter groups of a 16-row tile: calls f(rows, id) for every group that
// falls to this workgroup, rows a mask of the tile's rows.  Uniform over the
// workgroup (every wave reads the same ids).
template <typename F>
__device__ __forceinline__ void for_groups(const int32_t* __restrict__ ids, int64_t m0, int64_t M,
                                           int adapters, int mine, int of, F f) {
  const int lane = threadIdx.x & 63;
  const int64_t row = m0 + (lane & 15);
  const int id = row < M ? ids[row] : -1;
  unsigned left = static_cast<unsigned>(__ballot(id >= 0 && id < adapters)) & 0xFFFFu;
  for (int n = 0; left != 0u; ++n) {
    const int first = __builtin_ctz(left);
    const int a = __builtin_amdgcn_readlane(id, first);
    const unsigned same = static_cast<unsigned>(__ballot(id == a)) & left;
    left &= ~same;
    if (n % of == mine) f(same, a);
  }
}

// Rows of the tile inside [0, M) that have no adapter.
__device__ __forceinline__ unsigned rows_without(const int32_t* __restrict__ ids, int64_t m0,
                                                 int64_t M, int adapters) {
  const int64_t row = m0 + (threadIdx.x & 15);
  const int id = row < M ? ids[row] : 0;
  return static_cast<unsigned>(__ballot(row < M && (id < 0 || id >= adapters))) & 0xFFFFu;
}

// Eight consecutive elements c .. c + 7 of a row of C elements (zeros past
// its end); VEC: C % 8 == 0 and the row is 16-byte aligned.
template <bool VEC, typename T>
__device__ __forceinline__ void row8(const T* __restrict__ row, int64_t c, int64_t C, float (&v)[8]) {
  if constexpr (VEC) {
    if (c < C) {
      if constexpr (sizeof(T) == 4) {
        float lo[4], hi[4];
        load_f32<4>(row + c, lo);
        load_f32<4>(row + c + 4, hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = lo[e]; v[4 + e] = hi[e]; }
      } else {
        load_f32<8>(row + c, v);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < C ? to_f32(row[c + e]) : 0.f;
  }
}

// P[split][m][j] = sum over the split's part of c of Z[m, c] F_a[j, c] for the
// rows of each group.  F_a is [R][C] (FT false: A_a) or [C][R] (FT true: B_a,
// reduced over its rows).
template <typename T, typename TA, bool FT, bool VEC, int RT>
__device__ __forceinline__ void down_body(const T* __restrict__ Z, const TA* __restrict__ F,
                                          const int32_t* __restrict__ ids, float* __restrict__ P,
                                          int64_t M, int64_t C, int R, int adapters, int64_t tile,
                                          int split, int64_t span, int mine, int of,
                                          f32x4 (*red)[64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int64_t m0 = tile * LT;
  const T* zrow = Z + min(m0 + i, M - 1) * C;
  const int64_t c0 = split * span, c1 = min(C, c0 + span);
  for_groups(ids, m0, M, adapters, mine, of, [&](unsigned rows, int a) {
    const TA* f = F + static_cast<int64_t>(a) * R * C;
    f32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int64_t cs = c0 + wave * DOWN_STEP; cs < c1; cs += DOWN_WAVES * DOWN_STEP) {
      const int64_t c = cs + 8 * g;  // this lane's reduction indices c .. c + 7
      float z[8], w[RT][8];
      row8<VEC>(zrow, c, C, z);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int j = 16 * t + i;
        if constexpr (FT) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[t][e] = (j < R && c + e < C) ? to_f32(f[(c + e) * R + j]) : 0.f;
        } else {
          if (j < R) {
            row8<true>(f + static_cast<int64_t>(j) * C, c, C, w[t]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[t][e] = 0.f;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = mfma_f32(z[e], w[t][e], acc[t]);
    }
    // the waves' parts, added in wave order
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      red[wave][lane] = acc[t];
      __syncthreads();
      if (wave == 0) {
        f32x4 s = red[0][lane];
#pragma unroll
        for (int w = 1; w < DOWN_WAVES; ++w) s += red[w][lane];
        const int j = 16 * t + i;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int row = 4 * g + v;
          if (((rows >> row) & 1u) && j < R)
            P[(static_cast<int64_t>(split) * M + m0 + row) * R + j] = s[v];
        }
      }
      __syncthreads();
    }
  });
}

template <typename T, typename TA, int RT>
__global__ __launch_bounds__(64 * DOWN_WAVES) void lora_down_kernel(
    const T* __restrict__ X, const TA* __restrict__ A, const int32_t* __restrict__ ids,
    float* __restrict__ P, int64_t M, int64_t K, int R, int adapters, int splits, int64_t span) {
  __shared__ f32x4 red[DOWN_WAVES][64];
  const int64_t tile = blockIdx.x / splits;
  const int split = static_cast<int>(blockIdx.x - tile * splits);
  down_body<T, TA, false, true, RT>(X, A, ids, P, M, K, R, adapters, tile, split, span, blockIdx.y,
                                    gridDim.y, red);
}

// Both rank vectors of the backward pass: workgroups below `hblocks` h (from
// x), the rest g (from dy).
template <typename T, typename TA, int RT, bool VEC>
__global__ __launch_bounds__(64 * DOWN_WAVES) void lora_down2_kernel(
    const T* __restrict__ X, const T* __restrict__ DY, const TA* __restrict__ A,
    const TA* __restrict__ B, const int32_t* __restrict__ ids, float* __restrict__ PH,
    float* __restrict__ PG, int64_t M, int64_t N, int64_t K, int R, int adapters, int hsplits,
    int64_t hspan, int gsplits, int64_t gspan, unsigned hblocks) {
  __shared__ f32x4 red[DOWN_WAVES][64];
  if (blockIdx.x < hblocks) {
    const int64_t tile = blockIdx.x / hsplits;
    const int split = static_cast<int>(blockIdx.x - tile * hsplits);
    down_body<T, TA, false, true, RT>(X, A, ids, PH, M, K, R, adapters, tile, split, hspan,
                                      blockIdx.y, gridDim.y, red);
  } else {
    const unsigned b = blockIdx.x - hblocks;
    const int64_t tile = b / gsplits;
    const int split = static_cast<int>(b - tile * gsplits);
    down_body<T, TA, true, VEC, RT>(DY, B, ids, PG, M, N, R, adapters, tile, split, gspan,
                                    blockIdx.y, gridDim.y, red);
  }
}

// hs[row][j] = s_a * (the slices' sum), for the rows of a group; zero for the
// other rows and for j in [R, R rounded up to 16).
constexpr int HS_LD = 132;  // row stride in floats: 16-byte aligned, rows on different banks
__device__ __forceinline__ void load_rank(const float* __restrict__ P, int splits, int64_t M, int R,
                                          int64_t m0, unsigned rows, float scale,
                                          float (*hs)[HS_LD]) {
  const int R16 = (R + 15) & ~15;
  for (int e = threadIdx.x; e < LT * R16; e += blockDim.x) {
    const int row = e / R16, j = e - row * R16;
    float s = 0.f;
    if (((rows >> row) & 1u) && j < R) {
      const float* p = P + (m0 + row) * R + j;
      for (int t = 0; t < splits; ++t) s += p[static_cast<int64_t>(t) * M * R];
      s *= scale;
    }
    hs[row][j] = s;
  }
}

// y[m, n] = r[m, n] + sum_j hs[m][j] B_a[n, j] for one tile of rows and the
// columns [n0, n1).  Per wave 64 columns at a time: MFMA row rho of tile t is
// column n = base + 16 (rho / 4) + 4 t + rho % 4, so a lane's results are 16
// consecutive columns of one row.
template <typename T, typename TA, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void lora_up_kernel(
    const float* __restrict__ P, const TA* __restrict__ B, const float* __restrict__ scale,
    const int32_t* __restrict__ ids, const T* R_, T* Y, int64_t M, int64_t N, int R, int adapters,
    int splits, int chunks, int64_t chunk) {
  __shared__ float hs[LT][HS_LD];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int64_t tile = blockIdx.x / chunks;
  const int64_t n0 = (blockIdx.x - tile * chunks) * chunk, n1 = min(N, n0 + chunk);
  const int64_t m0 = tile * LT;
  const bool vec = (N & 3) == 0;  // rows start on a 4-element boundary

  auto write = [&](int64_t base, int row, const f32x4 (&acc)[4]) {
    const int64_t at = (m0 + row) * N + base + 16 * g;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t n = base + 16 * g + 4 * t;
      float v[4] = {acc[t].x, acc[t].y, acc[t].z, acc[t].w};
      if (vec) {
        if (n < n1) {
          if (R_) {
            float q[4];
            load_f32<4>(R_ + at + 4 * t, q);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += q[e];
          }
          store_f32<4>(Y + at + 4 * t, v);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < n1)
            Y[at + 4 * t + e] = from_f32<T>(R_ ? to_f32(R_[at + 4 * t + e]) + v[e] : v[e]);
      }
    }
  };

  for_groups(ids, m0, M, adapters, blockIdx.y, gridDim.y, [&](unsigned rows, int a) {
    __syncthreads();  // the previous group's rank vectors are no longer read
    load_rank(P, splits, M, R, m0, rows, scale ? scale[a] : 1.f, hs);
    __syncthreads();
    const TA* b = B + static_cast<int64_t>(a) * N * R;
    for (int64_t base = n0 + 64 * wave; base < n1; base += 64 * WAVES) {
      f32x4 acc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      const TA* brow[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        brow[t] = b + min(base + 16 * (i >> 2) + 4 * t + (i & 3), N - 1) * R;
      for (int j0 = 0; j0 < R; j0 += 16) {
        const int j = j0 + 4 * g;
        const f32x4 h = *reinterpret_cast<const f32x4*>(&hs[i][j]);
        float w[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if (j < R) {
            load_f32<4>(brow[t] + j, w[t]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[t][e] = 0.f;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[t] = mfma_f32(w[t][e], h[e], acc[t]);
      }
      if ((rows >> i) & 1u) write(base, i, acc);
    }
  });
  // rows without an adapter: y = r
  if (blockIdx.y == 0 && R_ != Y) {
    const unsigned rows = rows_without(ids, m0, M, adapters);
    if (rows != 0u) {
      const f32x4 zero[4] = {};
      for (int64_t base = n0 + 64 * wave; base < n1; base += 64 * WAVES)
        if ((rows >> i) & 1u) write(base, i, zero);
    }
  }
}

// dx[m, k] = r[m, k] + sum_j hs[m][j] A_a[j, k], 64 columns per wave at a
// time: MFMA column i of tile t is k = base + 4 i + t, so a lane's loads and
// stores are four consecutive elements and a row's 256.
template <typename T, typename TA, int WAVES>
__device__ __forceinline__ void dx_body(const float* __restrict__ PG, const TA* __restrict__ A,
                                        const float* __restrict__ scale,
                                        const int32_t* __restrict__ ids, const T* R_, T* DX,
                                        int64_t M, int64_t K, int R, int adapters, int splits,
                                        int64_t tile, int64_t k0, int64_t k1, float (*hs)[HS_LD]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int64_t m0 = tile * LT;
  auto write = [&](unsigned rows, int64_t base, const f32x4 (&acc)[4]) {
    const int64_t k = base + 4 * i;
    if (k >= k1) return;  // K % 32 == 0: four columns are in or out together
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 4 * g + v;
      if (!((rows >> row) & 1u)) continue;
      const int64_t at = (m0 + row) * K + k;
      float o[4] = {acc[0][v], acc[1][v], acc[2][v], acc[3][v]};
      if (R_) {
        float q[4];
        load_f32<4>(R_ + at, q);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += q[e];
      }
      store_f32<4>(DX + at, o);
    }
  };
  for_groups(ids, m0, M, adapters, 0, 1, [&](unsigned rows, int a) {
    __syncthreads();
    load_rank(PG, splits, M, R, m0, rows, scale ? scale[a] : 1.f, hs);
    __syncthreads();
    const TA* ad = A + static_cast<int64_t>(a) * R * K;
    for (int64_t base = k0 + 64 * wave; base < k1; base += 64 * WAVES) {
      f32x4 acc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int64_t k = min(base + 4 * i, K - 4);
      for (int j0 = 0; j0 < R; j0 += 8) {  // R % 8 == 0
        float w[2][4], h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          load_f32<4>(ad + static_cast<int64_t>(j0 + 4 * e + g) * K + k, w[e]);
          h[e] = hs[i][j0 + 4 * e + g];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[t] = mfma_f32(h[e], w[e][t], acc[t]);
      }
      write(rows, base, acc);
    }
  });
  if (R_ != DX) {
    const unsigned rows = rows_without(ids, m0, M, adapters);
    if (rows != 0u) {
      const f32x4 zero[4] = {};
      for (int64_t base = k0 + 64 * wave; base < k1; base += 64 * WAVES) write(rows, base, zero);
    }
  }
}

// Sum over the rows m of adapter a of l[m][j] Z[m, c], l the scaled rank
// vectors: 64 columns c per workgroup, the rows split over its waves.  OT
// false: out[j][c] (dA), true: out[c][j] (dB).  Rows of other adapters are
// read as zeros on both sides, so nothing of theirs (infinities, NaN) enters.
template <typename T, bool OT, int RT, int WAVES, bool VEC>
__device__ __forceinline__ void outer_body(const float* __restrict__ P, const T* __restrict__ Z,
                                           float scale, const int32_t* __restrict__ ids,
                                           float* __restrict__ out, int64_t M, int64_t C, int R,
                                           int a, int splits, int64_t c0, f32x4 (*red)[4][64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  f32x4 acc[RT][4];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int u = 0; u < 4; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t c = c0 + 4 * i;  // this lane's columns c .. c + 3
  for (int64_t r0 = 64 * wave; r0 < M; r0 += 64 * WAVES) {
    const int64_t mine = r0 + lane;
    const uint64_t match = __ballot(mine < M && ids[min(mine, M - 1)] == a);
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {  // 16 rows at a time
      const unsigned rows = static_cast<unsigned>(match >> (16 * q)) & 0xFFFFu;
      if (rows == 0u) continue;
      float l[4][RT], z[4][4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bool ok = (rows >> (4 * s + g)) & 1u;
        const int64_t m = min(r0 + 16 * q + 4 * s + g, M - 1);
        const T* zr = Z + m * C;
        if constexpr (VEC) {
          if (ok && c < C) {
            load_f32<4>(zr + c, z[s]);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) z[s][u] = 0.f;
          }
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) z[s][u] = ok && c + u < C ? to_f32(zr[c + u]) : 0.f;
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const int j = 16 * t + i;
          float v = 0.f;
          if (ok && j < R) {
            for (int p = 0; p < splits; ++p) v += P[(static_cast<int64_t>(p) * M + m) * R + j];
            v *= scale;
          }
          l[s][t] = v;
        }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int u = 0; u < 4; ++u) acc[t][u] = mfma_f32(l[s][t], z[s][u], acc[t][u]);
    }
  }
  // the waves' sums, added in wave order; then lane (i, g) of tile (t, u)
  // holds j = 16 t + 4 g + v, c = c0 + 4 i + u
#pragma unroll
  for (int t = 0; t < RT; ++t) {
#pragma unroll
    for (int u = 0; u < 4; ++u) red[wave][u][lane] = acc[t][u];
    __syncthreads();
    if (wave < 4) {
      if constexpr (OT) {
        // wave u: column c + u, four consecutive j
        f32x4 s = red[0][wave][lane];
        for (int w = 1; w < WAVES; ++w) s += red[w][wave][lane];
        const int j = 16 * t + 4 * g;
        if (c + wave < C && j < R)
          *reinterpret_cast<f32x4*>(out + (c + wave) * R + j) = s;
      } else {
        // wave v: rank row j, four consecutive columns
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < WAVES; ++w)
#pragma unroll
          for (int u = 0; u < 4; ++u) s[u] += red[w][u][lane][wave];
        const int j = 16 * t + 4 * g + wave;
        if (c < C && j < R) *reinterpret_cast<f32x4*>(out + static_cast<int64_t>(j) * C + c) = s;
      }
    }
    __syncthreads();
  }
}

// Second launch of the backward pass: workgroups [0, dxblocks) dx, the next
// adapters * achunks dA, the rest dB.
constexpr int G_WAVES = 8;
template <typename T, typename TA, int RT, bool VEC>
__global__ __launch_bounds__(64 * G_WAVES) void lora_grad_kernel(
    const float* __restrict__ PH, const float* __restrict__ PG, const T* __restrict__ X,
    const T* __restrict__ DY, const TA* __restrict__ A, const float* __restrict__ scale,
    const int32_t* __restrict__ ids, const T* R_, T* DX, float* __restrict__ DA,
    float* __restrict__ DB, int64_t M, int64_t N, int64_t K, int R, int adapters, int hsplits,
    int gsplits, int chunks, int64_t chunk, unsigned dxblocks, unsigned ablocks, int achunks,
    int bchunks) {
  __shared__ f32x4 red[G_WAVES][4][64];
  const unsigned bid = blockIdx.x;
  if (bid < dxblocks) {
    float(*hs)[HS_LD] = reinterpret_cast<float(*)[HS_LD]>(&red[0][0][0]);
    const int64_t tile = bid / chunks;
    const int64_t k0 = (bid - tile * chunks) * chunk;
    dx_body<T, TA, G_WAVES>(PG, A, scale, ids, R_, DX, M, K, R, adapters, gsplits, tile, k0,
                            min(K, k0 + chunk), hs);
  } else if (bid < dxblocks + ablocks) {
    const unsigned b = bid - dxblocks;
    const int a = static_cast<int>(b / achunks);
    const int64_t c0 = static_cast<int64_t>(b - static_cast<unsigned>(a) * achunks) * 64;
    outer_body<T, false, RT, G_WAVES, true>(PG, X, scale ? scale[a] : 1.f, ids,
                                            DA + static_cast<int64_t>(a) * R * K, M, K, R, a,
                                            gsplits, c0, red);
  } else {
    const unsigned b = bid - dxblocks - ablocks;
    const int a = static_cast<int>(b / bchunks);
    const int64_t c0 = static_cast<int64_t>(b - static_cast<unsigned>(a) * bchunks) * 64;
    outer_body<T, true, RT, G_WAVES, VEC>(PH, DY, scale ? scale[a] : 1.f, ids,
                                          DB + static_cast<int64_t>(a) * N * R, M, N, R, a, hsplits,
                                          c0, red);
  }
}

// Slices of a long axis of C for M rows: enough workgroups to fill the GPU,
// at least DOWN_WAVES steps each.
struct Split {
  int n;
  int64_t span;
};
Split down_split(int64_t M, int64_t C, int cus) {
  const int64_t tiles = (M + LT - 1) / LT;
  constexpr int64_t unit = DOWN_WAVES * DOWN_STEP;
  const int64_t units = (C + unit - 1) / unit;
  int64_t n = std::min<int64_t>(units, std::max<int64_t>(1, 2 * cus / tiles));
  n = std::min<int64_t>(n, 16);
  const int64_t span = (units + n - 1) / n * unit;
  return {static_cast<int>((C + span - 1) / span), span};
}

// Workgroups a tile's adapter groups are dealt to: one per possible group
// for a decode batch, two for longer inputs (a tile of a prompt holds one
// request, or the seam of two).
unsigned group_blocks(int64_t M) { return M <= 256 ? static_cast<unsigned>(std::min<int64_t>(M, LT)) : 2u; }

template <typename T, typename TA, int RT>
hipError_t lora_rt(const LoraArgs& p, int cus) {
  const int64_t tiles = (p.M + LT - 1) / LT;
  const Split sp = down_split(p.M, p.K, cus);
  float* P = static_cast<float*>(p.ws);
  const unsigned gy = group_blocks(p.M);
  hipLaunchKernelGGL((lora_down_kernel<T, TA, RT>), dim3(static_cast<unsigned>(tiles * sp.n), gy),
                     dim3(64 * DOWN_WAVES), 0, p.stream, static_cast<const T*>(p.x),
                     static_cast<const TA*>(p.a), p.ids, P, p.M, p.K, static_cast<int>(p.R),
                     static_cast<int>(p.adapters), sp.n, sp.span);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int WAVES = 4;
  const int64_t unit = 64 * WAVES, units = (p.N + unit - 1) / unit;
  const int64_t want = std::max<int64_t>(1, 4 * cus / tiles);
  const int64_t per = std::max<int64_t>(1, units / want);
  const int chunks = static_cast<int>((units + per - 1) / per);
  hipLaunchKernelGGL((lora_up_kernel<T, TA, WAVES>),
                     dim3(static_cast<unsigned>(tiles * chunks), gy), dim3(64 * WAVES), 0, p.stream,
                     P, static_cast<const TA*>(p.b), p.scale, p.ids, static_cast<const T*>(p.r),
                     static_cast<T*>(p.y), p.M, p.N, static_cast<int>(p.R),
                     static_cast<int>(p.adapters), sp.n, chunks, per * unit);
  return hipGetLastError();
}

template <typename T, typename TA, int RT, bool VEC>
hipError_t lora_grad_vec(const LoraArgs& p, int cus) {
  const int64_t tiles = (p.M + LT - 1) / LT;
  const Split sh = down_split(p.M, p.K, cus), sg = down_split(p.M, p.N, cus);
  float* PH = static_cast<float*>(p.ws);
  float* PG = PH + static_cast<int64_t>(sh.n) * p.M * p.R;
  const unsigned hb = p.db ? static_cast<unsigned>(tiles * sh.n) : 0u;
  const unsigned gb = p.y || p.da ? static_cast<unsigned>(tiles * sg.n) : 0u;
  hipLaunchKernelGGL((lora_down2_kernel<T, TA, RT, VEC>), dim3(hb + gb, group_blocks(p.M)),
                     dim3(64 * DOWN_WAVES), 0, p.stream, static_cast<const T*>(p.x),
                     static_cast<const T*>(p.dy), static_cast<const TA*>(p.a),
                     static_cast<const TA*>(p.b), p.ids, PH, PG, p.M, p.N, p.K,
                     static_cast<int>(p.R), static_cast<int>(p.adapters), sh.n, sh.span, sg.n,
                     sg.span, hb);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t unit = 64 * G_WAVES, units = (p.K + unit - 1) / unit;
  const int64_t per = std::max<int64_t>(1, units / std::max<int64_t>(1, 2 * cus / tiles));
  const int chunks = static_cast<int>((units + per - 1) / per);
  const int achunks = static_cast<int>((p.K + 63) / 64), bchunks = static_cast<int>((p.N + 63) / 64);
  const unsigned dxb = p.y ? static_cast<unsigned>(tiles * chunks) : 0u;
  const unsigned ab = p.da ? static_cast<unsigned>(p.adapters * achunks) : 0u;
  const unsigned bb = p.db ? static_cast<unsigned>(p.adapters * bchunks) : 0u;
  hipLaunchKernelGGL((lora_grad_kernel<T, TA, RT, VEC>), dim3(dxb + ab + bb), dim3(64 * G_WAVES), 0,
                     p.stream, PH, PG, static_cast<const T*>(p.x), static_cast<const T*>(p.dy),
                     static_cast<const TA*>(p.a), p.scale, p.ids, static_cast<const T*>(p.r),
                     static_cast<T*>(p.y), p.da, p.db, p.M, p.N, p.K, static_cast<int>(p.R),
                     static_cast<int>(p.adapters), sh.n, sg.n, chunks, per * unit, dxb, ab, achunks,
                     bchunks);
  return hipGetLastError();
}

template <typename T, typename TA>
hipError_t lora_types(const LoraArgs& p, int cus) {
  if (p.grad) {
    const bool vec = p.N % 8 == 0;
    if (p.R <= 16) return vec ? lora_grad_vec<T, TA, 1, true>(p, cus) : lora_grad_vec<T, TA, 1, false>(p, cus);
    if (p.R <= 32) return vec ? lora_grad_vec<T, TA, 2, true>(p, cus) : lora_grad_vec<T, TA, 2, false>(p, cus);
    if (p.R <= 64) return vec ? lora_grad_vec<T, TA, 4, true>(p, cus) : lora_grad_vec<T, TA, 4, false>(p, cus);
    return vec ? lora_grad_vec<T, TA, 8, true>(p, cus) : lora_grad_vec<T, TA, 8, false>(p, cus);
  }
  if (p.R <= 16) return lora_rt<T, TA, 1>(p, cus);
  if (p.R <= 32) return lora_rt<T, TA, 2>(p, cus);
  if (p.R <= 64) return lora_rt<T, TA, 4>(p, cus);
  return lora_rt<T, TA, 8>(p, cus);
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t R, int cus) {
  return static_cast<size_t>(down_split(M, K, cus).n) * M * R * sizeof(float);
}

size_t lora_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int cus) {
  return static_cast<size_t>(down_split(M, K, cus).n + down_split(M, N, cus).n) * M * R *
         sizeof(float);
}

bool lora_types_ok(int type, int atype) {
  return type_ok(type) && type_ok(atype) && (type == TYPE_F32 || atype == TYPE_F32 || atype == type);
}

hipError_t launch_lora(const LoraArgs& p, int cus) {
  if (p.type == TYPE_F32) {
    if (p.atype == TYPE_F32) return lora_types<float, float>(p, cus);
    if (p.atype == TYPE_F16) return lora_types<float, _Float16>(p, cus);
    return lora_types<float, __bf16>(p, cus);
  }
  if (p.type == TYPE_F16)
    return p.atype == TYPE_F32 ? lora_types<_Float16, float>(p, cus)
                               : lora_types<_Float16, _Float16>(p, cus);
  return p.atype == TYPE_F32 ? lora_types<__bf16, float>(p, cus)
                             : lora_types<__bf16, __bf16>(p, cus);
}

}  // namespace q4
