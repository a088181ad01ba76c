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
// step the two dependent launches.  Products run on the matrix cores as
// bfloat16 with float32 sums, in a fixed order: a value enters as one, two or
// three bfloat16 parts (bfloat16, float16, float32: the leading 8 bits of
// what is left, exact), of which the second is below 2^-7 of the whole and the
// third below 2^-15.  Of the products of parts only that of two third ones is
// left out (below 2^-30).  One v_mfma_f32_16x16x32_bf16 takes the reduction
// steps of eight float32 MFMAs in a sixteenth of their time, so eight of them
// are still twice as fast.
//
// A first launch contracts the long axis ("down": rank vectors h and g),
// split over workgroups into slices that the next launch adds.  Rows are
// taken 64 at a time; within a tile the rows that share an adapter (not
// necessarily adjacent) form a group, and the groups of a tile are dealt to
// gridDim.y workgroups, so a decode batch whose rows all use different
// adapters reads those adapters in parallel, and a prompt reads its adapter
// once for 64 rows.
//
// MFMA operand layout: lane l = i + 16 g (i < 16, g < 4) carries row / column
// i and one reduction index of group g; any permutation of the reduction axis
// may be used if both operands agree.  Result: column l % 16, rows 4 g + v.

#include <algorithm>

#include "q4_kernels.h"
#include "q4_types.h"

namespace q4 {
namespace {

constexpr int LT = 64;          // rows per tile
constexpr int SUB = LT / 16;    // MFMA row blocks of a tile
constexpr int DOWN_WAVES = 8;   // waves of a "down" workgroup, each its part of the long axis
constexpr int DOWN_STEP = 32;   // reduction indices per wave and step
constexpr int DECODE_ROWS = 256;  // calls of up to this many rows may be a decode batch
constexpr int FEW = 8;          // groups of up to this many rows take the vector unit

__device__ __forceinline__ f32x4 mfma_f32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight values as sums of NP bfloat16 parts.
template <int NP>
struct Parts {
  bf16x8 p[NP];
};
template <typename T>
constexpr int parts_of = sizeof(T) == 4 ? 3 : (__is_same(T, __bf16) ? 1 : 2);

__device__ __forceinline__ uint32_t pack_high(float a, float b) {  // the high halves of a and b
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// Leading 8 significant bits, then the rest's (truncation: exact remainders).
template <int NP>
__device__ __forceinline__ Parts<NP> split8(const float (&v)[8]) {
  Parts<NP> out;
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_high(r[2 * e], r[2 * e + 1]);
    out.p[p] = __builtin_bit_cast(bf16x8, w);
    if (p + 1 < NP) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] -= __uint_as_float(__float_as_uint(r[e]) & 0xFFFF0000u);
    }
  }
  return out;
}

template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma_parts(const Parts<NA>& a, const Parts<NB>& b, f32x4 c) {
#pragma unroll
  for (int s = 3; s >= 0; --s)  // small products first; (2, 2) is left out
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[s - i], c, 0, 0, 0);
  return c;
}

// The rows of a tile that share an adapter, packed: member u is the tile's
// row of(u), u < count.
struct Group {
  uint64_t rows;
  int count, packed;  // packed: lane u holds member u's row
  __device__ __forceinline__ explicit Group(uint64_t mask)
      : rows(mask), count(__builtin_popcountll(mask)) {
    // members first, in order, then the others: a permutation of the lanes
    const int lane = threadIdx.x & 63;
    const int before = __builtin_popcountll(mask & ((uint64_t(1) << lane) - 1));
    const int to = (mask >> lane) & 1u ? before : count + lane - before;
    packed = __builtin_amdgcn_ds_permute(4 * to, lane);
  }
  __device__ __forceinline__ int of(int u) const { return __shfl(packed, u); }
  __device__ __forceinline__ int blocks() const { return (count + 15) >> 4; }
};

// The adapter groups of a 64-row tile: calls f(group, id) for every group that
// falls to this workgroup.  Uniform over the workgroup (every wave reads the
// same ids).
template <typename F>
__device__ __forceinline__ void for_groups(const int32_t* __restrict__ ids, int64_t m0, int64_t M,
                                           int adapters, int mine, int of, F f) {
  const int64_t row = m0 + (threadIdx.x & 63);
  const int id = row < M ? ids[row] : -1;
  uint64_t left = __ballot(id >= 0 && id < adapters);
  int next = mine;  // the next group of this workgroup's
  for (int n = 0; left != 0u; ++n) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t same = __ballot(id == a);
    left &= ~same;
    if (n == next) {
      f(Group(same), a);
      next += of;
    }
    if (next - n > __builtin_popcountll(left)) break;  // there are not that many left
  }
}

// Rows of the tile inside [0, M) that have no adapter.
__device__ __forceinline__ uint64_t rows_without(const int32_t* __restrict__ ids, int64_t m0,
                                                 int64_t M, int adapters) {
  const int64_t row = m0 + (threadIdx.x & 63);
  const int id = row < M ? ids[row] : 0;
  return __ballot(row < M && (id < 0 || id >= adapters));
}

// Eight consecutive elements c .. c + 7 of a row of C elements (zeros past
// its end, or where `live` is false); VEC: C % 8 == 0 and the row is 16-byte
// aligned (the model's K; N may be anything).
template <bool VEC, typename T>
__device__ __forceinline__ void row8(const T* __restrict__ row, int64_t c, int64_t C, bool live,
                                     float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
  if constexpr (VEC) {
    if (live && c < C) {
      if constexpr (sizeof(T) == 4) {
        float lo[4], hi[4];
        load_f32<4>(row + c, lo);
        load_f32<4>(row + c + 4, hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = lo[e]; v[4 + e] = hi[e]; }
      } else {
        load_f32<8>(row + c, v);
      }
    }
  } else if (live && c + 8 <= C) {
    load_any_f32<8>(row + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (live && c + e < C) v[e] = to_f32(row[c + e]);
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ Parts<parts_of<T>> load_parts(const T* __restrict__ row, int64_t c,
                                                         int64_t C, bool live) {
  if constexpr (VEC && __is_same(T, __bf16)) {
    Parts<1> out = {};
    if (live && c < C) out.p[0] = *reinterpret_cast<const bf16x8*>(row + c);
    return out;
  } else {
    float v[8];
    row8<VEC>(row, c, C, live, v);
    return split8<parts_of<T>>(v);
  }
}

// Part of the sum over c of Z[m, c] F_a[j, c] for NS blocks of 16 rows (row
// block s starts at zrow[s]): this wave's steps of [c0, c1).
template <typename T, typename TA, bool FT, bool VEC, int RT, int NS>
__device__ __forceinline__ void down_steps(const T* const (&zrow)[NS], const bool (&live)[NS],
                                           const TA* __restrict__ f, int64_t c0, int64_t c1,
                                           int64_t C, int R, int i, int g, f32x4 (&acc)[NS][RT]) {
#pragma unroll 1
  for (int64_t cs = c0; cs < c1; cs += DOWN_WAVES * DOWN_STEP) {
    const int64_t c = cs + 8 * g;  // this lane's reduction indices c .. c + 7
    Parts<parts_of<T>> z[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) z[s] = load_parts<VEC>(zrow[s], c, C, live[s]);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int j = 16 * t + i;
      Parts<parts_of<TA>> w;
      if constexpr (FT && __is_same(TA, __bf16)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w.p[0][e] = (j < R && c + e < C) ? f[(c + e) * R + j] : static_cast<__bf16>(0.f);
      } else if constexpr (FT) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = (j < R && c + e < C) ? to_f32(f[(c + e) * R + j]) : 0.f;
        w = split8<parts_of<TA>>(v);
      } else {
        w = load_parts<true>(f + static_cast<int64_t>(j) * C, c, C, j < R);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) acc[s][t] = mfma_parts(z[s], w, acc[s][t]);
    }
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
                                          f32x4 (*red)[4][64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int64_t m0 = tile * LT;
  const int64_t c0 = split * span + wave * DOWN_STEP, c1 = min(C, (split + 1) * span);
  for_groups(ids, m0, M, adapters, mine, of, [&](const Group& group, int a) {
    const TA* f = F + static_cast<int64_t>(a) * R * C;
    // the waves' parts of the 16 x 16 results of blocks s0, s0 + 1, ..., four at
    // a time, added in wave order
    auto finish = [&](auto& acc, int s0) {
      constexpr int NB = sizeof(acc) / sizeof(f32x4);
#pragma unroll
      for (int q = 0; q < NB; q += 4) {
#pragma unroll
        for (int u = 0; u < 4 && q + u < NB; ++u) red[wave][u][lane] = acc[(q + u) / RT][(q + u) % RT];
        __syncthreads();
        const int mine = q + wave;
        if (wave < 4 && mine < NB) {
          f32x4 sum = red[0][wave][lane];
#pragma unroll
          for (int w = 1; w < DOWN_WAVES; ++w) sum += red[w][wave][lane];
          const int j = 16 * (mine % RT) + i;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int u = 16 * (s0 + mine / RT) + 4 * g + v;
            const int row = group.of(u);
            if (u < group.count && j < R)
              P[(static_cast<int64_t>(split) * M + m0 + row) * R + j] = sum[v];
          }
        }
        __syncthreads();
      }
    };
    auto steps = [&](auto ns, int s0) {
      constexpr int NS = decltype(ns)::value;
      const T* zrow[NS];
      bool live[NS];
      f32x4 acc[NS][RT];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int u = 16 * (s0 + s) + i;
        live[s] = u < group.count;
        zrow[s] = Z + min(m0 + group.of(u), M - 1) * C;
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[s][t] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      down_steps<T, TA, FT, VEC, RT, NS>(zrow, live, f, c0, c1, C, R, i, g, acc);
      finish(acc, s0);
    };
    // as many blocks at once as the registers hold beside the factor
    constexpr int NS = RT <= 2 && sizeof(T) == 4 ? SUB : SUB / 2;
    if (group.count <= 16)
      steps(std::integral_constant<int, 1>{}, 0);
    else
      for (int s0 = 0; s0 < group.blocks(); s0 += NS) steps(std::integral_constant<int, NS>{}, s0);
  });
}

// Measured: one row of 3072, rank 16 3.9 us; 64 rows 7.3 us; 1500 x 1280, rank 64
// bfloat16 9.7 us.  Latency of a short pass over the row, and for prompts of the
// adapter's columns, which every tile reads again from the L2.
template <typename T, typename TA, int RT>
__global__ __launch_bounds__(64 * DOWN_WAVES, RT <= 2 && sizeof(T) == 2 ? 4 : 2) void lora_down_kernel(
    const T* __restrict__ X, const TA* __restrict__ A, const int32_t* __restrict__ ids,
    float* __restrict__ P, int64_t M, int64_t K, int R, int adapters, int splits, int64_t span) {
  __shared__ f32x4 red[DOWN_WAVES][4][64];
  const int64_t tile = blockIdx.x / splits;
  const int split = static_cast<int>(blockIdx.x - tile * splits);
  down_body<T, TA, false, true, RT>(X, A, ids, P, M, K, R, adapters, tile, split, span, blockIdx.y,
                                    gridDim.y, red);
}

// Both rank vectors of the backward pass: workgroups below `hblocks` h (from
// x), the rest g (from dy).
// Measured: 76 rows, 4096 and 3072 wide, rank 8 float32 6.4 us; 1500 rows, 1280 and
// 5120 wide, rank 32 bfloat16 15 us (19 MB, 1.3 TB/s; B is read down its columns,
// two bytes a lane).
template <typename T, typename TA, int RT, bool VEC>
__global__ __launch_bounds__(64 * DOWN_WAVES, RT <= 2 && sizeof(T) == 2 ? 4 : 2) void lora_down2_kernel(
    const T* __restrict__ X, const T* __restrict__ DY, const TA* __restrict__ A,
    const TA* __restrict__ B, const int32_t* __restrict__ ids, float* __restrict__ PH,
    float* __restrict__ PG, int64_t M, int64_t N, int64_t K, int R, int adapters, int hsplits,
    int64_t hspan, int gsplits, int64_t gspan, unsigned hblocks) {
  __shared__ f32x4 red[DOWN_WAVES][4][64];
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

// The slices' sum of one element, in slice order, eight loads in flight.
__device__ __forceinline__ float sum_slices(const float* __restrict__ p, int splits, int64_t step) {
  float s = 0.f;
  for (int t = 0; t < splits; t += 8) {
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = t + u < splits ? p[(t + u) * step] : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) s += v[u];
  }
  return s;
}

// The slices of h and g summed and scaled, once for the many workgroups that
// read them.  H, G: [M][R].  HT, GT (nullable): their three bfloat16 parts,
// transposed, [3][R][MP] with MP = M rounded up to 32.
// Measured: 3 us (1500 rows, rank 64) to 4.9 us (rank 32, both vectors and their
// parts).
__global__ __launch_bounds__(256) void lora_sum_kernel(
    const float* __restrict__ PH, const float* __restrict__ PG, const float* __restrict__ scale,
    const int32_t* __restrict__ ids, float* __restrict__ H, float* __restrict__ G,
    uint16_t* __restrict__ HT, uint16_t* __restrict__ GT, int64_t M, int R, int adapters,
    int hsplits, int gsplits, int64_t MP) {
  const int64_t n = M * R;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < n;
       e += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t m = e / R, j = e - m * R;
    const int id = ids[m];
    const bool ok = id >= 0 && id < adapters;
    const float s = ok && scale ? scale[id] : 1.f;
    auto put = [&](const float* p, int splits, float* out, uint16_t* t) {
      float v = ok ? s * sum_slices(p + e, splits, n) : 0.f;
      out[e] = v;
      if (!t) return;
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const uint32_t bits = __float_as_uint(v);
        t[(q * R + j) * MP + m] = static_cast<uint16_t>(bits >> 16);
        v -= __uint_as_float(bits & 0xFFFF0000u);
      }
    };
    if (hsplits) put(PH, hsplits, H, HT);
    if (gsplits) put(PG, gsplits, G, GT);
  }
}

// Rank vectors of a group as three bfloat16 parts (exact: two would leave up to
// 2^-15 of them out, 1500 rows of rank 64 in bfloat16 25.5 us against 26.1) in
// LDS, hs[part][member][ld]:
// scale * (the slices' sum); zero past the last member and for j in [R, R
// rounded up to 32).  ld = that + 8: rows 16-byte aligned, on different banks.
__device__ __forceinline__ int rank_ld(int R) { return ((R + 31) & ~31) + 8; }
constexpr int RANK_NP = 3;
constexpr size_t rank_lds(int64_t R) { return static_cast<size_t>(RANK_NP) * LT * (((R + 31) & ~31) + 8) * 2; }

__device__ __forceinline__ void load_rank(const float* __restrict__ P, int splits, int64_t M, int R,
                                          int64_t m0, const Group& group, float scale,
                                          uint16_t* hs) {
  const int ld = rank_ld(R), o8 = (ld - 8) / 8;  // groups of eight in a row
  for (int e = threadIdx.x; e < LT * o8; e += blockDim.x) {
    const int u8 = e / o8, j = 8 * (e - u8 * o8);  // (whole waves: LT is 64)
    const int row = group.of(u8);
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = 0.f;
    if (u8 < group.count && j < R) {
      const float* p = P + (m0 + row) * R + j;
      for (int t = 0; t < splits; ++t) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p + static_cast<int64_t>(t) * M * R);
        const f32x4 b = *reinterpret_cast<const f32x4*>(p + static_cast<int64_t>(t) * M * R + 4);
#pragma unroll
        for (int u = 0; u < 4; ++u) { v[u] += a[u]; v[4 + u] += b[u]; }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] *= scale;
    }
    const Parts<RANK_NP> q = split8<RANK_NP>(v);
#pragma unroll
    for (int u = 0; u < RANK_NP; ++u) *reinterpret_cast<bf16x8*>(hs + (u * LT + u8) * ld + j) = q.p[u];
  }
}

__device__ __forceinline__ Parts<RANK_NP> rank_parts(const uint16_t* hs, int ld, int row, int j) {
  Parts<RANK_NP> q;
#pragma unroll
  for (int u = 0; u < RANK_NP; ++u) q.p[u] = *reinterpret_cast<const bf16x8*>(hs + (u * LT + row) * ld + j);
  return q;
}

// y[m, n] = r[m, n] + sum_j hs[m][j] B_a[n, j] for one tile of rows and the
// columns [n0, n1).
//  - Groups of up to FEW rows (decode): a lane per column, its row of B read
//    in full, on the vector unit; loads and stores are contiguous.
//  - Larger groups: 64 columns per wave on the matrix cores.  MFMA row rho of
//    block t is column n = base + 16 (rho / 4) + 4 t + rho % 4, so a lane's
//    results are 16 consecutive columns of one row; B is read once for the
//    tile's 64 rows.
// NS: blocks of 16 rows multiplied at a time.  All four read B once (prompts);
// one keeps the registers low, for decode batches, whose groups mostly are
// few rows and whose speed is in how many workgroups are resident.
// Measured: one row x 6144, rank 16 5.2 us (latency); 64 rows x 18432 with up to 48
// adapters 13 us (34 MB, 2.6 TB/s); 1500 x 5120, rank 64 bfloat16 14.5 us (31 MB,
// 2.1 TB/s).
template <typename T, typename TA, int WAVES, int NS>
__global__ __launch_bounds__(64 * WAVES, NS == 1 ? 4 : 2) void lora_up_kernel(
    const float* __restrict__ P, const TA* __restrict__ B, const float* __restrict__ scale,
    const int32_t* __restrict__ ids, const T* R_, T* Y, int64_t M, int64_t N, int R, int adapters,
    int splits, int chunks, int64_t chunk) {
  extern __shared__ __attribute__((aligned(16))) uint16_t hs[];  // rank_lds(R) bytes
  const int ld = rank_ld(R);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int64_t tile = blockIdx.x / chunks;
  const int64_t n0 = (blockIdx.x - tile * chunks) * chunk, n1 = min(N, n0 + chunk);
  const int64_t m0 = tile * LT;
  constexpr int V = 16 / sizeof(T);       // elements of a 16-byte access
  const bool vec = N % V == 0;            // rows start on a 16-byte boundary

  // 16 consecutive columns of a row, base + 16 g on
  auto write = [&](int64_t base, int row, const f32x4 (&acc)[4]) {
    const int64_t n = base + 16 * g, at = (m0 + row) * N + n;
#pragma unroll
    for (int u = 0; u < 16; u += V) {
      float v[V];
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = acc[(u + e) / 4][(u + e) % 4];
      if (vec) {
        if (n + u < n1) {
          if (R_) {
            float q[V];
            load_f32<V>(R_ + at + u, q);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] += q[e];
          }
          store_f32<V>(Y + at + u, v);
        }
      } else if (n + u + V <= n1) {
        if (R_) {
          float q[V];
          load_any_f32<V>(R_ + at + u, q);
#pragma unroll
          for (int e = 0; e < V; ++e) v[e] += q[e];
        }
        store_any_f32<V>(Y + at + u, v);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (n + u + e < n1)
            Y[at + u + e] = from_f32<T>(R_ ? to_f32(R_[at + u + e]) + v[e] : v[e]);
      }
    }
  };

  for_groups(ids, m0, M, adapters, blockIdx.y, gridDim.y, [&](const Group& group, int a) {
    __syncthreads();  // the previous group's rank vectors are no longer read
    const TA* b = B + static_cast<int64_t>(a) * N * R;
    const float sc = scale ? scale[a] : 1.f;
    const int count = group.count;
    if (count <= FEW) {
      float* hf = reinterpret_cast<float*>(hs);  // [FEW][R]
      for (int e = threadIdx.x; e < FEW * R; e += 64 * WAVES) {
        const int u = e / R, j = e - u * R;
        const int row = group.of(u);  // (FEW * R is a multiple of 64: whole waves)
        if (u < count) hf[e] = sc * sum_slices(P + (m0 + row) * R + j, splits, M * R);
      }
      __syncthreads();
      // two rows and two columns per thread at a time: four sums, two rows of B
      // in flight (short code matters: each workgroup runs it a few times)
#pragma unroll 1
      for (int u = 0; u < count; u += 2) {
        const bool both = u + 1 < count;
        const int64_t row0 = (m0 + __builtin_amdgcn_readlane(group.packed, u)) * N;
        const int64_t row1 = both ? (m0 + __builtin_amdgcn_readlane(group.packed, u + 1)) * N : row0;
        const float *h0 = hf + u * R, *h1 = both ? h0 + R : h0;
#pragma unroll 1
        for (int64_t n = n0 + threadIdx.x; n < n1; n += 2 * 64 * WAVES) {
          const bool two = n + 64 * WAVES < n1;
          const int64_t n2 = two ? n + 64 * WAVES : n;
          float q[4] = {0.f, 0.f, 0.f, 0.f}, acc[4] = {0.f, 0.f, 0.f, 0.f};
          if (R_) {
            q[0] = to_f32(R_[row0 + n]);
            q[1] = to_f32(R_[row0 + n2]);
            q[2] = to_f32(R_[row1 + n]);
            q[3] = to_f32(R_[row1 + n2]);
          }
          const TA *b0 = b + n * R, *b1 = b + n2 * R;
#pragma unroll 2
          for (int j = 0; j < R; j += 8) {
            float w0[8], w1[8];
            row8<true>(b0, j, R, true, w0);
            row8<true>(b1, j, R, true, w1);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x0 = h0[j + e], x1 = h1[j + e];
              acc[0] = __builtin_fmaf(w0[e], x0, acc[0]);
              acc[1] = __builtin_fmaf(w1[e], x0, acc[1]);
              acc[2] = __builtin_fmaf(w0[e], x1, acc[2]);
              acc[3] = __builtin_fmaf(w1[e], x1, acc[3]);
            }
          }
          Y[row0 + n] = from_f32<T>(q[0] + acc[0]);
          if (two) Y[row0 + n2] = from_f32<T>(q[1] + acc[1]);
          if (both) Y[row1 + n] = from_f32<T>(q[2] + acc[2]);
          if (both && two) Y[row1 + n2] = from_f32<T>(q[3] + acc[3]);
        }
      }
      return;
    }
    load_rank(P, splits, M, R, m0, group, sc, hs);
    __syncthreads();
    for (int64_t base = n0 + 64 * wave; base < n1; base += 64 * WAVES) {
      const TA* brow[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        brow[t] = b + min(base + 16 * (i >> 2) + 4 * t + (i & 3), N - 1) * R;
#pragma unroll 1
      for (int s0 = 0; s0 < group.blocks(); s0 += NS) {
        f32x4 acc[NS][4];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[s][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int j0 = 0; j0 < R; j0 += 32) {
          Parts<parts_of<TA>> w[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) w[t] = load_parts<true>(brow[t], j0 + 8 * g, R, true);
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            if (NS > 1 && s >= group.blocks()) break;
            const Parts<RANK_NP> h = rank_parts(hs, ld, 16 * (s0 + s) + i, j0 + 8 * g);
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[s][t] = mfma_parts(w[t], h, acc[s][t]);
          }
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const int u = 16 * (s0 + s) + i, row = group.of(u);
          if (u < count) write(base, row, acc[s]);
        }
      }
    }
  });
  // rows without an adapter: y = r
  if (blockIdx.y == 0 && R_ != Y) {
    const Group group(rows_without(ids, m0, M, adapters));
    typedef T piece __attribute__((ext_vector_type(V)));
    const int step = vec ? V : 1, per = static_cast<int>((n1 - n0 + step - 1) / step);
    const int total = group.count * per;
    for (int e0 = 0; e0 < total; e0 += 64 * WAVES) {
      const int e = e0 + static_cast<int>(threadIdx.x), u = e / per;
      const int64_t at = (m0 + group.of(u < LT ? u : 0)) * N + n0 + static_cast<int64_t>(e - u * per) * step;
      if (e >= total) continue;
      if (vec) {
        piece p = {};
        if (R_) p = *reinterpret_cast<const piece*>(R_ + at);
        *reinterpret_cast<piece*>(Y + at) = p;
      } else {
        Y[at] = R_ ? R_[at] : from_f32<T>(0.f);
      }
    }
  }
}

// dx[m, k] = r[m, k] + sum_j G[m][j] A_a[j, k], 64 columns per wave at a
// time: MFMA column i of block t is k = base + 4 i + t, so a lane's loads and
// stores are four consecutive elements and a row's 64.
template <typename T, typename TA, int WAVES>
__device__ __forceinline__ void dx_body(const float* __restrict__ G, const TA* __restrict__ A,
                                        const int32_t* __restrict__ ids, const T* R_, T* DX,
                                        int64_t M, int64_t K, int R, int adapters, int64_t tile,
                                        int64_t k0, int64_t k1, int mine, int of, uint16_t* hs) {
  const int ld = rank_ld(R);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int64_t m0 = tile * LT;
  // members 4 g .. 4 g + 3 of block s, four columns each
  auto write = [&](const Group& group, int s, int64_t base, const f32x4 (&acc)[4]) {
    const int64_t k = base + 4 * i;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int u = 16 * s + 4 * g + v, row = group.of(u);
      if (u >= group.count || k >= k1) continue;  // K % 32 == 0: four columns in or out together
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
  for_groups(ids, m0, M, adapters, mine, of, [&](const Group& group, int a) {
    __syncthreads();
    load_rank(G, 1, M, R, m0, group, 1.f, hs);
    __syncthreads();
    const TA* ad = A + static_cast<int64_t>(a) * R * K;
    // blocks of 16 rows at a time: two leave the registers for two workgroups on
    // a CU (1500 x 5120 x 1280, rank 32: 30.6 -> 18.0 us for the kernel, with two
    // parts of the rank vectors)
    constexpr int NS = sizeof(T) == 2 ? 2 : SUB;
    for (int64_t base = k0 + 64 * wave; base < k1; base += 64 * WAVES) {
      const int64_t k = min(base + 4 * i, K - 4);
#pragma unroll 1
      for (int s0 = 0; s0 < group.blocks(); s0 += NS) {
        f32x4 acc[NS][4];
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[s][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int j0 = 0; j0 < R; j0 += 32) {
          // rows j0 + 8 g .. + 7 of A, four columns each, turned into the
          // operands of the four columns
          const int j = j0 + 8 * g;
          typedef TA piece __attribute__((ext_vector_type(4)));
          piece v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = piece{};
            if (j < R) v[e] = *reinterpret_cast<const piece*>(ad + static_cast<int64_t>(j + e) * K + k);  // R % 8 == 0
          }
          Parts<RANK_NP> h[NS];
#pragma unroll
          for (int s = 0; s < NS; ++s) h[s] = rank_parts(hs, ld, 16 * (s0 + s) + i, j);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            Parts<parts_of<TA>> w;
            if constexpr (__is_same(TA, __bf16)) {
              w.p[0] = bf16x8{v[0][t], v[1][t], v[2][t], v[3][t], v[4][t], v[5][t], v[6][t], v[7][t]};
            } else {
              float col[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) col[e] = to_f32(static_cast<TA>(v[e][t]));
              w = split8<parts_of<TA>>(col);
            }
#pragma unroll
            for (int s = 0; s < NS; ++s) acc[s][t] = mfma_parts(h[s], w, acc[s][t]);
          }
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) write(group, s0 + s, base, acc[s]);
      }
    }
  });
  if (mine == 0 && R_ != DX) {
    const uint64_t rows = rows_without(ids, m0, M, adapters);
    if (rows != 0u) {
      const Group group(rows);
      const f32x4 zero[4] = {};
      for (int64_t base = k0 + 64 * wave; base < k1; base += 64 * WAVES)
        for (int s = 0; s < group.blocks(); ++s) write(group, s, base, zero);
    }
  }
}

// Sum over the rows m of adapter a of L[m][j] Z[m, c], L the scaled rank
// vectors: 64 columns c per workgroup, the rows split over its waves.  OT
// false: out[j][c] (dA), true: out[c][j] (dB).  Rows of other adapters are
// read as zeros on both sides, so nothing of theirs (infinities, NaN) enters.
template <typename T, bool OT, int RT, int WAVES>
__device__ __forceinline__ void outer_body(const float* __restrict__ L, const T* __restrict__ Z,
                                           const int32_t* __restrict__ ids, float* __restrict__ out,
                                           const uint16_t* __restrict__ LT3, int64_t MP, int64_t M,
                                           int64_t C, int R, int a, int64_t c0,
                                           f32x4 (*red)[4][64]) {
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
    if constexpr (sizeof(T) == 2) {
      // 32 rows at a time: lane (i, g) has rows 8 g .. 8 g + 7, four columns
      // each as they are in memory
#pragma unroll 1
      for (int q = 0; q < 2; ++q) {
        if ((static_cast<uint32_t>(match >> (32 * q))) == 0u) continue;
        const unsigned ok = static_cast<unsigned>(match >> (32 * q + 8 * g)) & 0xFFu;
        const int64_t m = r0 + 32 * q + 8 * g;
        typedef T piece __attribute__((ext_vector_type(4)));
        piece z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const T* zr = Z + min(m + e, M - 1) * C;
          z[e] = piece{};
          if (c + 4 <= C) {
            if ((ok >> e) & 1u) z[e] = load_any<4>(zr + c);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (((ok >> e) & 1u) && c + u < C) z[e][u] = zr[c + u];
          }
        }
        u32x4 keep;  // both halves of a dword: two rows
#pragma unroll
        for (int e = 0; e < 4; ++e)
          keep[e] = ((ok >> (2 * e)) & 1u ? 0xFFFFu : 0u) | ((ok >> (2 * e + 1)) & 1u ? 0xFFFF0000u : 0u);
        Parts<3> l[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const int j = 16 * t + i;
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            u32x4 v = {0u, 0u, 0u, 0u};
            if (j < R && ok)  // MP is M rounded up to 32: eight rows are there where one is
              v = *reinterpret_cast<const u32x4*>(LT3 + (static_cast<int64_t>(p) * R + j) * MP + m);
            l[t].p[p] = __builtin_bit_cast(bf16x8, v & keep);
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          Parts<parts_of<T>> w;
          if constexpr (__is_same(T, __bf16)) {
            w.p[0] = bf16x8{z[0][u], z[1][u], z[2][u], z[3][u], z[4][u], z[5][u], z[6][u], z[7][u]};
          } else {
            float col[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) col[e] = to_f32(static_cast<T>(z[e][u]));
            w = split8<parts_of<T>>(col);
          }
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[t][u] = mfma_parts(l[t], w, acc[t][u]);
        }
      }
    } else {
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
#pragma unroll
          for (int u = 0; u < 4; ++u) z[s][u] = 0.f;
          if (c + 4 <= C) {
            if (ok) load_any_f32<4>(zr + c, z[s]);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (ok && c + u < C) z[s][u] = to_f32(zr[c + u]);
          }
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            const int j = 16 * t + i;
            l[s][t] = ok && j < R ? L[m * R + j] : 0.f;
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
  }
  // the waves' sums, added in wave order; then lane (i, g) of block (t, u)
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

// Last launch of the backward pass: workgroups [0, dxblocks) dx, the next
// adapters * achunks dA, the rest dB.
constexpr int G_WAVES = 8;
// Measured: 76 rows, rank 8 float32 10 us; 1500 rows, rank 32 bfloat16 19 us (34 MB,
// 1.8 TB/s).  Each adapter's workgroups look through all rows' ids for theirs.
template <typename T, typename TA, int RT>
__global__ __launch_bounds__(64 * G_WAVES, RT <= 2 && sizeof(T) == 2 ? 4 : 2) void lora_grad_kernel(
    const float* __restrict__ H, const float* __restrict__ G, const uint16_t* __restrict__ HT,
    const uint16_t* __restrict__ GT, int64_t MP, const T* __restrict__ X,
    const T* __restrict__ DY, const TA* __restrict__ A, const int32_t* __restrict__ ids,
    const T* R_, T* DX, float* __restrict__ DA, float* __restrict__ DB, int64_t M, int64_t N,
    int64_t K, int R, int adapters, int chunks, int64_t chunk, int gy, unsigned dxblocks,
    unsigned ablocks, int achunks, int bchunks) {
  __shared__ __attribute__((aligned(16))) union {
    f32x4 red[G_WAVES][4][64];
    uint16_t hs[rank_lds(16 * RT) / 2];
  } sh;
  const unsigned bid = blockIdx.x;
  if (bid < dxblocks) {
    const unsigned b = bid / gy;
    const int64_t tile = b / chunks;
    const int64_t k0 = (b - tile * chunks) * chunk;
    dx_body<T, TA, G_WAVES>(G, A, ids, R_, DX, M, K, R, adapters, tile, k0, min(K, k0 + chunk),
                            bid % gy, gy, sh.hs);
  } else if (bid < dxblocks + ablocks) {
    const unsigned b = bid - dxblocks;
    const int a = static_cast<int>(b / achunks);
    const int64_t c0 = static_cast<int64_t>(b - static_cast<unsigned>(a) * achunks) * 64;
    outer_body<T, false, RT, G_WAVES>(G, X, ids, DA + static_cast<int64_t>(a) * R * K, GT, MP,
                                            M, K, R, a, c0, sh.red);
  } else {
    const unsigned b = bid - dxblocks - ablocks;
    const int a = static_cast<int>(b / bchunks);
    const int64_t c0 = static_cast<int64_t>(b - static_cast<unsigned>(a) * bchunks) * 64;
    outer_body<T, true, RT, G_WAVES>(H, DY, ids, DB + static_cast<int64_t>(a) * N * R, HT, MP, M,
                                          N, R, a, c0, sh.red);
  }
}

// Workgroups a tile's adapter groups are dealt to: one per possible group
// for a decode batch, two for longer inputs (a tile of a prompt holds one
// request, or the seam of two).
unsigned group_blocks(int64_t M, int64_t adapters) {
  return static_cast<unsigned>(std::min<int64_t>({M, adapters, M <= DECODE_ROWS ? LT : 2}));
}

// Slices of a long axis of C for M rows: workgroups to fill the GPU once (a
// decode batch, whose groups may all be at work) or twice (a prompt, where
// about half find no group of theirs).
struct Split {
  int n;
  int64_t span;
};
Split down_split(int64_t M, int64_t C, int64_t adapters, int cus) {
  const int64_t tiles = (M + LT - 1) / LT;
  constexpr int64_t unit = DOWN_WAVES * DOWN_STEP;
  const int64_t units = (C + unit - 1) / unit;
  int64_t n = std::min<int64_t>(units, std::max<int64_t>(1, M <= DECODE_ROWS ? cus / (tiles * group_blocks(M, adapters)) : 2 * cus / tiles));
  n = std::min<int64_t>(n, 24);
  const int64_t span = (units + n - 1) / n * unit;
  return {static_cast<int>((C + span - 1) / span), span};
}

// Whether the slices of M rows are summed by a launch of their own.
bool sum_first(int64_t M, int splits) { return M > DECODE_ROWS && splits > 1; }

template <typename T, typename TA, int RT>
hipError_t lora_rt(const LoraArgs& p, int cus) {
  const int64_t tiles = (p.M + LT - 1) / LT;
  const Split sp = down_split(p.M, p.K, p.adapters, cus);
  float* P = static_cast<float*>(p.ws);
  const unsigned gy = group_blocks(p.M, p.adapters);
  hipLaunchKernelGGL((lora_down_kernel<T, TA, RT>), dim3(static_cast<unsigned>(tiles * sp.n), gy),
                     dim3(64 * DOWN_WAVES), 0, p.stream, static_cast<const T*>(p.x),
                     static_cast<const TA*>(p.a), p.ids, P, p.M, p.K, static_cast<int>(p.R),
                     static_cast<int>(p.adapters), sp.n, sp.span);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // a prompt's many workgroups read summed rank vectors; a decode batch adds
  // the slices itself and saves the launch
  const float* H = P;
  const float* scale = p.scale;
  int slices = sp.n;
  if (sum_first(p.M, sp.n)) {
    const int64_t MR = p.M * p.R;
    float* sum = P + sp.n * MR;
    hipLaunchKernelGGL(lora_sum_kernel, dim3(static_cast<unsigned>(std::min<int64_t>((MR + 255) / 256, 4096))),
                       dim3(256), 0, p.stream, P, nullptr, p.scale, p.ids, sum, nullptr, nullptr,
                       nullptr, p.M, static_cast<int>(p.R), static_cast<int>(p.adapters), sp.n, 0, 0);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    H = sum;
    scale = nullptr;
    slices = 1;
  }
  constexpr int WAVES = 4;
  const int64_t unit = 64 * WAVES, units = (p.N + unit - 1) / unit;
  // all workgroups resident at once (four per CU), so that each pays for its
  // rank vectors once
  const int64_t want = std::max<int64_t>(1, 4 * cus / (tiles * (p.M <= DECODE_ROWS ? gy : 1)));
  const int64_t per = (units + want - 1) / want;
  const int chunks = static_cast<int>((units + per - 1) / per);
  auto up = [&](auto ns) {
    hipLaunchKernelGGL((lora_up_kernel<T, TA, WAVES, decltype(ns)::value>),
                       dim3(static_cast<unsigned>(tiles * chunks), gy), dim3(64 * WAVES),
                       rank_lds(p.R), p.stream, H, static_cast<const TA*>(p.b), scale,
                       p.ids, static_cast<const T*>(p.r), static_cast<T*>(p.y), p.M, p.N,
                       static_cast<int>(p.R), static_cast<int>(p.adapters), slices, chunks,
                       per * unit);
  };
  if (p.M <= DECODE_ROWS)
    up(std::integral_constant<int, 1>{});
  else
    up(std::integral_constant<int, SUB>{});
  return hipGetLastError();
}

template <typename T, typename TA, int RT>
hipError_t lora_grad_rt(const LoraArgs& p, int cus) {
  const int64_t tiles = (p.M + LT - 1) / LT;
  const Split sh = down_split(p.M, p.K, p.adapters, cus), sg = down_split(p.M, p.N, p.adapters, cus);
  const int64_t MR = p.M * p.R;
  float* H = static_cast<float*>(p.ws);
  float* G = H + MR;
  float* PH = G + MR;
  float* PG = PH + sh.n * MR;
  const int64_t MP = (p.M + 31) & ~int64_t(31);
  uint16_t* HT = sizeof(T) == 2 ? reinterpret_cast<uint16_t*>(PG + sg.n * MR) : nullptr;
  uint16_t* GT = HT ? HT + 3 * MP * p.R : nullptr;
  const bool need_h = p.db != nullptr, need_g = p.y || p.da;
  const unsigned hb = need_h ? static_cast<unsigned>(tiles * sh.n) : 0u;
  const unsigned gb = need_g ? static_cast<unsigned>(tiles * sg.n) : 0u;
  const unsigned gy = group_blocks(p.M, p.adapters);
  const int R = static_cast<int>(p.R), adapters = static_cast<int>(p.adapters);
  // N is a multiple of 8: dy's rows are whole 16-byte pieces
  auto* down2 = p.N % 8 == 0 ? lora_down2_kernel<T, TA, RT, true> : lora_down2_kernel<T, TA, RT, false>;
  hipLaunchKernelGGL(down2, dim3(hb + gb, gy), dim3(64 * DOWN_WAVES),
                     0, p.stream, static_cast<const T*>(p.x), static_cast<const T*>(p.dy),
                     static_cast<const TA*>(p.a), static_cast<const TA*>(p.b), p.ids, PH, PG, p.M,
                     p.N, p.K, R, adapters, sh.n, sh.span, sg.n, sg.span, hb);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(lora_sum_kernel, dim3(static_cast<unsigned>(std::min<int64_t>((MR + 255) / 256, 4096))),
                     dim3(256), 0, p.stream, PH, PG, p.scale, p.ids, H, G, HT, GT, p.M, R, adapters,
                     need_h ? sh.n : 0, need_g ? sg.n : 0, MP);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t unit = 64 * G_WAVES, units = (p.K + unit - 1) / unit;
  const int64_t per = std::max<int64_t>(1, units / std::max<int64_t>(1, 2 * cus / tiles));
  const int chunks = static_cast<int>((units + per - 1) / per);
  const int achunks = static_cast<int>((p.K + 63) / 64), bchunks = static_cast<int>((p.N + 63) / 64);
  const unsigned dxb = p.y ? static_cast<unsigned>(tiles * chunks * gy) : 0u;
  const unsigned ab = p.da ? static_cast<unsigned>(p.adapters * achunks) : 0u;
  const unsigned bb = p.db ? static_cast<unsigned>(p.adapters * bchunks) : 0u;
  hipLaunchKernelGGL((lora_grad_kernel<T, TA, RT>), dim3(dxb + ab + bb), dim3(64 * G_WAVES), 0,
                     p.stream, H, G, HT, GT, MP, static_cast<const T*>(p.x), static_cast<const T*>(p.dy),
                     static_cast<const TA*>(p.a), p.ids, static_cast<const T*>(p.r),
                     static_cast<T*>(p.y), p.da, p.db, p.M, p.N, p.K, R, adapters, chunks,
                     per * unit, static_cast<int>(gy), dxb, ab, achunks, bchunks);
  return hipGetLastError();
}

template <typename T, typename TA>
hipError_t lora_types(const LoraArgs& p, int cus) {
  if (p.grad) {
    if (p.R <= 16) return lora_grad_rt<T, TA, 1>(p, cus);
    if (p.R <= 32) return lora_grad_rt<T, TA, 2>(p, cus);
    if (p.R <= 64) return lora_grad_rt<T, TA, 4>(p, cus);
    return lora_grad_rt<T, TA, 8>(p, cus);
  }
  if (p.R <= 16) return lora_rt<T, TA, 1>(p, cus);
  if (p.R <= 32) return lora_rt<T, TA, 2>(p, cus);
  if (p.R <= 64) return lora_rt<T, TA, 4>(p, cus);
  return lora_rt<T, TA, 8>(p, cus);
}

}  // namespace

// The size for any number of adapters: one gives the most slices.
size_t lora_workspace_bytes(int64_t M, int64_t K, int64_t R, int cus) {
  const int n = down_split(M, K, 1, cus).n;
  return static_cast<size_t>(n + (sum_first(M, n) ? 1 : 0)) * M * R * sizeof(float);
}

size_t lora_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int cus) {
  // slices, sums, and the sums' transposed parts (16-bit activations)
  return static_cast<size_t>(2 + down_split(M, K, 1, cus).n + down_split(M, N, 1, cus).n) * M * R *
             sizeof(float) +
         static_cast<size_t>(2 * 3) * ((M + 31) & ~int64_t(31)) * R * sizeof(uint16_t);
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
