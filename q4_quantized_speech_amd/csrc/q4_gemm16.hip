// Prepared binary16 products on the CDNA4 matrix cores (see q4_gemm16.h for
// the operand layout), and the gradient of a Q4_0 projection built on them:
// dX[m, k] = sum_n dY[m, n] deq(W)[n, k] (section "Architecture" of
// "Implémentation en Rust du modèle Voxtral Mini 4B Realtime de Mistral pour
// l'exécuter dans le navigateur": the quantised projections).

#include <algorithm>

#include "q4_gemm16.h"
#include "q4_kernels.h"

namespace q4 {
namespace {

constexpr int XCDS = 8;

// The hardware deals workgroups to the XCDs round-robin; give XCD x a
// contiguous range of tiles, so tiles that share operands share an L2.
__device__ __forceinline__ unsigned xcd_order(unsigned bid, unsigned n) {
  const unsigned per = n / XCDS, rem = n % XCDS, x = bid % XCDS, i = bid / XCDS;
  return (x < rem ? x * (per + 1) : rem * (per + 1) + (x - rem) * per) + i;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// Power of two that brings `top` (a row's largest magnitude) to [2^14, 2^15);
// 1 for rows of zeros or with a magnitude that is not finite.
__device__ __forceinline__ float row_scale(float top) {
  if (!(top > 0.f) || !(top < __builtin_inff())) return 1.f;
  int e;
  frexpf(top, &e);  // top in [2^(e-1), 2^e)
  return ldexpf(1.f, min(15 - e, 126));
}

// Memory to LDS without registers: lane l's `SIZE` bytes at g land at
// l + SIZE * lane.  Asynchronous: arrived() before the barrier that publishes.
template <int SIZE>
__device__ __forceinline__ void to_lds(const void* g, void* l) {
  static_assert(SIZE == 16 || SIZE == 4, "bytes per lane");
  const auto gp = (const __attribute__((address_space(1))) void*)g;
  const auto lp = (__attribute__((address_space(3))) void*)l;
  if constexpr (SIZE == 16)
    __builtin_amdgcn_global_load_lds(gp, lp, 16, 0, 0);
  else
    __builtin_amdgcn_global_load_lds(gp, lp, 4, 0, 0);
}
// The loads to LDS before this point are issued before the work after it (they
// touch other arrays, so the compiler would be free to start them late).
__device__ __forceinline__ void issued() { asm volatile("" ::: "memory"); }
// This wave's loads to LDS are complete, and no LDS access moves across.
__device__ __forceinline__ void arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// ---------------------------------------------------------------------------
// Operand preparation
// ---------------------------------------------------------------------------

// One wave per row, 16 rows per workgroup, gridDim.y parts of the columns.
// Every workgroup takes the rows' maxima over all columns (its siblings' reads
// come from the L2), then its columns, 1024 at a time.  The fragments are put
// together in LDS and written whole: a wave's own 16-byte pieces lie 256 bytes
// apart (12.4 us for 16 x 3072 float32 that way).
// VEC: C % 4 == 0 (without it, reading the last elements one by one makes the
// kernel 18.7 us long for 1500 x 5120 bfloat16, with it 15).
// Measured: 16 x 3072 float32 6.5 us and 375 x 1280 7 us (latency of two passes
// over the row), 1500 x 5120 bfloat16 15 us (31 MB, 2 TB/s).
template <typename T, bool NIB, int PARTS, bool VEC>
__global__ __launch_bounds__(1024) void prep_rows_kernel(const T* __restrict__ X,
                                                         f16x8* __restrict__ out,
                                                         float* __restrict__ inv, int64_t M,
                                                         int64_t C, int64_t CB, int64_t bspan) {
  constexpr int SL = 2;  // slots of eight values per lane and pass: 32 blocks
  __shared__ f16x8 tile[2][PARTS][16 * SL][64];  // [buffer][part][block][swizzled lane]
  const int lane = threadIdx.x & 63, i = threadIdx.x >> 6;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * 16 + i;
  const bool live = m < M;
  const T* row = X + (live ? m : 0) * C;
  auto load4 = [&](int64_t c, float* v) {
    float t[4] = {0.f, 0.f, 0.f, 0.f};
    if (VEC ? live && c < C : live && c + 4 <= C) {
      if constexpr (VEC)
        load_f32<4>(row + c, t);
      else
        load_any_f32<4>(row + c, t);
    } else if (!VEC && live) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < C) t[e] = to_f32(row[c + e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t[e];
  };
  // float16 needs no scale: every value is one already
  float s = 1.f;
  if constexpr (!__is_same(T, _Float16)) {
    constexpr int PU = sizeof(T) == 4 ? 4 : 8;  // groups of eight values in flight
    float top = 0.f;
    for (int64_t c = 8 * lane; c < C; c += 512 * PU) {
      float v[PU][8];
#pragma unroll
      for (int u = 0; u < PU; ++u) {
        load4(c + 512 * u, v[u]);
        load4(c + 512 * u + 4, v[u] + 4);
      }
#pragma unroll
      for (int u = 0; u < PU; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[u][e]));
    }
    s = row_scale(wave_max(top));
  }
  if (live && lane == 0 && blockIdx.y == 0) inv[m] = 1.f / s;
  const int64_t part = static_cast<int64_t>(gridDim.x) * CB * 64;
  const int64_t b0 = blockIdx.y * bspan, b1 = min(CB, b0 + bspan);
  const int blk = lane >> 2, g = lane & 3;  // this lane's slot of each 16 blocks
  float v[SL][8];
  auto load = [&](int64_t b) {
#pragma unroll
    for (int u = 0; u < SL; ++u) {
      const int64_t c = 32 * (b + 16 * u + blk);
      load4(c + (NIB ? 4 * g : 8 * g), v[u]);
      load4(c + (NIB ? 16 + 4 * g : 8 * g + 4), v[u] + 4);
    }
  };
  load(b0);
  int cur = 0;
  for (int64_t b = b0; b < b1; b += 16 * SL, cur ^= 1) {
    // lane i + 16 g of a block sits at (i ^ (4 blk + g)) + 16 g: the lanes of a
    // wave (one i) then hit distinct banks, and so do the readers (one block)
    const int at = 16 * g + (i ^ (lane & 15));
#pragma unroll
    for (int u = 0; u < SL; ++u) {
      f16x8 hi, lo;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = v[u][e] * s;
        hi[e] = static_cast<_Float16>(x);
        if constexpr (PARTS == 2) lo[e] = static_cast<_Float16>(x - static_cast<float>(hi[e]));
      }
      tile[cur][0][16 * u + blk][at] = hi;
      if constexpr (PARTS == 2) tile[cur][1][16 * u + blk][at] = lo;
    }
    if (b + 16 * SL < b1) load(b + 16 * SL);
    __syncthreads();
    const int from = (lane & 48) + ((lane & 15) ^ ((4 * i + (lane >> 4)) & 15));
#pragma unroll
    for (int u = 0; u < SL; ++u) {  // wave i writes blocks b + i and b + 16 + i
      const int64_t mine = b + 16 * u + i;
      if (mine >= b1) break;
      const int64_t to = (static_cast<int64_t>(blockIdx.x) * CB + mine) * 64 + lane;
      out[to] = tile[cur][0][16 * u + i][from];
      if constexpr (PARTS == 2) out[part + to] = tile[cur][1][16 * u + i][from];
    }
  }
}

template <typename T>
void prep_rows_t(const T* x, Order order, f16x8* frag, float* inv, int64_t M, int64_t C,
                 hipStream_t s) {
  const int64_t CB = blocks32(C), tiles = (M + 15) / 16;
  // about a workgroup per CU, each at least 32 blocks
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>((CB + 31) / 32, 256 / tiles));
  const int64_t bspan = ((CB + want - 1) / want + 31) / 32 * 32;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((CB + bspan - 1) / bspan));
  const dim3 block(1024);
  constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;
  if (order == Order::NIBBLE)  // C is K, a multiple of 32
    hipLaunchKernelGGL((prep_rows_kernel<T, true, PARTS, true>), grid, block, 0, s, x, frag, inv, M,
                       C, CB, bspan);
  else if (C % 4 == 0)
    hipLaunchKernelGGL((prep_rows_kernel<T, false, PARTS, true>), grid, block, 0, s, x, frag, inv, M,
                       C, CB, bspan);
  else
    hipLaunchKernelGGL((prep_rows_kernel<T, false, PARTS, false>), grid, block, 0, s, x, frag, inv, M,
                       C, CB, bspan);
}

// (q - 8) of the eight codes of a dword, binary16, NIBBLE order.
__device__ __forceinline__ f16x8 codes8(uint32_t qs) {
  const uint32_t lo = qs & 0x0F0F0F0Fu, hi = (qs >> 4) & 0x0F0F0F0Fu;
  const uint32_t magic = 0x64646464u;  // 0x64xx: the binary16 value 1024 + q
  const f16x2 off = {static_cast<_Float16>(-1032.0f), static_cast<_Float16>(-1032.0f)};
  const f16x2 h0 = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(magic, lo, 0x04010400u)) + off;
  const f16x2 h1 = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(magic, lo, 0x04030402u)) + off;
  const f16x2 h2 = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(magic, hi, 0x04010400u)) + off;
  const f16x2 h3 = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(magic, hi, 0x04030402u)) + off;
  return f16x8{h0[0], h0[1], h1[0], h1[1], h2[0], h2[1], h3[0], h3[1]};
}

// One thread per block of 32 weights: 16 rows x 16 blocks per workgroup.
// Measured: 32768 x 3072 51 us (57 MB read, 214 MB written: 5.3 TB/s); bound by
// the writes.
__global__ __launch_bounds__(256) void prep_codes_kernel(const uint8_t* __restrict__ W, int64_t n0,
                                                         int64_t N, int64_t kblocks, int64_t KB,
                                                         f16x8* __restrict__ qfrag,
                                                         float* __restrict__ scale) {
  const int i = threadIdx.x & 15;
  const int64_t kb = static_cast<int64_t>(blockIdx.y) * 16 + (threadIdx.x >> 4);
  if (kb >= KB) return;
  const int64_t rt = blockIdx.x, n = n0 + rt * 16 + i;
  uint32_t d = 0, qs[4] = {0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u};
  if (n < N && kb < kblocks) load_block_any(W, n * kblocks + kb, d, qs);
  const int64_t f = rt * KB + kb;
#pragma unroll
  for (int g = 0; g < 4; ++g) qfrag[f * 64 + i + 16 * g] = codes8(qs[g]);
  scale[f * 16 + i] = half_bits_to_float(d);
}

// A wave's 32 rows x 72 bytes (128 columns from column 128 kt, first row even)
// to its own LDS, as consecutive dwords.  ODD: K is an odd multiple of 32, so a
// row's bytes are an odd number of half dwords and odd rows start in the middle
// of one: a row takes 19 dwords from the one it starts in, its bytes at 0 (even
// rows) or 2 (odd).  An even last row of the table ends in the middle of a
// dword, which is not loaded but put there by last_codes.
template <bool ODD>
struct Raw {
  static constexpr int ROW = ODD ? 19 : 18;    // dwords of a row
  static constexpr int LOADS = ODD ? 10 : 9;   // per lane
  static constexpr int SIZE = ODD ? 640 : 592;  // with what the last row's pair of reads touches
  static __device__ __forceinline__ int most(int rb, int kt) {  // a row's last dword
    return (ODD ? rb + 2 : rb) / 4 - 1 - kt * 18;
  }
  // Byte offsets of this lane's dwords from the first row, `left` of the table
  // (at most 32) from there on.  Rows past them repeat the last one, dwords past
  // the row (rb bytes) its last.
  static __device__ __forceinline__ void offsets(int left, int rb, int kt, uint32_t (&off)[LOADS]) {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // nothing of this is kept in registers for the last block
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int e = u * 64 + lane;
      const int row = min(e / ROW, left - 1);
      const bool cut = ODD && (left & 1) && row + 1 == left;
      const int at = min(e % ROW, most(rb, kt) - (cut ? 1 : 0));
      off[u] = static_cast<uint32_t>(row * rb - (ODD ? 2 * (row & 1) : 0) + at * 4);
    }
  }
  // The table's last two bytes, where its last row is one of these and even
  // (after the loads have arrived, by the wave that reads them).
  static __device__ __forceinline__ void last_codes(const uint8_t* __restrict__ W, int64_t N,
                                                    int left, int rb, int kt, uint32_t* raw) {
    if constexpr (ODD) {
      const int at = most(rb, kt);
      if ((left & 1) && at < 18) {
        if ((threadIdx.x & 63) == 0)
          raw[(left - 1) * ROW + at] = *reinterpret_cast<const uint16_t*>(W + N * rb - 2);
        issued();
      }
    }
  }
};

// Lane (i, g): dword i % 4 of the codes of block i / 4 and that block's scale
// in rows 8 g .. 8 g + 7.  A block starts at byte 18 (i / 4) of a row: its
// scale in either half of a dword, its codes from the next half on.
template <bool ODD>
struct RawCodes {
  uint32_t q[8];
  f16x2 d[4];
  // `live` rows (ODD: the scales of those past them, which may be any bytes,
  // are zero).
  __device__ __forceinline__ RawCodes(const uint32_t* raw, int live) {
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int first = 18 * (i >> 2) + (ODD ? 2 * (r & 1) : 0), code = first + 2 + 4 * (i & 3);
      const uint32_t* p = raw + (8 * g + r) * Raw<ODD>::ROW;
      const uint32_t* c = p + (code >> 2);
      q[r] = __builtin_amdgcn_alignbit(c[1], c[0], 8 * (code & 2));
      const _Float16 v = reinterpret_cast<const _Float16*>(p)[first >> 1];
      d[r >> 1][r & 1] = !ODD || 8 * g + r < live ? v : static_cast<_Float16>(0.f);
    }
  }
  // Low (h = 0) or high codes of every byte.
  __device__ __forceinline__ void half(int h, uint32_t (&nib)[8]) const {
#pragma unroll
    for (int r = 0; r < 8; ++r) nib[r] = (h ? q[r] >> 4 : q[r]) & 0x0F0F0F0Fu;
  }
  // The eight rows' weights (q - 8) d of byte b: hi rounded once to binary16,
  // lo the exact rest.
  template <int PB>
  __device__ __forceinline__ void column(const uint32_t (&nib)[8], int b, f16x8& hi, f16x8& lo) const {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t pair =
          __builtin_amdgcn_perm(nib[2 * p + 1], nib[2 * p], 0x0C000C00u | ((4u + b) << 16) | b) | 0x64006400u;
      const f16x2 off8 = {static_cast<_Float16>(-1032.0f), static_cast<_Float16>(-1032.0f)};
      const f16x2 w = __builtin_bit_cast(f16x2, pair) + off8;
      const f16x2 wd = w * d[p];
      hi[2 * p] = wd[0];
      hi[2 * p + 1] = wd[1];
      if constexpr (PB == 2) {
        // w has at most 15 significant bits and is a multiple of 2^-24 like
        // its scale, so the rest fits binary16
        const f16x2 rest = __builtin_elementwise_fma(w, d[p], -wd);
        lo[2 * p] = rest[0];
        lo[2 * p + 1] = rest[1];
      }
    }
  }
};

// The transposed weights: a wave takes 32 rows x 128 columns, turned in
// registers, put together in LDS and written as whole fragments (one thread
// per dword, its 16-byte pieces 64 bytes apart, takes 1.9 times as long on
// 32768 rows of 3072).
// Measured: 32768 x 3072 47 us with one part, 72 with two (258 and 460 MB);
// bound by the writes.
template <int PARTS, bool ODD>
__global__ __launch_bounds__(256) void prep_transpose_kernel(const uint8_t* __restrict__ W,
                                                               int64_t n0, int64_t N, int64_t K,
                                                               int64_t NB, int ktiles,
                                                               f16x8* __restrict__ tfrag) {
  using R = Raw<ODD>;
  __shared__ uint32_t raw[4][R::SIZE];
  __shared__ f16x8 tile[4][8][64];  // [wave][fragment][swizzled lane]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  const int64_t nb = item / ktiles;
  const int kt = static_cast<int>(item - nb * ktiles);
  if (nb >= NB) return;
  const int64_t rb = K / 32 * BLOCK_BYTES, n = n0 + nb * 32;
  // a block past the matrix (its weights are zero) loads its last even row
  const int64_t from = min(n, (N - 1) & ~int64_t(1));
  const int left = static_cast<int>(min<int64_t>(32, N - from)), row_bytes = static_cast<int>(rb);
  uint32_t off[R::LOADS];
  R::offsets(left, row_bytes, kt, off);
  const uint8_t* base = W + from * rb + static_cast<int64_t>(kt) * 72;
#pragma unroll
  for (int u = 0; u < R::LOADS; ++u) to_lds<4>(base + off[u], raw[wave] + u * 64);
  arrived();
  R::last_codes(W, N, left, row_bytes, kt, raw[wave]);
  RawCodes<ODD> codes(raw[wave], 32);
  // rows past the matrix: weights of zero
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (n + 8 * g + r >= N) codes.d[r >> 1][r & 1] = static_cast<_Float16>(0.f);
  const int64_t part = K / 16 * NB * 64;
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t nib[8];
      codes.half(h, nib);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        f16x8 hi, lo;
        codes.template column<PARTS>(nib, b, hi, lo);
        // fragment 2 (i / 4) + h, its lane 4 (i % 4) + b + 16 g; the low bits
        // are mixed with g so that the lanes of a store spread over the banks
        tile[wave][2 * (i >> 2) + h][4 * (i & 3) + (b ^ g) + 16 * g] = p ? lo : hi;
      }
    }
    // the tile is the wave's own, and LDS operations of a wave complete in order
    asm volatile("" ::: "memory");
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      const int64_t kf = static_cast<int64_t>(kt) * 8 + f;
      const f16x8 v = tile[wave][f][lane ^ (lane >> 4)];
      if (kf < K / 16) tfrag[p * part + (kf * NB + nb) * 64 + lane] = v;
    }
    asm volatile("" ::: "memory");
  }
}

// ---------------------------------------------------------------------------
// The product.  WM x WN waves, each FM x FN fragments of 16 x 16 outputs; a
// stage is KS blocks of 32 reduction indices of every fragment row of the
// tile, loaded straight to LDS while the previous stage is multiplied.
// ---------------------------------------------------------------------------
template <int WM_, int WN_, int FM_, int FN_>
struct Shape {
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_;
  static constexpr int THREADS = 64 * WM * WN, M = 16 * WM * FM, N = 16 * WN * FN;
};
using S256 = Shape<2, 4, 8, 4>;
using S128 = Shape<2, 2, 4, 4>;

template <typename S, int PA, int PB, int KS>
struct Stage {
  static constexpr int WAVES = S::WM * S::WN;
  static constexpr int FA = S::WM * S::FM * PA * KS, FB = S::WN * S::FN * PB * KS;
  static constexpr int NF = FA + FB, PER = (NF + WAVES - 1) / WAVES;

  const f16x8* at[PER];  // this wave's fragments of block 0

  // Fragments of a stage: A's first, [part][row tile][block].  Row tiles past
  // the matrix repeat its last one (their results are dropped).
  __device__ __forceinline__ Stage(const f16x8* __restrict__ A, const f16x8* __restrict__ B,
                                   int64_t ma, int64_t rta, int64_t mb, int64_t rtb, int64_t CB,
                                   int wave) {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int f = wave * PER + u;
      const bool isa = f < FA;
      const int h = isa ? f : f - FA;
      const int rows = (isa ? S::WM * S::FM : S::WN * S::FN);
      const int part = h / (rows * KS), row = h / KS % rows, k = h % KS;
      const int64_t rt = isa ? min(ma + row, rta - 1) : min(mb + row, rtb - 1);
      const int64_t all = isa ? rta : rtb;
      at[u] = (isa ? A : B) + ((part * all + rt) * CB + k) * 64;
    }
  }
  // Starts the loads of blocks c .. c + KS - 1.
  __device__ __forceinline__ void issue(f16x8 (*buf)[64], int64_t c, int wave, int lane) const {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      if (NF % WAVES != 0 && wave * PER + u >= NF) break;  // wave-uniform
      to_lds<16>(at[u] + c * 64 + lane, &buf[wave * PER + u][0]);
    }
    issued();
  }
};

// Measured, 256 x 256 tiles: 375 x 3072 over 32768 with three products per pair
// 227 us (998 TFLOP/s of binary16), 1500 with one 296 us (1020); the matrix cores
// are busy 43 % of the time, the rest waits on LDS and on the loads of the next
// stage.
template <typename S, int PA, int PB, int KS>
__global__ __launch_bounds__(S::THREADS) __attribute__((amdgpu_waves_per_eu(2, 2)))
void gemm_plain_kernel(const f16x8* __restrict__ A, const f16x8* __restrict__ B, int64_t M,
                       int64_t N, int64_t CB, int tiles_m, int tiles, int64_t span,
                       float* __restrict__ out, int64_t ld, const float* __restrict__ alpha) {
  using St = Stage<S, PA, PB, KS>;
  // two arrays rather than one of two: the compiler then knows that reading
  // one does not have to wait for loads into the other
  __shared__ f16x8 buf0[St::NF][64], buf1[St::NF][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned item = xcd_order(blockIdx.x, gridDim.x);
  const int split = item / tiles, tile = item % tiles;
  const int tm = tile % tiles_m, tn = tile / tiles_m;
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int64_t ma = static_cast<int64_t>(tm) * (S::M / 16), mb = static_cast<int64_t>(tn) * (S::N / 16);
  const int64_t rta = (M + 15) / 16, rtb = (N + 15) / 16;
  const int64_t c0 = split * span, c1 = min(CB, c0 + span);

  f32x4 acc[S::FM][S::FN];
#pragma unroll
  for (int i = 0; i < S::FM; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const St st(A, B, ma, rta, mb, rtb, CB, wave);
  // Steps of one row of fragments; a row's operand is read from LDS two steps
  // before its products, the next block's B half a block before.  The empty
  // volatile asm keeps that order.
  auto compute = [&](const f16x8 (*buf)[64]) {
    constexpr int STEPS = KS * S::FM;
    f16x8 a[3][PA], b[2][PB][S::FN];
    auto load_a = [&](int s) {
#pragma unroll
      for (int p = 0; p < PA; ++p)
        a[s % 3][p] = buf[(p * S::WM * S::FM + wm * S::FM + s % S::FM) * KS + s / S::FM][lane];
    };
    auto load_b = [&](int k) {
#pragma unroll
      for (int p = 0; p < PB; ++p)
#pragma unroll
        for (int j = 0; j < S::FN; ++j)
          b[k & 1][p][j] = buf[St::FA + (p * S::WN * S::FN + wn * S::FN + j) * KS + k][lane];
    };
    load_b(0);
    load_a(0);
    if constexpr (STEPS > 1) load_a(1);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int i = s % S::FM, k = s / S::FM;
      if (s + 2 < STEPS) load_a(s + 2);
      if (i == S::FM / 2 && k + 1 < KS) load_b(k + 1);
      // D rows are B's (the columns of out), D columns A's (its rows)
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[k & 1][0][j], a[s % 3][0], acc[i][j], 0, 0, 0);
        if constexpr (PB == 2)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[k & 1][1][j], a[s % 3][0], acc[i][j], 0, 0, 0);
        if constexpr (PA == 2)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[k & 1][0][j], a[s % 3][1], acc[i][j], 0, 0, 0);
      }
      asm volatile("" : "+v"(acc[i][0]), "+v"(acc[i][1]), "+v"(acc[i][2]), "+v"(acc[i][3])::"memory");
    }
  };
  if (c0 < c1) {  // a slice of a short reduction may be empty: its sum is zero
    st.issue(buf0, c0, wave, lane);
    arrived();
  }
  __syncthreads();
  int64_t c = c0;
  for (; c + 2 * KS <= c1; c += 2 * KS) {
    st.issue(buf1, c + KS, wave, lane);
    compute(buf0);
    arrived();
    __syncthreads();
    if (c + 2 * KS < c1) st.issue(buf0, c + 2 * KS, wave, lane);
    compute(buf1);
    arrived();
    __syncthreads();
  }
  if (c < c1) compute(buf0);
  // lane (i, g): row i of a fragment row, columns 4 g .. 4 g + 3 (N % 16 == 0)
  float* o = out + static_cast<int64_t>(split) * M * ld;
#pragma unroll
  for (int i = 0; i < S::FM; ++i) {
    const int64_t m = (ma + wm * S::FM + i) * 16 + (lane & 15);
    if (m >= M) continue;
    const float al = alpha ? alpha[m] : 0.f;
#pragma unroll
    for (int j = 0; j < S::FN; ++j) {
      const int64_t n = (mb + wn * S::FN + j) * 16 + 4 * (lane >> 4);
      if (n >= N) continue;
      f32x4* p = reinterpret_cast<f32x4*>(o + m * ld + n);
      f32x4 v = acc[i][j];
      if (alpha) {
        const f32x4 q = *p;
        v.x = __builtin_fmaf(al, q.x, v.x);
        v.y = __builtin_fmaf(al, q.y, v.y);
        v.z = __builtin_fmaf(al, q.z, v.z);
        v.w = __builtin_fmaf(al, q.w, v.w);
      }
      *p = v;
    }
  }
}

// Maximum over the 16 lanes of a DPP row, in all of them.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_f32<0xB1>(v));
  v = fmaxf(v, dpp_f32<0x4E>(v));
  v = fmaxf(v, dpp_f32<0x141>(v));
  v = fmaxf(v, dpp_f32<0x140>(v));
  return v;
}

// What the logits' accumulators leave: fragments of 16 rows from row `m0` and
// four of 16 columns from local column c0 (of `cols`, a multiple of 64); lane:
// column lane % 16 of a fragment, rows 4 g + v.
template <bool STATS, int FM>
__device__ __forceinline__ void logits_out(const f32x4 (&acc)[FM][4], int64_t m0, int64_t c0,
                                           int64_t cols, const float* __restrict__ inv, int64_t M,
                                           int64_t n0, int64_t N, const int32_t* __restrict__ targets,
                                           float* __restrict__ logits, float* __restrict__ tmax,
                                           float* __restrict__ tsum, float* __restrict__ tlogit,
                                           int64_t ld, int64_t tld) {
  if (c0 >= cols) return;
  const int lane = threadIdx.x & 63;
  const int64_t nl = c0 + (lane & 15), entry = c0 / 64;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t m = m0 + 16 * i + 4 * (lane >> 4) + v;
      const bool live = m < M;
      const float is = live ? inv[m] : 0.f;
      const int64_t t = live ? static_cast<int64_t>(targets[m]) - n0 - nl : -1;
      float l[4], top = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        l[j] = n0 + nl + 16 * j < N ? acc[i][j][v] * is : -__builtin_inff();
        if (STATS || t != 16 * j) top = fmaxf(top, l[j]);
      }
      top = row16_max(top);
      if constexpr (STATS) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool is_target = t == 16 * j && n0 + nl + 16 * j < N;
          if (is_target) tlogit[m] = l[j];
          if (!is_target && l[j] != -__builtin_inff()) s += expf(l[j] - top);
        }
        s = row16_sum(s);
        if (live && (lane & 15) == 0) {
          tmax[m * tld + entry] = top;
          tsum[m * tld + entry] = s;
        }
      } else if (live) {
#pragma unroll
        for (int j = 0; j < 4; ++j) logits[m * ld + nl + 16 * j] = l[j];
        if ((lane & 15) == 0) tmax[m * tld + entry] = top;
      }
    }
  }
}

// Measured, 256 x 256 tiles: 375 x 32768 over 3072 in two parts 179 us, 1500 in
// one 354 us (845 and 853 TFLOP/s of binary16).  The block scale's FMAs keep the
// vector unit busy 48 % of the time beside the matrix cores' 33 %.
template <typename S, int PA, int KS, bool STATS>
__global__ __launch_bounds__(S::THREADS) __attribute__((amdgpu_waves_per_eu(2, 2)))
void gemm_logits_kernel(const f16x8* __restrict__ A, const f16x8* __restrict__ Q,
                        const float* __restrict__ scale, const float* __restrict__ inv, int64_t M,
                        int64_t cols, int64_t CB, int tiles_m, int64_t n0, int64_t N,
                        const int32_t* __restrict__ targets, float* __restrict__ logits,
                        float* __restrict__ tmax, float* __restrict__ tsum,
                        float* __restrict__ tlogit, int64_t ld, int64_t tld) {
  static_assert(S::FN == 4, "a wave's columns are one entry of tmax");
  using St = Stage<S, PA, 1, KS>;
  constexpr int SC = S::N * KS;  // block scales of a stage, [row tile][block][16]
  constexpr int SU = (SC / 64 + St::WAVES - 1) / St::WAVES;  // loads of 64 scales per wave
  __shared__ f16x8 buf0[St::NF][64], buf1[St::NF][64];
  __shared__ float sc0[SC], sc1[SC];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned item = xcd_order(blockIdx.x, gridDim.x);
  const int tm = item % tiles_m, tn = item / tiles_m;
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int64_t ma = static_cast<int64_t>(tm) * (S::M / 16), mb = static_cast<int64_t>(tn) * (S::N / 16);
  const int64_t rta = (M + 15) / 16, rtb = cols / 16;

  f32x4 acc[S::FM][S::FN];
#pragma unroll
  for (int i = 0; i < S::FM; ++i)
#pragma unroll
    for (int j = 0; j < S::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const St st(A, Q, ma, rta, mb, rtb, CB, wave);
  auto issue = [&](f16x8 (*buf)[64], float* sc, int64_t c) {
    st.issue(buf, c, wave, lane);
#pragma unroll
    for (int u = 0; u < SU; ++u) {
      const int first = (wave * SU + u) * 64;
      if (SC / 64 % St::WAVES != 0 && first >= SC) break;
      const int e = first + lane;
      const int64_t rt = min(mb + e / (16 * KS), rtb - 1);
      to_lds<4>(scale + (rt * CB + c) * 16 + e % (16 * KS), sc + first);
    }
    issued();
  };
  // Row s + 1's products are started before row s's scaled sums are taken, so
  // the matrix cores and the vector unit overlap within the wave, and operands
  // are read from LDS two rows (B and its scales half a block) ahead.  The
  // empty volatile asm keeps that order (pure arithmetic would otherwise be
  // regrouped, all products first, whose temporaries then spill).
  auto compute = [&](const f16x8 (*buf)[64], const float* sc) {
    constexpr int STEPS = KS * S::FM;
    f16x8 a[3][PA], b[2][S::FN];
    float d[2][S::FN];
    auto load_a = [&](int s) {
#pragma unroll
      for (int p = 0; p < PA; ++p)
        a[s % 3][p] = buf[(p * S::WM * S::FM + wm * S::FM + s % S::FM) * KS + s / S::FM][lane];
    };
    auto load_b = [&](int k) {
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        b[k & 1][j] = buf[St::FA + (wn * S::FN + j) * KS + k][lane];
        d[k & 1][j] = sc[((wn * S::FN + j) * KS + k) * 16 + (lane & 15)];
      }
    };
    f32x4 t[2][S::FN];
    auto products = [&](int s) {
      const int k = s / S::FM;
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        t[s & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[s % 3][0], b[k & 1][j],
                                                             f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        if constexpr (PA == 2)
          t[s & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[s % 3][1], b[k & 1][j], t[s & 1][j], 0, 0, 0);
      }
      asm volatile("" : "+v"(t[s & 1][0]), "+v"(t[s & 1][1]), "+v"(t[s & 1][2]), "+v"(t[s & 1][3])::"memory");
    };
    load_b(0);
    load_a(0);
    if constexpr (STEPS > 1) load_a(1);
    products(0);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int i = s % S::FM, k = s / S::FM;
      if (s + 2 < STEPS) load_a(s + 2);
      if (i == S::FM / 2 - 1 && k + 1 < KS) load_b(k + 1);
      if (s + 1 < STEPS) products(s + 1);
#pragma unroll
      for (int j = 0; j < S::FN; ++j) {
        acc[i][j].x = __builtin_fmaf(d[k & 1][j], t[s & 1][j].x, acc[i][j].x);
        acc[i][j].y = __builtin_fmaf(d[k & 1][j], t[s & 1][j].y, acc[i][j].y);
        acc[i][j].z = __builtin_fmaf(d[k & 1][j], t[s & 1][j].z, acc[i][j].z);
        acc[i][j].w = __builtin_fmaf(d[k & 1][j], t[s & 1][j].w, acc[i][j].w);
      }
      asm volatile("" : "+v"(acc[i][0]), "+v"(acc[i][1]), "+v"(acc[i][2]), "+v"(acc[i][3]));
    }
  };
  issue(buf0, sc0, 0);
  arrived();
  __syncthreads();
  int64_t c = 0;
  for (; c + 2 * KS <= CB; c += 2 * KS) {
    issue(buf1, sc1, c + KS);
    compute(buf0, sc0);
    arrived();
    __syncthreads();
    if (c + 2 * KS < CB) issue(buf0, sc0, c + 2 * KS);
    compute(buf1, sc1);
    arrived();
    __syncthreads();
  }
  if (c < CB) compute(buf0, sc0);

  logits_out<STATS>(acc, (ma + wm * S::FM) * 16, (mb + wn * S::FN) * 16, cols, inv, M, n0, N, targets,
                    logits, tmax, tsum, tlogit, ld, tld);
}

// ---------------------------------------------------------------------------
// Logits of up to 64 rows straight from the Q4_0 bytes: they are read once, at
// their size, and bound by it.  A workgroup of eight waves owns 512 weight
// rows, each wave 64 of them; per chunk of 128 k the waves' raw bytes (72 a
// row) and the rows' fragments go to LDS by DMA while the previous chunk is
// multiplied.  A lane (i, g) of a wave reads dword g of a block's codes of
// weight row i: the operand of the exact codes q - 8, the block scale applied
// to the product (as in gemm_logits_kernel).
//
// ANY: K is no multiple of 128.  A row takes 19 dwords from the one it starts
// in: with K an odd multiple of 32, odd rows start in the middle of it.  The
// last chunk has one to three blocks; the scales of the others are zero.
// ---------------------------------------------------------------------------
constexpr int DW = 8;  // waves

// Measured: 38 x 131072 x 3072 float32 114 us (61 GFLOP of binary16 in two parts:
// 540 TFLOP/s; the table at 2 TB/s), bound by decoding, scaling and the latency of
// one chunk in flight; 8 rows of 65392 x 1280 bfloat16 36 us in all.
template <int RT, int PA, bool STATS, bool ANY>
__global__ __launch_bounds__(64 * DW) __attribute__((amdgpu_waves_per_eu(2, 2)))
void logits_direct_kernel(const f16x8* __restrict__ A, const uint8_t* __restrict__ W,
                          const float* __restrict__ inv, int64_t M, int64_t cols, int64_t K,
                          int64_t n0, int64_t N, const int32_t* __restrict__ targets,
                          float* __restrict__ logits, float* __restrict__ tmax,
                          float* __restrict__ tsum, float* __restrict__ tlogit, int64_t ld,
                          int64_t tld) {
  constexpr int FA = RT * PA * 4, PER = (FA + DW - 1) / DW;  // fragments of a chunk, per wave
  constexpr int ROW = ANY ? 19 : 18;                         // dwords of a row in LDS
  __shared__ f16x8 a0[FA][64], a1[FA][64];                   // [part][row tile][block]
  __shared__ uint32_t raw0[DW][64 * ROW], raw1[DW][64 * ROW];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int64_t rb = K / 32 * BLOCK_BYTES, CB = K / 32, rta = (M + 15) / 16;
  const int64_t AB = (CB + 1) / 2 * 2;  // blocks of a row of A (blocks32)
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * (64 * DW) + 64 * wave;

  // this lane's dwords of the wave's 64 rows; rows past the matrix repeat its
  // last one (their logits are dropped)
  auto start = [&](int64_t row) { return row * rb & ~int64_t(3); };
  const int64_t row0 = min(n0 + c0, N - 1);
  const uint8_t* base = W + start(row0);
  uint32_t off[ROW];
#pragma unroll
  for (int u = 0; u < ROW; ++u) {
    const int e = u * 64 + lane;
    off[u] = static_cast<uint32_t>(start(min(n0 + c0 + e / ROW, N - 1)) - start(row0) + e % ROW * 4);
  }
  // the last dword of a row that lies in the table
  auto most = [&](int64_t row) { return ((min((row + 1) * rb + 3, N * rb) - start(row)) >> 2) - 1; };
  const int64_t chunks = (CB + 3) / 4;
  auto issue = [&](f16x8 (*a)[64], uint32_t* raw, int64_t chunk) {
    if (ANY && chunk == chunks - 1) {
#pragma unroll
      for (int u = 0; u < ROW; ++u) {
        const int e = u * 64 + lane;
        const int64_t over = chunk * 18 + e % ROW - most(min(n0 + c0 + e / ROW, N - 1));
        to_lds<4>(base + chunk * 72 + off[u] - 4 * max<int64_t>(0, over), raw + u * 64);
      }
    } else {
#pragma unroll
      for (int u = 0; u < ROW; ++u) to_lds<4>(base + chunk * 72 + off[u], raw + u * 64);
    }
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int f = wave * PER + u;
      if (FA % DW != 0 && f >= FA) break;  // wave-uniform
      const int p = f / (RT * 4), t = f / 4 % RT, b = f % 4;
      const int64_t rt = min<int64_t>(t, rta - 1);
      const int64_t block = ANY ? min(chunk * 4 + b, CB - 1) : chunk * 4 + b;
      to_lds<16>(A + ((p * rta + rt) * AB + block) * 64 + lane, &a[f][0]);
    }
    issued();
  };
  // the last chunk's bytes, once they have arrived: a lane per row
  auto finish = [&](uint32_t* raw) {
    const int64_t n = n0 + c0 + lane;
    uint16_t* h = reinterpret_cast<uint16_t*>(raw + lane * ROW) + (CB & lane & 1);
    for (int b = static_cast<int>(CB % 4); b < 4; ++b) h[9 * b] = 0;
    // an even last row of the table may end in the middle of a dword
    if (n == N - 1 && (N * rb & 3) != 0)
      raw[lane * ROW + most(n) + 1 - (chunks - 1) * 18] = *reinterpret_cast<const uint16_t*>(W + N * rb - 2);
    issued();
  };

  f32x4 acc[RT][4];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // 16 steps: block b = s / 4, weight rows 16 j .. of j = s % 4; a step's
  // codes are read one step ahead, and its scaled sums are taken while the
  // next step's products run
  const int odd = static_cast<int>(CB & i & 1);  // ANY: this lane's rows start at byte 2
  const int at0 = i * ROW + g;
  auto compute = [&](const f16x8 (*a)[64], const uint32_t* raw) {
    uint32_t lo[2], hi[2];
    uint32_t dw[3];
    f16x8 x[RT][PA];
    f32x4 t[2][RT];
    auto codes = [&](int s) {
      const int b = s / 4, j = s % 4, at = 18 * b + 2;  // byte of the block's codes in a row
      const uint32_t* p = raw + 16 * j * ROW + at0 + at / 4;
      if constexpr (ANY) {
        if (at & 2) p += odd;
        lo[s & 1] = p[0];
        hi[s & 1] = p[1];
        dw[s % 3] = reinterpret_cast<const uint16_t*>(raw + 16 * j * ROW + i * ROW)[9 * b + odd];
      } else {
        lo[s & 1] = p[0];
        if (at & 2) hi[s & 1] = p[1];
        dw[s % 3] = raw[(16 * j + i) * ROW + 18 * b / 4];
      }
    };
    auto acts = [&](int b) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int p = 0; p < PA; ++p) x[r][p] = a[(p * RT + r) * 4 + b][lane];
    };
    auto products = [&](int s) {
      const int b = s / 4, at = 18 * b + 2;
      const f16x8 q = codes8(ANY ? __builtin_amdgcn_alignbit(hi[s & 1], lo[s & 1], at & 2 ? 16 - 16 * odd : 16 * odd)
                             : at & 2 ? shift16(hi[s & 1], lo[s & 1]) : lo[s & 1]);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        t[s & 1][r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[r][0], q, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        asm volatile("" : "+v"(t[s & 1][r])::"memory");
      }
      if constexpr (PA == 2) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          t[s & 1][r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[r][1], q, t[s & 1][r], 0, 0, 0);
          asm volatile("" : "+v"(t[s & 1][r])::"memory");
        }
      }
    };
    codes(0);
    acts(0);
    codes(1);
    products(0);
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      if (s + 2 < 16) codes(s + 2);
      if (s + 1 < 16) {
        if ((s + 1) % 4 == 0) acts((s + 1) / 4);
        products(s + 1);
      }
      const int b = s / 4, j = s % 4;
      const float d = half_bits_to_float(ANY ? dw[s % 3] : (18 * b) & 2 ? dw[s % 3] >> 16 : dw[s % 3] & 0xFFFFu);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        acc[r][j].x = __builtin_fmaf(d, t[s & 1][r].x, acc[r][j].x);
        acc[r][j].y = __builtin_fmaf(d, t[s & 1][r].y, acc[r][j].y);
        acc[r][j].z = __builtin_fmaf(d, t[s & 1][r].z, acc[r][j].z);
        acc[r][j].w = __builtin_fmaf(d, t[s & 1][r].w, acc[r][j].w);
        asm volatile("" : "+v"(acc[r][j]));
      }
    }
  };
  issue(a0, raw0[wave], 0);
  arrived();
  __syncthreads();
  int64_t c = 0;
  for (; c + 2 <= chunks; c += 2) {
    issue(a1, raw1[wave], c + 1);
    compute(a0, raw0[wave]);
    arrived();
    __syncthreads();
    if (c + 2 < chunks) issue(a0, raw0[wave], c + 2);
    if (ANY && c + 2 == chunks) finish(raw1[wave]);
    compute(a1, raw1[wave]);
    arrived();
    __syncthreads();
  }
  if (c < chunks) {
    if constexpr (ANY) finish(raw0[wave]);
    compute(a0, raw0[wave]);
  }
  logits_out<STATS>(acc, 0, c0, cols, inv, M, n0, N, targets, logits, tmax, tsum, tlogit, ld, tld);
}

// ---------------------------------------------------------------------------
// The transposed product straight from the Q4_0 bytes: out[m, k] = sum_n
// G[m, n] deq(W)[n, k] for 16 RT rows and 128 columns per workgroup.  Its
// eight waves take every eighth block of 32 weight rows of the workgroup's
// range and add their sums at the end.
//
// A block's 32 rows x 72 bytes go to the wave's own LDS as they are, by DMA of
// consecutive dwords (each lane's codes straight from memory, 20 loads of four
// rows a block: 39.9 us against 38.7 at 1500 x 5120 x 1280 bfloat16 with one
// part of the weights).  A lane
// (i, g) takes one dword of codes of block i / 4 of the 128 columns from each
// of the rows 8 g .. 8 g + 7: eight rows of eight columns, turned
// in registers into the operands of the columns k = 32 (i / 4) + 4 (i % 4) +
// (c & 3) + 16 (c >> 2), c < 8, with the rows as the reduction.  A result lane
// then holds 32 consecutive columns of one row of G.  Weights are decoded
// once per 64 rows of G; at 64 rows that takes the vector unit about as long
// as the products take the matrix cores.
// ---------------------------------------------------------------------------
constexpr int TW = 8;  // waves

// Measured: 1500 x 5120 x 1280 bfloat16 49 us (two products per pair: 800
// TFLOP/s; one, with the weights rounded, 39), 375 x 1280 x 5120 float32 23.9 us
// (three: 620), 16 x 3072 x 4096 float32 8.2 us.
// Waves wait 41 to 44 % of their cycles, mostly for a block's bytes: two per SIMD
// do not cover them.
template <int RT, int PA, int PB, typename T, bool ODD>
__global__ __launch_bounds__(64 * TW) __attribute__((amdgpu_waves_per_eu(2, RT <= 1 ? 4 : 2)))
void gemm_transposed_kernel(const f16x8* __restrict__ G, const uint8_t* __restrict__ W, int64_t n0,
                            int64_t N, int64_t M, int64_t K, int64_t CB, int mtiles, int tiles,
                            int64_t span, float* __restrict__ part, const float* __restrict__ alpha,
                            const float* __restrict__ inv, T* __restrict__ out) {
  constexpr int RP = RT > 2 ? 2 : RT;  // row blocks added at a time
  __shared__ f32x4 red[4][RP * 8][64];
  // two arrays: reading one does not have to wait for loads into the other
  using R = Raw<ODD>;
  __shared__ uint32_t raw0[TW][R::SIZE], raw1[TW][R::SIZE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const unsigned item = xcd_order(blockIdx.x, gridDim.x);
  const int split = item / tiles, tile = item % tiles;
  const int mt = tile % mtiles, kt = tile / mtiles;
  const int64_t rb = K / 32 * BLOCK_BYTES;
  const int64_t rta = (M + 15) / 16, live = min(CB, (N - n0 + 31) / 32);
  const int64_t b1 = min(live, (split + 1) * span);

  // rows past the matrix repeat its last one (G is zero there), columns past it
  // its last dword (their results are dropped)
  uint32_t off[R::LOADS];
  const int row_bytes = static_cast<int>(rb);
  auto left = [&](int64_t nb) { return static_cast<int>(min<int64_t>(32, N - n0 - nb * 32)); };
  R::offsets(left(0), row_bytes, kt, off);

  struct Acts {
    f16x8 a[RT][PA];
  };
  auto load = [&](int64_t nb, uint32_t* raw, Acts& x) {
    if (left(nb) < 32) R::offsets(left(nb), row_bytes, kt, off);  // the last, partial block
    const uint8_t* base = W + (n0 + nb * 32) * rb + static_cast<int64_t>(kt) * 72;
#pragma unroll
    for (int u = 0; u < R::LOADS; ++u) to_lds<4>(base + off[u], raw + u * 64);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int p = 0; p < PA; ++p) {
        const int64_t rt = min(static_cast<int64_t>(mt) * RT + t, rta - 1);
        x.a[t][p] = G[((p * rta + rt) * CB + nb) * 64 + lane];
      }
    issued();
  };

  f32x4 acc[RT][8];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](int64_t nb, uint32_t* raw, const Acts& x) {
    R::last_codes(W, N, left(nb), row_bytes, kt, raw);
    const RawCodes<ODD> codes(raw, left(nb));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t nib[8];
      codes.half(h, nib);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        f16x8 hi, lo;
        codes.template column<PB>(nib, b, hi, lo);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          f32x4& s = acc[t][4 * h + b];
          s = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, x.a[t][0], s, 0, 0, 0);
          if constexpr (PB == 2) s = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, x.a[t][0], s, 0, 0, 0);
          if constexpr (PA == 2) s = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, x.a[t][1], s, 0, 0, 0);
        }
      }
    }
  };

  // one block is multiplied while the next one's loads are in flight; the
  // bytes are the wave's own, so its counter of loads is all there is to wait
  // for
  Acts x0, x1;
  int64_t nb = split * span + wave;
  if (nb < b1) load(nb, raw0[wave], x0);
  for (; nb < b1; nb += 2 * TW) {
    arrived();
    const bool two = nb + TW < b1;
    if (two) load(nb + TW, raw1[wave], x1);
    compute(nb, raw0[wave], x0);
    if (two) {
      arrived();
      if (nb + 2 * TW < b1) load(nb + 2 * TW, raw0[wave], x0);
      compute(nb + TW, raw1[wave], x1);
    }
  }

  // the waves' sums, RP row blocks at a time: 4-7 onto 0-3, then those four;
  // wave w finishes half (c >> 2) = w & 1 of the pass's row block w >> 1
  const int h = wave & 1;
  f32x4 s[4];
#pragma unroll
  for (int t0 = 0; t0 < RT; t0 += RP) {
    if (t0) __syncthreads();
#pragma unroll
    for (int e = 0; e < RP * 8; ++e)
      if (wave >= 4) red[wave - 4][e][lane] = acc[t0 + e / 8][e % 8];
    __syncthreads();
    if (wave < 4) {
#pragma unroll
      for (int e = 0; e < RP * 8; ++e)
        red[wave][e][lane] = acc[t0 + e / 8][e % 8] + red[wave][e][lane];
    }
    __syncthreads();
    const int t = wave >> 1;
    if (t >= t0 && t < t0 + RP) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[c] = red[0][(t - t0) * 8 + 4 * h + c][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) s[c] += red[w][(t - t0) * 8 + 4 * h + c][lane];
      }
    }
  }
  const int t = wave >> 1;
  const int64_t m = (static_cast<int64_t>(mt) * RT + t) * 16 + i;
  const int64_t k = static_cast<int64_t>(kt) * 128 + 32 * g + 16 * h;
  if (t >= RT || m >= M || k >= K) return;
  if (part) {
    f32x4* o = reinterpret_cast<f32x4*>(part + (static_cast<int64_t>(split) * M + m) * K + k);
    const float al = alpha ? alpha[m] : 0.f;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      f32x4 r = {s[0][v], s[1][v], s[2][v], s[3][v]};
      if (alpha) {
        const f32x4 q = o[v];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = __builtin_fmaf(al, q[e], r[e]);
      }
      o[v] = r;
    }
  } else {
    const float f = inv[m];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float r[4] = {f * s[0][v], f * s[1][v], f * s[2][v], f * s[3][v]};
      store_f32<4>(out + m * K + k + 4 * v, r);
    }
  }
}

// Measured: 16 x 4096 float32 3 us (a launch).
template <typename T>
__global__ __launch_bounds__(256) void fold_kernel(const float* __restrict__ part, int splits,
                                                   const float* __restrict__ inv,
                                                   T* __restrict__ out, int64_t M, int64_t K) {
  const int64_t quads = K / 4, total = M * quads;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t m = e / quads;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int t = 0; t < splits; t += 4) {  // four slices in flight
      f32x4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[u] = t + u < splits
                   ? *reinterpret_cast<const f32x4*>(part + static_cast<int64_t>(t + u) * M * K + 4 * e)
                   : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 4; ++u) s += v[u];
    }
    const float f = inv[m];
    const float v[4] = {s.x * f, s.y * f, s.z * f, s.w * f};
    store_f32<4>(out + 4 * e, v);
  }
}

template <typename F>
hipError_t with_tile(Tile t, F f) {
  if (t == Tile::T256x256)
    f(S256{});
  else
    f(S128{});
  return hipGetLastError();
}

}  // namespace

hipError_t prep_rows(const void* x, int type, Order order, f16x8* frag, float* inv, int64_t M,
                     int64_t C, hipStream_t s) {
  if (type == TYPE_F32)
    prep_rows_t(static_cast<const float*>(x), order, frag, inv, M, C, s);
  else if (type == TYPE_F16)
    prep_rows_t(static_cast<const _Float16*>(x), order, frag, inv, M, C, s);
  else
    prep_rows_t(static_cast<const __bf16*>(x), order, frag, inv, M, C, s);
  return hipGetLastError();
}

hipError_t prep_weights(const uint8_t* w, int64_t n0, int64_t rows, int64_t N, int64_t K,
                        f16x8* qfrag, float* scale, f16x8* tfrag, int parts, hipStream_t s) {
  const int64_t kblocks = K / 32, KB = blocks32(K);
  const unsigned gy = static_cast<unsigned>((KB + 15) / 16);
  if (qfrag)
    hipLaunchKernelGGL(prep_codes_kernel, dim3(static_cast<unsigned>(rows / 16), gy), dim3(256), 0,
                       s, w, n0, N, kblocks, KB, qfrag, scale);
  if (tfrag) {
    const int ktiles = static_cast<int>((K + 127) / 128);
    const dim3 grid(static_cast<unsigned>((rows / 32 * ktiles + 3) / 4));
    auto* kernel = K % 64 == 0 ? (parts == 2 ? prep_transpose_kernel<2, false> : prep_transpose_kernel<1, false>)
                               : (parts == 2 ? prep_transpose_kernel<2, true> : prep_transpose_kernel<1, true>);
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, w, n0, N, K, rows / 32, ktiles, tfrag);
  }
  return hipGetLastError();
}

TileDim tile_dim(Tile t) {
  return t == Tile::T256x256 ? TileDim{256, 256} : TileDim{128, 128};
}

double tile_time_us(Tile t, int64_t M, int64_t N, int64_t C, int units, int splits, int cus) {
  const TileDim d = tile_dim(t);
  const int64_t items = ((M + d.m - 1) / d.m) * ((N + d.n - 1) / d.n) * splits;
  const int per_cu = t == Tile::T256x256 ? 1 : 2;
  const double eff = t == Tile::T256x256 ? 0.45 : 0.30;
  const double cu_rate = 2.5e9 / 256 * eff;  // flops per microsecond of one CU
  const double rounds = static_cast<double>((items + per_cu * cus - 1) / (static_cast<int64_t>(per_cu) * cus));
  const double gemm = rounds * per_cu * 2.0 * d.m * d.n * (static_cast<double>(C) / splits) * units / cu_rate;
  return gemm + 2.0 * splits * M * N * 4.0 / 4e6;  // slices written and read at 4 TB/s
}

TransposedPlan transposed_plan(int64_t M, int64_t N, int64_t K, int units, int cus) {
  const int rt = transposed_rt(M);
  const int64_t tiles = (M + 16 * rt - 1) / (16 * rt) * ((K + 127) / 128);
  const int64_t blocks = (N + 31) / 32;
  TransposedPlan best = {1e30, 1};
  for (int s = 1; s <= 64 && (s == 1 || blocks >= s * TW); s = s < 4 ? s + 1 : s + s / 4) {
    const double rounds = static_cast<double>((tiles * s + cus - 1) / cus);
    // a wave's blocks, two waves on a SIMD; cycles of one: products and decode
    const int64_t per_wave = ((blocks + s - 1) / s + TW - 1) / TW;
    const double clk = std::max(8.0 * rt * units * 16, 800.0) * 1.4;
    double us = rounds * (2.0 * per_wave * clk / 2400.0 + 3.0);
    if (s > 1) us += 3.0 + 2.0 * s * M * K * 4 / 4e6;
    if (us < best.us) best = {us, s};
  }
  return best;
}

hipError_t launch_gemm_plain(Tile t, const PlainGemm& p, hipStream_t s) {
  const TileDim d = tile_dim(t);
  const int tm = static_cast<int>((p.M + d.m - 1) / d.m), tn = static_cast<int>((p.N + d.n - 1) / d.n);
  const int64_t span = ((p.CB / 2 + p.splits - 1) / p.splits) * 2;
  return with_tile(t, [&](auto shape) {
    using S = decltype(shape);
    auto go = [&](auto pa, auto pb, auto ks) {
      hipLaunchKernelGGL((gemm_plain_kernel<S, decltype(pa)::value, decltype(pb)::value, decltype(ks)::value>),
                         dim3(static_cast<unsigned>(static_cast<int64_t>(tm) * tn * p.splits)),
                         dim3(S::THREADS), 0, s, p.a, p.b, p.M, p.N, p.CB, tm, tm * tn, span, p.out,
                         p.ld, p.alpha);
    };
    using std::integral_constant;
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    if (p.pa == 1 && p.pb == 1) go(one, one, two);
    else if (p.pa == 1) go(one, two, one);
    else go(two, two, one);
  });
}

hipError_t launch_gemm_transposed(const TransposedGemm& p, hipStream_t s) {
  const int rt = transposed_rt(p.M);
  const int mtiles = static_cast<int>((p.M + 16 * rt - 1) / (16 * rt));
  const int tiles = static_cast<int>(mtiles * ((p.K + 127) / 128));
  const int64_t span = (p.CB + p.splits - 1) / p.splits;
  auto go = [&](auto rtc, auto pa, auto pb, auto type) {
    using T = decltype(type);
    constexpr int RT = decltype(rtc)::value, PA = decltype(pa)::value, PB = decltype(pb)::value;
    auto* kernel = p.K % 64 == 0 ? gemm_transposed_kernel<RT, PA, PB, T, false>
                                 : gemm_transposed_kernel<RT, PA, PB, T, true>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(static_cast<int64_t>(tiles) * p.splits)),
                       dim3(64 * TW), 0, s, p.g, p.w, p.n0, p.N, p.M, p.K, p.CB, mtiles, tiles, span,
                       p.part, p.alpha, p.inv, static_cast<T*>(p.out));
  };
  using std::integral_constant;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  auto parts = [&](auto rtc) {
    // float32 has two parts of both, float16 and bfloat16 one of G; the head's
    // gradient, which writes slices whatever its type, one of both there
    if (p.pa == 2) go(rtc, two, two, float{});
    else if (p.pb == 1) go(rtc, one, one, float{});
    else if (p.type == TYPE_F16) go(rtc, one, two, _Float16{});
    else go(rtc, one, two, __bf16{});
  };
  if (rt == 1) parts(one);
  else if (rt == 2) parts(two);
  else parts(integral_constant<int, 4>{});
  return hipGetLastError();
}

hipError_t launch_gemm_logits(Tile t, const LogitGemm& p, hipStream_t s) {
  const TileDim d = tile_dim(t);
  const int tm = static_cast<int>((p.M + d.m - 1) / d.m), tn = static_cast<int>((p.cols + d.n - 1) / d.n);
  return with_tile(t, [&](auto shape) {
    using S = decltype(shape);
    auto go = [&](auto pa, auto ks, auto stats) {
      hipLaunchKernelGGL((gemm_logits_kernel<S, decltype(pa)::value, decltype(ks)::value, decltype(stats)::value>),
                         dim3(static_cast<unsigned>(static_cast<int64_t>(tm) * tn)), dim3(S::THREADS), 0, s,
                         p.a, p.q, p.scale, p.inv, p.M, p.cols, p.CB, tm, p.n0, p.N, p.targets, p.logits,
                         p.tmax, p.tsum, p.tlogit, p.ld, p.tld);
    };
    using std::integral_constant;
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    const std::true_type yes;
    const std::false_type no;
    if (p.logits) {
      if (p.pa == 1) go(one, two, no); else go(two, one, no);
    } else {
      if (p.pa == 1) go(one, two, yes); else go(two, one, yes);
    }
  });
}

hipError_t launch_logits_direct(const uint8_t* w, const LogitGemm& p, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>((p.cols + 64 * DW - 1) / (64 * DW));
  auto go = [&](auto rt, auto pa, auto stats) {
    constexpr int RT = decltype(rt)::value, PA = decltype(pa)::value;
    constexpr bool STATS = decltype(stats)::value;
    auto* kernel = p.K % 128 == 0 ? logits_direct_kernel<RT, PA, STATS, false>
                                 : logits_direct_kernel<RT, PA, STATS, true>;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * DW), 0, s, p.a, w, p.inv, p.M, p.cols, p.K, p.n0, p.N,
                       p.targets, p.logits, p.tmax, p.tsum, p.tlogit, p.ld, p.tld);
  };
  using std::integral_constant;
  auto parts = [&](auto rt) {
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    if (p.logits) {
      if (p.pa == 1) go(rt, one, std::false_type{}); else go(rt, two, std::false_type{});
    } else {
      if (p.pa == 1) go(rt, one, std::true_type{}); else go(rt, two, std::true_type{});
    }
  };
  if (p.M <= 16) parts(integral_constant<int, 1>{});
  else if (p.M <= 32) parts(integral_constant<int, 2>{});
  else if (p.M <= 48) parts(integral_constant<int, 3>{});
  else parts(integral_constant<int, 4>{});
  return hipGetLastError();
}

hipError_t launch_fold(const float* part, int splits, const float* inv, void* out, int type,
                       int64_t M, int64_t K, hipStream_t s) {
  const int64_t total = M * (K / 4);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((total + 255) / 256, 8192));
  if (type == TYPE_F32)
    hipLaunchKernelGGL(fold_kernel<float>, dim3(grid), dim3(256), 0, s, part, splits, inv,
                       static_cast<float*>(out), M, K);
  else if (type == TYPE_F16)
    hipLaunchKernelGGL(fold_kernel<_Float16>, dim3(grid), dim3(256), 0, s, part, splits, inv,
                       static_cast<_Float16*>(out), M, K);
  else
    hipLaunchKernelGGL(fold_kernel<__bf16>, dim3(grid), dim3(256), 0, s, part, splits, inv,
                       static_cast<__bf16*>(out), M, K);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// dX = dY deq(W)
// ---------------------------------------------------------------------------
namespace {

struct DxPlan {
  bool direct;  // straight from the Q4_0 bytes
  Tile tile;
  int pa, pb, splits;
  int64_t rows;  // weight rows, padded
  size_t dy, inv, w, part, total;
};

DxPlan dx_plan(int type, int64_t M, int64_t N, int64_t K, int cus) {
  DxPlan p;
  p.pa = type == TYPE_F32 ? 2 : 1;
  p.pb = 2;  // exact weights: rounded ones show where a sum's terms cancel
  const int units = p.pa + p.pb - 1;
  p.rows = (N + 63) / 64 * 64;
  double best = 1e30;
  for (Tile t : {Tile::T256x256, Tile::T128x128}) {
    for (int s = 1; s <= 16 && (s == 1 || p.rows / s >= 128); ++s) {
      const double us = tile_time_us(t, M, K, p.rows, units, s, cus);
      if (us < best) {
        best = us;
        p.tile = t;
        p.splits = s;
      }
    }
  }
  // the transposed copy: written and read at about 3 TB/s, and its launch
  best += 2.0 * N * K * p.pb * 2 / 3e6 + 3;
  const TransposedPlan d = transposed_plan(M, N, K, units, cus);
  p.direct = d.us < best;
  p.splits = p.direct ? d.splits : even_splits(p.rows / 32, p.splits);
  Carver c;
  p.dy = c.take(static_cast<size_t>(frag_elems(M, p.rows)) * 16 * p.pa);
  p.inv = c.take(static_cast<size_t>(M) * 4);
  p.w = c.take(p.direct ? 0 : static_cast<size_t>(K) * p.rows * 2 * p.pb);
  p.part = c.take(p.direct && p.splits == 1 ? 0 : static_cast<size_t>(p.splits) * M * K * 4);
  p.total = c.at;
  return p;
}

}  // namespace

size_t matmul_dx_workspace_bytes(int type, int64_t M, int64_t N, int64_t K, int cus) {
  return dx_plan(type, M, N, K, cus).total;
}

hipError_t launch_matmul_dx(const uint8_t* w, const void* dy, void* dx, int type, int64_t M,
                            int64_t N, int64_t K, void* ws, int cus, hipStream_t s) {
  const DxPlan p = dx_plan(type, M, N, K, cus);
  char* base = static_cast<char*>(ws);
  f16x8* fa = reinterpret_cast<f16x8*>(base + p.dy);
  float* inv = reinterpret_cast<float*>(base + p.inv);
  f16x8* fb = reinterpret_cast<f16x8*>(base + p.w);
  float* part = reinterpret_cast<float*>(base + p.part);
  hipError_t e = prep_rows(dy, type, Order::NATURAL, fa, inv, M, N, s);
  if (e == hipSuccess && p.direct) {
    TransposedGemm g = {};
    g.g = fa;
    g.pa = p.pa;
    g.pb = p.pb;
    g.type = type;
    g.w = w;
    g.N = N;
    g.M = M;
    g.K = K;
    g.CB = p.rows / 32;
    g.splits = p.splits;
    g.part = p.splits > 1 ? part : nullptr;
    g.inv = inv;
    g.out = dx;
    e = launch_gemm_transposed(g, s);
    if (e == hipSuccess && p.splits > 1) e = launch_fold(part, p.splits, inv, dx, type, M, K, s);
    return e;
  }
  if (e == hipSuccess) e = prep_weights(w, 0, p.rows, N, K, nullptr, nullptr, fb, p.pb, s);
  if (e == hipSuccess) {
    const PlainGemm g = {fa, fb, p.pa, p.pb, M, K, p.rows / 32, p.splits, part, K, nullptr};
    e = launch_gemm_plain(p.tile, g, s);
  }
  if (e == hipSuccess) e = launch_fold(part, p.splits, inv, dx, type, M, K, s);
  return e;
}

}  // namespace q4
