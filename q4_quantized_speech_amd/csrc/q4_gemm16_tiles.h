// Building blocks of the kernels on prepared binary16 operands (see q4_gemm16.h
// for the operand layout), shared by the translation units that hold them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_gemm16.h"

namespace q4 {

constexpr int XCDS = 8;

// The hardware deals workgroups to the XCDs round-robin; give XCD x a
// contiguous range of tiles, so tiles that share operands share an L2.
__device__ __forceinline__ unsigned xcd_order(unsigned bid, unsigned n) {
  const unsigned per = n / XCDS, rem = n % XCDS, x = bid % XCDS, i = bid / XCDS;
  return (x < rem ? x * (per + 1) : rem * (per + 1) + (x - rem) * per) + i;
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

// A tile of A Q^T with exact codes: sum over the blocks b of scale[n][b]
// (A[m, block b] . Q[n, block b]), `cols` rows of Q.  Row 4 g + v and column
// lane % 16 of the wave's fragments (i, j) in acc[i][j][v]; the wave's first row
// of A and of Q in m0 and c0.
template <typename S, int PA, int KS>
__device__ __forceinline__ void scaled_tile(const f16x8* __restrict__ A, const f16x8* __restrict__ Q,
                                            const float* __restrict__ scale, int64_t M, int64_t cols,
                                            int64_t CB, int tiles_m, f32x4 (&acc)[S::FM][S::FN],
                                            int64_t& m0, int64_t& c0) {
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
  m0 = (ma + wm * S::FM) * 16;
  c0 = (mb + wn * S::FN) * 16;
}

}  // namespace q4
