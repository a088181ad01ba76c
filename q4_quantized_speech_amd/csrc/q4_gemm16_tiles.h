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

// The wave's loads to LDS but the latest `N` are complete, and no LDS access moves
// across.
template <int N>
__device__ __forceinline__ void arrived_but() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}
// A barrier alone: what the waves have in flight to LDS stays in flight.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Memory to LDS as to_lds, from lane l's SIZE bytes at base + own + at of a
// range-checked buffer (own: the lane's offset, at: the wave's).  Beside these
// loads the compiler counts LDS reads one by one; beside to_lds it waits for all
// of them each time.
template <int SIZE>
__device__ __forceinline__ void buffer_to_lds(__amdgpu_buffer_rsrc_t base, int own, int at, void* l) {
  const auto lp = (__attribute__((address_space(3))) void*)l;
  if constexpr (SIZE == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(base, lp, 16, own, at, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(base, lp, 4, own, at, 0, 0);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00020000);
}

// A tile of A Q^T with exact codes: sum over the blocks b of scale[n][b]
// (A[m, block b] . Q[n, block b]), `cols` rows of Q.  Row 4 g + v and column
// lane % 16 of the wave's fragments (i, j) in acc[i][j][v]; the wave's first row
// of A and of Q in m0 and c0.
//
// A ring of NB stages of one block each.  When stage c begins, stage c + NB - 1
// is asked for and stage c + 1 is already there, so its first operands are read
// before c ends and a barrier finds work on both sides of it.
template <typename S, int PA>
__device__ __forceinline__ void scaled_tile(const f16x8* __restrict__ A, const f16x8* __restrict__ Q,
                                            const float* __restrict__ scale, int64_t M, int64_t cols,
                                            int64_t CB, int tiles_m, f32x4 (&acc)[S::FM][S::FN],
                                            int64_t& m0, int64_t& c0) {
  using St = Stage<S, PA, 1, 1>;
  constexpr int NB = PA == 1 ? 4 : 3, FM = S::FM, FN = S::FN;
  constexpr int SC = S::N;  // block scales of a stage, [row tile][16]
  static_assert(St::NF % St::WAVES == 0 && SC / 64 <= St::WAVES && FM % 4 == 0, "");
  // arrays of their own rather than one of all: the compiler then knows that
  // reading one does not have to wait for loads into the others
  __shared__ f16x8 buf0[St::NF][64], buf1[St::NF][64], buf2[St::NF][64], buf3[NB == 4 ? St::NF : 1][64];
  // (the waves past SC / 64 load scales in vain, so that all have as many loads
  // in flight)
  constexpr int SL = 64 * St::WAVES;
  __shared__ float sc0[SL], sc1[SL], sc2[SL], sc3[NB == 4 ? SL : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned item = xcd_order(blockIdx.x, gridDim.x);
  const int tm = item % tiles_m, tn = item / tiles_m;
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int64_t ma = static_cast<int64_t>(tm) * (S::M / 16), mb = static_cast<int64_t>(tn) * (S::N / 16);
  const int64_t rta = (M + 15) / 16, rtb = cols / 16;

#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const St st(A, Q, ma, rta, mb, rtb, CB, wave);
  __amdgpu_buffer_rsrc_t from[St::PER];
#pragma unroll
  for (int u = 0; u < St::PER; ++u) from[u] = buffer(st.at[u], CB * 1024);
  const int tiles = static_cast<int>(min<int64_t>(S::N / 16, rtb - mb));  // that have scales
  const __amdgpu_buffer_rsrc_t scales = buffer(scale + mb * CB * 16, tiles * CB * 64);
  const int own = min(wave * 4 + lane / 16, tiles - 1) * static_cast<int>(CB) * 64 + lane % 16 * 4;
  auto buf = [&](auto k) {
    constexpr int K = decltype(k)::value;
    if constexpr (K == 0) return buf0;
    else if constexpr (K == 1) return buf1;
    else if constexpr (K == 2) return buf2;
    else return buf3;
  };
  auto sc = [&](auto k) {
    constexpr int K = decltype(k)::value;
    if constexpr (K == 0) return sc0;
    else if constexpr (K == 1) return sc1;
    else if constexpr (K == 2) return sc2;
    else return sc3;
  };
  // past the last stage: it again, so that the loads in flight can be counted
  auto fill = [&](auto k, int64_t c) {
    const int at = static_cast<int>(min(c, CB - 1)) * 1024;
#pragma unroll
    for (int u = 0; u < St::PER; ++u) buffer_to_lds<16>(from[u], lane * 16, at, &buf(k)[wave * St::PER + u][0]);
    buffer_to_lds<4>(scales, own, at / 16, sc(k) + wave * 64);
    issued();
  };
  f16x8 a[4][PA], b[2][FN];
  float d[2][FN];
  f32x4 t[2][FN];
  auto load_a = [&](const f16x8 (*from)[64], int i) {
#pragma unroll
    for (int p = 0; p < PA; ++p) a[i % 4][p] = from[p * S::WM * FM + wm * FM + i % FM][lane];
  };
  auto load_b = [&](const f16x8 (*from)[64], const float* s, int k) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      b[k][j] = from[St::FA + wn * FN + j][lane];
      d[k][j] = s[(wn * FN + j) * 16 + (lane & 15)];
    }
  };
  auto products = [&](int i, int k) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
      t[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[i % 4][0], b[k][j], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
    if constexpr (PA == 2)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        t[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[i % 4][1], b[k][j], t[i & 1][j], 0, 0, 0);
    asm volatile("" : "+v"(t[i & 1][0]), "+v"(t[i & 1][1]), "+v"(t[i & 1][2]), "+v"(t[i & 1][3])::"memory");
  };
  // Stage c in buffer k: row i + 1's products are started before row i's scaled
  // sums are taken, so the matrix cores and the vector unit overlap within the
  // wave, and operands are read from LDS two rows (B and its scales half a
  // stage) ahead, at a stage's end from the next one's buffer (past the last
  // stage they are read in vain).  The empty volatile asm keeps that order (pure
  // arithmetic would otherwise be regrouped, all products first, whose
  // temporaries then spill).
  auto stage = [&](auto k, auto par, int64_t c) {
    constexpr int K = decltype(k)::value, P = decltype(par)::value;
    const std::integral_constant<int, (K + 1) % NB> next;
    const std::integral_constant<int, (K + NB - 1) % NB> last;
    // stage c + 1 is there, and all waves are past stage c - 1
    arrived_but<(NB - 3) * (St::PER + 1)>();
    meet();
    fill(last, c + NB - 1);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (i + 3 < FM) load_a(buf(k), i + 3);
      else load_a(buf(next), i + 3);
      if (i == FM / 2 - 1) load_b(buf(next), sc(next), P ^ 1);
      __builtin_amdgcn_sched_barrier(0);  // the reads stay ahead of the products
      products(i + 1, i + 1 < FM ? P : P ^ 1);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        acc[i][j].x = __builtin_fmaf(d[P][j], t[i & 1][j].x, acc[i][j].x);
        acc[i][j].y = __builtin_fmaf(d[P][j], t[i & 1][j].y, acc[i][j].y);
        acc[i][j].z = __builtin_fmaf(d[P][j], t[i & 1][j].z, acc[i][j].z);
        acc[i][j].w = __builtin_fmaf(d[P][j], t[i & 1][j].w, acc[i][j].w);
      }
      asm volatile("" : "+v"(acc[i][0]), "+v"(acc[i][1]), "+v"(acc[i][2]), "+v"(acc[i][3]));
    }
  };
  using std::integral_constant;
  const integral_constant<int, 0> z0;
  const integral_constant<int, 1> z1;
  const integral_constant<int, 2> z2;
  const integral_constant<int, 3> z3;
  fill(z0, 0);
  fill(z1, 1);
  if constexpr (NB == 4) fill(z2, 2);
  arrived();
  meet();
  load_b(buf0, sc0, 0);
  load_a(buf0, 0);
  load_a(buf0, 1);
  load_a(buf0, 2);
  products(0, 0);
  int64_t c = 0;  // (CB is even)
  if constexpr (NB == 4) {
    for (; c + 4 <= CB; c += 4) {
      stage(z0, z0, c);
      stage(z1, z1, c + 1);
      stage(z2, z0, c + 2);
      stage(z3, z1, c + 3);
    }
    if (c < CB) {
      stage(z0, z0, c);
      stage(z1, z1, c + 1);
    }
  } else {
    for (; c + 6 <= CB; c += 6) {
      stage(z0, z0, c);
      stage(z1, z1, c + 1);
      stage(z2, z0, c + 2);
      stage(z0, z1, c + 3);
      stage(z1, z0, c + 4);
      stage(z2, z1, c + 5);
    }
    if (c < CB) {
      stage(z0, z0, c);
      stage(z1, z1, c + 1);
    }
    if (c + 2 < CB) {
      stage(z2, z0, c + 2);
      stage(z0, z1, c + 3);
    }
  }
  arrived();  // the loads in vain: LDS may be another workgroup's after this one
  m0 = (ma + wm * FM) * 16;
  c0 = (mb + wn * FN) * 16;
}

}  // namespace q4
