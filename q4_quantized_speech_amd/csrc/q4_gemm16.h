// Matrix products on prepared binary16 operands: the shared core of the
// Q4_0 gradient product and of the head's cross entropy (internal).
//
// Fragment layout.  A matrix of R rows with a reduction axis of C is stored
// as fragments of 16 rows x 32 reduction indices, 1 KiB each, in the matrix
// cores' operand order: fragment (R / 16 index, C / 32 index), lane
// l = i + 16 g holds row i and eight reduction indices of group g.  Which
// eight is the producer's choice, the same for both operands:
//   NIBBLE   {4g .. 4g+3, 16+4g .. 16+4g+3}: what one dword of Q4_0 codes holds
//   NATURAL  8g .. 8g+7
// A value that binary16 cannot hold is stored as two fragments, hi = its
// rounding and lo = the rounding of the rest.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_device.h"
#include "q4_types.h"

namespace q4 {

enum class Order { NIBBLE, NATURAL };

// Fragments of M x C activations: [ceil(M / 16)][CB] of them, CB = ceil(C / 64)
// * 2 blocks of 32, zeros past M and C, in two copies (hi, then lo) for float32
// and one for the 16-bit types.  Each row of float32 or bfloat16 is scaled by a
// power of two that brings its largest magnitude to [2^14, 2^15); inv[m] is the
// inverse (1 for float16).
hipError_t prep_rows(const void* x, int type, Order order, f16x8* frag, float* inv, int64_t M,
                     int64_t C, hipStream_t s);

inline int64_t blocks32(int64_t c) { return (c + 63) / 64 * 2; }
inline int64_t frag_elems(int64_t rows, int64_t c) { return (rows + 15) / 16 * blocks32(c) * 64; }

// Weight rows [n0, n0 + rows) of a Q4_0 matrix of N rows of K (zeros past N):
//   qfrag  codes q - 8 (exact), NIBBLE over K, [rows / 16][blocks32(K)]
//   scale  float32 block scales, [rows / 16][blocks32(K)][16]
//   tfrag  the transpose, w = (q - 8) d, NATURAL over the rows, `parts` copies
//          of [K / 16][blocks32(rows)]; two parts hold every w exactly
// rows a multiple of 64; qfrag / scale or tfrag may be null.
hipError_t prep_weights(const uint8_t* w, int64_t n0, int64_t rows, int64_t N, int64_t K,
                        f16x8* qfrag, float* scale, f16x8* tfrag, int parts, hipStream_t s);

// Tile shapes.
enum class Tile { T256x256, T128x128 };
struct TileDim {
  int m, n;
};
TileDim tile_dim(Tile t);
// Estimated microseconds of a product of M x N outputs over C reduction
// indices with `units` MFMAs per pair of fragments, on `splits` slices.
double tile_time_us(Tile t, int64_t M, int64_t N, int64_t C, int units, int splits, int cus);

// Slices of CB blocks (even) that all hold some, at most n of them.
inline int even_splits(int64_t CB, int n) {
  const int64_t span = (CB / 2 + n - 1) / n;
  return static_cast<int>((CB / 2 + span - 1) / span);
}

// Hands out 256-byte aligned ranges of a workspace.
struct Carver {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~size_t(255);
    return o;
  }
};

// out[slice][m][n] (+)= sum over the slice's part of the reduction of
// A[m] . B[n], `ld` floats a row: A `pa` parts, B `pb` parts (products hi hi,
// hi lo, lo hi).  alpha (nullable): out = alpha[m] * out + the sum.
struct PlainGemm {
  const f16x8 *a, *b;
  int pa, pb;
  int64_t M, N, CB;  // CB: blocks of 32 reduction indices (even)
  int splits;        // from even_splits
  float* out;
  int64_t ld;
  const float* alpha;
};
hipError_t launch_gemm_plain(Tile t, const PlainGemm& p, hipStream_t s);

// part[slice][m][k] (alpha as above), or with splits == 1 and part null out[m][k]
// = inv[m] * the sum rounded once to `type`: sum over n of G[m, n] deq(W)[n, k]
// for the weight rows [n0, min(N, n0 + 32 CB)), read as Q4_0 (n0 even).
struct TransposedGemm {
  const f16x8* g;
  int pa, pb, type;
  const uint8_t* w;
  int64_t n0, N, M, K, CB;
  int splits;
  float* part;
  const float *alpha, *inv;
  void* out;
  // w2 (nullable): a second matrix of N rows with its own G, two parts of both; its
  // slices follow the first one's in part
  const f16x8* g2;
  const uint8_t* w2;
  int rt;  // with w2: 16-row tiles of a workgroup, 1 to 4 (else 0: transposed_rt(M))
};
struct TransposedPlan {
  double us;  // estimate
  int splits;
};
inline int transposed_rt(int64_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }
TransposedPlan transposed_plan(int64_t M, int64_t N, int64_t K, int units, int cus, int rt = 0);
hipError_t launch_gemm_transposed(const TransposedGemm& p, hipStream_t s);

// Logits of weight rows n0 .. n0 + cols: l[m][n] = inv[m] sum_b scale[n][b]
// (A[m, block b] . (q - 8)[n, block b]), float32 over exact products.  With
// `logits`, [M][ld] floats are written and tmax[m][n / 64 cols] holds the
// maxima of the others than the target; else tmax and tsum hold the maximum
// (the target among them) and the sum of exp(l - maximum) of each 64 columns
// without the target's, and tlogit[m] the target's.
struct LogitGemm {
  const f16x8 *a, *q;
  int pa;
  const float *scale, *inv;
  int64_t M, cols, K, CB;
  int64_t n0, N;
  const int32_t* targets;
  float *logits, *tmax, *tsum, *tlogit;
  int64_t ld, tld;
};
hipError_t launch_gemm_logits(Tile t, const LogitGemm& p, hipStream_t s);

// The same for up to 64 rows, straight from the Q4_0 bytes (q and scale unused;
// n0 even).
constexpr int64_t DIRECT_ROWS = 64;
hipError_t launch_logits_direct(const uint8_t* w, const LogitGemm& p, hipStream_t s);

// dx[m][k] = inv[m] * sum over the slices of part[slice][m][k], rounded once.
hipError_t launch_fold(const float* part, int splits, const float* inv, void* out, int type,
                       int64_t M, int64_t K, hipStream_t s);

}  // namespace q4
