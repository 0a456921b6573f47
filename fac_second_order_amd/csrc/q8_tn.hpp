// What the backward pass and the K-FAC factor make of rows in 8 bits (Osawa et al., CVPR 2019, eq. 5 and 7):
//   dW = sum over rows of g_t^T a_t, db = the sum of g_t,   A = 1/C sum of (a_t, 1)^T (a_t, 1),
// a_t = s_t q_t, over the C rows with s_t != 0.
//
// Both sum over the rows, whose elements lie side by side: operands are staged in LDS a row a
// line and read with the transposing loads, 8 rows of one column a lane. s_t is a power of two,
// so a_t is exact in 16 bits: the products are those of the checkpoint's values, summed in fp32
// by the matrix unit. bf16 gradients meet a_t in bf16. fp16 gradients meet it in fp16, relative
// to the largest scale of the block's rows (exact down to 2^-29 of that). fp32 gradients are cut
// into three bf16 parts of 8 bits each, which is exact, and take three products. The factor is
// formed in integers, rows of one scale after the other.
//
// Rows with s_t = 0 are taken out of a list of the block's rows, before anything of them is
// read: their gradients may hold anything, and cost nothing.
#pragma once
#include "q8.hpp"

namespace kfac {

// One weight gradient, or one layer's factor.
struct TnJob {
  const void* g;  // gradients; the factor has none
  const int8_t* q;
  const float* scale;
  float* out;          // dW, or the packed factor
  float* full;         // the factor's upper triangle in a full matrix, or NULL
  float* bias_out;     // db, or NULL
  float* part;         // [splits][tiles][T * T], with splits > 1
  float* part_col;     // [splits][shares][tile rows][T]: column sums, unless one tile has them (solo)
  int32_t* part_rows;  // [splits]: rows that count, negative if one has a scale that is none
  int64_t ldg, ldq, ldo, inc_b;
  int32_t m, n, rows;  // columns of both operands
  int32_t mt, nt;      // tiles along them
  int32_t tiles, splits, per_split;
  int32_t bias, accumulate;
  float decay;
  int32_t f;       // tiles of 64 f x 64 f; 0: the plain kernel, of gradients
  int32_t any;     // a factor of any columns and pitch (kAny)
  int32_t solo;    // with splits = 1: a row of tiles' first one adds up the columns alone
  int32_t shares;  // who adds up the columns of a row of tiles
  int32_t begin, join_begin;  // first work items
};

template <int N>
struct TnJobs {
  TnJob j[N];
  int32_t n, items, joins;
  __device__ int owner(int item, int32_t TnJob::*first) const {
    int p = 0;
    for (int i = 1; i < n; ++i)
      if (j[i].*first <= item) p = i;
    return __builtin_amdgcn_readfirstlane(p);
  }
};
// A factor call's layers go in the kernels' arguments, this many a launch (under 4 KB).
constexpr int kTnMany = 16;
// Most rows of a block of the factor's tiles of 64 f (of tiles of 128, two blocks share a compute unit's LDS).
constexpr int factor_rows(int f) { return f == 2 ? 4096 : 8192; }
template <bool FACTOR>
using TnArgs = TnJobs<FACTOR ? kTnMany : 1>;

// Tile t of the factor's upper triangle of nb x nb tiles: bands of 4 rows of tiles, each column by column, so that the
// tiles that run at a time on an XCD share the rows of both operands.
__device__ inline void factor_tile(int t, int nb, int& ti, int& tj) {
  int first = 0;
  for (;;) {
    const int left = nb - first, high = min(4, left), corner = high * (high + 1) / 2, all = corner + (left - high) * high;
    if (t < all) {
      int x = 0;
      if (t >= corner) {
        x = high + (t - corner) / high, t = (t - corner) % high;
      } else {
        while (t > x) t -= ++x;
      }
      ti = first + t, tj = first + x;
      return;
    }
    t -= all, first += 4;
  }
}

// Launches of the tile kernels. ragged: columns that are no whole groups of 8 (weight gradients) or 16.
template <class T, int F, bool RAGGED>
kfac_status launch_grad_tiles(const TnArgs<false>& a, hipStream_t s);
kfac_status launch_factor_tiles(const TnArgs<true>& a, int f, bool ragged, hipStream_t s);

}  // namespace kfac
