// Kronecker factors from rows in 8 bits, in 8-bit integers.
//
// a_t = s_t q_t with powers of two s_t, so that rows of one scale add up in integers:
//   A = 1/C sum over the scales of s^2 (sum over its rows of q q^T).
// A block sorts its rows by their scales, largest first, and forms the inner sums on the matrix unit's 8-bit
// products, twice the rate of 16 bits, exactly in 32 bits. From one scale to the next, 2^e times smaller, the
// sums are multiplied by 4^e, as long as that and the rows to come stay within 32 bits: by the rows' number and
// the largest code first, and where that does not show it, by the sums themselves. Where they would not, they
// are added to fp32 in the workspace. A layer's rows lie within some octaves, and most layers need none
// of that: a factor's error is that of a few roundings, however many its rows. Rows whose scale is no power of
// two make the factor NaN.
//
// Tiles of T x T, T = 64 F, of the upper triangle; four waves of 32 F x 32 F; steps of 64 rows, one scale each, which go
// from memory into registers three steps ahead and from there into LDS one step ahead, a row a line
// of T bytes. The transposing loads give a lane 8 rows of a column; the groups of 16 bytes of a
// line are moved so that the 8 rows that 32 lanes meet lie in different banks.
//
// 8192 x 4096, 5564 rows of which count: 97 us with tiles of 192 (253 tiles, a block each; 0.96e15 operations a second),
// 113 + 23 with 128, 170 with 64; in 16 bits with the scales multiplied in it took 155 + 22. What bounds it are the
// waits of the one wave a SIMD: the matrix unit is busy for a quarter of the time, LDS for
// another, and fetching four steps ahead (119) brings nothing. Tiles of 256 spill when the sums change their
// scale. Small factors take tiles of 64 (32 x 2048: 14 us, 19 and 30 with larger ones), sets of layers
// one edge for all.
#include "q8_tn_kernel.hpp"

namespace kfac {

constexpr int kFactorStep = 64, kFactorAhead = 3;

template <int F>
struct FactorTile {
  static constexpr int T = 64 * F;
  static constexpr int FETCH = kFactorStep * T / 16 / 256;  // groups of 16 codes of an operand, a thread
  static constexpr int OPERAND = kFactorStep * T, GROUPS = T / 16, LIST = factor_rows(F);
  // every scale may end in a step that is not full; behind them steps of no rows, which are fetched and not used
  static constexpr int STEPS = LIST / kFactorStep + 254 + kFactorAhead + 3;
  static __device__ inline int moved(int row) {
    return 2 * (F == 2 ? (row >> 1) & 3 : (row >> 2) & 1);
  }
};

// A block's rows by their scales.
template <int F>
struct SortedRows {
  uint16_t idx[FactorTile<F>::LIST + kFactorStep];  // a step that is not full reads on
  uint32_t step[FactorTile<F>::STEPS];  // a step's first row in idx, and how many it has in the low 7 bits
  float s[FactorTile<F>::STEPS];        // its scale
  uint16_t n[FactorTile<F>::STEPS];     // and how many rows have that
  int32_t count[256], at[256];
  int32_t waves[4][2];
};

// The class of a scale: its exponent, 255 if it is no power of two (or none at all: NaN), -1 for 0.
__device__ inline int scale_class(float s) {
  const unsigned b = __float_as_uint(s);
  if ((b & 0x7fffffffu) == 0) return -1;
  return b & 0x807fffffu || b < 0x00800000u ? 255 : static_cast<int>(b >> 23);
}

// Sorts the rows of [r0, r0 + n). Returns the steps; adds the rows that count to `counted`, and sets `bad` if one
// has no power of two.
template <int F>
__device__ inline int sort_rows(const float* scale, int64_t r0, int n, SortedRows<F>& l, int& counted, bool& bad) {
  constexpr int PER = FactorTile<F>::LIST / 256;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float s[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) s[i] = tid + 256 * i < n ? gp(scale)[r0 + tid + 256 * i] : 0.f;
  l.count[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (256 * i >= n) break;
    const int c = scale_class(s[i]);
    if (c >= 0) atomicAdd(&l.count[c], 1);
  }
  __syncthreads();
  bad |= l.count[255] != 0;
  // thread t has class 254 - t: its steps and rows behind those of the threads before
  const int cls = 254 - tid, own = cls > 0 ? l.count[cls] : 0, steps = (own + kFactorStep - 1) / kFactorStep;
  int step_sum = steps, row_sum = own;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int up = __shfl_up(step_sum, o), rows_up = __shfl_up(row_sum, o);
    if (lane >= o) step_sum += up, row_sum += rows_up;
  }
  if (lane == 63) l.waves[wave][0] = step_sum, l.waves[wave][1] = row_sum;
  __syncthreads();
  int first = step_sum - steps, row = row_sum - own, all = 0, live = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) first += l.waves[w][0], row += l.waves[w][1];
    all += l.waves[w][0], live += l.waves[w][1];
  }
  if (cls > 0) l.at[cls] = row;
  for (int k = 0; k < steps; ++k) {
    l.step[first + k] = static_cast<uint32_t>(row + k * kFactorStep) << 7 | min(own - k * kFactorStep, kFactorStep);
    l.s[first + k] = __uint_as_float(static_cast<unsigned>(cls) << 23);
    l.n[first + k] = static_cast<uint16_t>(own);
  }
  if (steps && first + steps == all)  // the last scale's
    for (int k = 0; k < kFactorAhead + 3; ++k) l.step[all + k] = 0, l.s[all + k] = l.s[all - 1], l.n[all + k] = 0;
  __syncthreads();
  // the order within a class is that of the atomics: its whole sum is exact, and no part of it is rounded
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (256 * i >= n) break;
    const int c = scale_class(s[i]);
    if (c > 0 && c < 255) l.idx[atomicAdd(&l.at[c], 1)] = static_cast<uint16_t>(tid + 256 * i);
  }
  __syncthreads();
  counted += live + (bad ? 1 : 0);
  return all;
}

// 16 codes as they come from memory.
struct Raw16 {
  v4u w;
  __device__ inline void load(const KG char* p) {
    w = __builtin_bit_cast(v4u, load_pack<false, int8_t>(reinterpret_cast<const KG int8_t*>(p)));
  }
  __device__ inline v4u codes(int, int) const { return w; }
  __device__ inline void shift(int k) {  // drops the first k
    uint64_t lo = uint64_t(w[1]) << 32 | w[0], hi = uint64_t(w[3]) << 32 | w[2];
    const int b = 8 * (k & 7);
    if (k & 8) lo = hi, hi = 0;
    lo = lo >> b | (b ? hi << (64 - b) : 0);
    hi >>= b;
    w = v4u{unsigned(lo), unsigned(lo >> 32), unsigned(hi), unsigned(hi >> 32)};
  }
};

// The first n of 16 codes, 0 <= n <= 16, and zeros, by loads from both ends that may overlap: nothing behind them is read.
// In rows of fewer than 16 columns, `row` of them and not 0, n is that or 0, and what is to be done the same for all lanes.
struct Raw16Some {
  uint64_t a, b;
  unsigned c;
  template <int N>
  static __device__ inline uint64_t bytes(const KG char* p) {
    uint64_t w = 0;
    const auto v = load_pack<false, int8_t, N>(reinterpret_cast<const KG int8_t*>(p));
    __builtin_memcpy(&w, &v, N);
    return w;
  }
  __device__ inline void load_n(const KG char* p, int n) {
    if (n >= 8) a = bytes<8>(p), b = bytes<8>(p + n - 8);
    else if (n >= 4) a = bytes<4>(p), b = bytes<4>(p + n - 4);
    else if (n > 0) a = uint8_t(p[0]), b = uint8_t(p[n / 2]), c = uint8_t(p[n - 1]);
  }
  __device__ inline v4u codes_n(int n) const {
    uint64_t lo = a, hi = 0;
    if (n > 8) hi = b >> (8 * (16 - n));
    else if (n >= 4) lo |= n < 8 ? b << (8 * (n - 4)) : 0;
    else if (n > 0) lo |= b << (8 * (n / 2)) | uint64_t(c) << (8 * (n - 1));
    return v4u{unsigned(lo), unsigned(lo >> 32), unsigned(hi), unsigned(hi >> 32)};
  }
  __device__ inline void load(const KG char* p, int n, int row) {
    a = 0, b = 0, c = 0;
    if (!row) load_n(p, n);
    else if (n) load_n(p, row);
  }
  __device__ inline v4u codes(int n, int row) const { return row ? codes_n(row) : codes_n(n); }
};

// COLS: how the columns are read. kWhole: in groups of 16; kRagged: the last group of a row shifted; kAny, in tiles
// of 64: as many of a group as there are, for rows of fewer than 16 columns or 2^32 bytes and more apart (100352 x 8:
// 28 us, 1000 x 12: 16; a row of one 8.4 by itself, of 16 in one group 7.1: the loads' cases).
enum { kWhole, kRagged, kAny };

template <int F, int COLS>
__global__ void __launch_bounds__(256, F == 3 ? 1 : 2) factor_q8_kernel(TnArgs<true> args) {
  constexpr bool RAGGED = COLS == kRagged;
  using L = FactorTile<F>;
  constexpr int T = L::T, G = L::FETCH, BUFS = kFactorAhead;
  __shared__ __attribute__((aligned(16))) char lds[2 * BUFS * L::OPERAND];
  __shared__ SortedRows<F> list;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int v = xcd_virtual(blockIdx.x, gridDim.x, args.items);
  if (v < 0) return;
  const TnJob& d = args.j[args.owner(v, &TnJob::begin)];
  const int item = v - d.begin, split = item / d.tiles, tile = item - split * d.tiles;
  int ti, tj;
  factor_tile(tile, d.mt, ti, tj);
  const int64_t r_begin = int64_t(split) * d.per_split;
  const int r_count = static_cast<int>(min(int64_t(d.per_split), d.rows - r_begin));
  char* const abuf = lds;
  char* const bbuf = lds + BUFS * L::OPERAND;
  const bool same = COLS == kAny && ti == tj;  // one operand is both

  // this thread's groups of 16 columns: row of a step, place in its line, offset in its rows, codes to shift out (kAny:
  // columns that there are)
  int row[G], at[G], a_col[G], b_col[G], a_cut[G], b_cut[G];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int u = tid + 256 * i, c = 16 * (u % L::GROUPS);
    row[i] = u / L::GROUPS;
    at[i] = row[i] * T + 16 * ((u % L::GROUPS) ^ L::moved(row[i]));
    auto column = [&](int c, int& off, int& cut) {
      if constexpr (COLS == kAny) {
        cut = max(0, min(16, d.m - c)), off = cut ? c : 0;
        return;
      }
      off = c + 16 <= d.m ? c : RAGGED && c < d.m ? d.m - 16 : 0;
      cut = RAGGED && c < d.m && c + 16 > d.m ? c + 16 - d.m : 0;
    };
    column(ti * T + c, a_col[i], a_cut[i]);
    column(tj * T + c, b_col[i], b_cut[i]);
  }
  [[maybe_unused]] bool cuts = false;  // of the wave: only the last tiles of ragged operands have any
  if constexpr (RAGGED) {
#pragma unroll
    for (int i = 0; i < G; ++i) cuts |= (a_cut[i] | b_cut[i]) != 0;
    cuts = __any(cuts);
  }
  using Raw = std::conditional_t<COLS == kAny, Raw16Some, Raw16>;
  Raw araw[kFactorAhead][G], braw[kFactorAhead][G];

  const int wm = (wave >> 1) * 32 * F, wn = (wave & 1) * 32 * F;
  v16i acc[F][F];
  int isum[F];
  float sums[F];
#pragma unroll
  for (int i = 0; i < F; ++i) {
    isum[i] = 0, sums[i] = 0.f;
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = v16i{};
  }
  // Column sums, by the diagonal tiles: of a block's two waves that hold the same columns one has the even groups of 32
  // and the other the odd ones. A wave has all rows of its columns, so that what is rounded is a whole scale's sum,
  // which does not know the rows' order. (Not tiles in turns: each block has its own order of rows.)
  const bool sums_here = d.bias && tj == ti;
  const int sums_at = sums_here ? wave & 1 : -1;  // its first group
  const int s16 = lane & 15, kk = 16 * (lane >> 5) + (s16 >> 1), cc = 16 * ((lane >> 4) & 1) + 8 * (s16 & 1);
  const char* fa_at[F];
  const char* fb_at[F];
#pragma unroll
  for (int i = 0; i < F; ++i) {
    auto place = [&](int c) { return kk * T + 16 * (((c + cc) >> 4) ^ L::moved(kk)) + (cc & 15); };
    fa_at[i] = abuf + place(wm + 32 * i);
    fb_at[i] = (same ? abuf : bbuf) + place(wn + 32 * i);
  }
  typedef int v2i __attribute__((ext_vector_type(2)));
  typedef v2i __attribute__((address_space(3))) lds_v2i;
  auto operand = [&](const char* from) {  // 16 rows of a column each lane; rows 8 apart are moved alike
    const v2i lo = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)from);
    const v2i hi = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)(from + 8 * T));
    return v4i{lo[0], lo[1], hi[0], hi[1]};
  };
  KG float* const part = uniform(gp(d.part) + (int64_t(split) * d.tiles + tile) * (T * T));
  const int narrow = COLS == kAny && d.m < 16 ? d.m : 0;
  bool flushed = false, bad = false;
  int counted = 0;
  const int steps = sort_rows<F>(d.scale, r_begin, r_count, list, counted, bad);
  float s_here = steps ? uniform(list.s[0]) : 1.f;  // scale of the sums' rows
  // times this the largest scale is 1: what lies far below it may be lost in sums that are 2^126 times larger, no sooner
  const float unit = __uint_as_float(max(1, 254 - static_cast<int>(__float_as_uint(s_here) >> 23)) << 23);
  uint64_t bound = 0, bound_col = 0;  // of the magnitudes of this wave's sums, and of those of columns
  // a lane's accumulators of (i, j): column 32 j + lane % 32 of the wave, rows 32 i + 8 (e / 4) + 4 (lane / 32) + e % 4
  const int lane_at = (wm + 4 * (lane >> 5)) * T + wn + (lane & 31);
  auto entry = [](int i, int j, int e) { return (32 * i + 8 * (e >> 2) + (e & 3)) * T + 32 * j; };
  // the sum of columns i, of rows of scale rel, to fp32: the lanes' halves, which have 16 rows each in turn, first
  auto add_columns = [&](int i, float rel) __attribute__((always_inline)) {
    sums[i] = fmaf(static_cast<float>(isum[i] + __shfl_xor(isum[i], 32)), rel, sums[i]);
  };
  // the sums, of rows of scale s, to fp32
  auto flush = [&](float s) __attribute__((always_inline)) {
    const float rel = s * unit, rel2 = rel * rel;
    unsigned here = lane_at;
    asm volatile("" : "+v"(here));  // addresses are formed here, not kept over the loop
#pragma unroll
    for (int i = 0; i < F; ++i) {
      add_columns(i, rel);
#pragma unroll
      for (int j = 0; j < F; ++j) {
        const v16f all = __builtin_convertvector(acc[i][j], v16f) * rel2;
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          KG float* const o = part + entry(i, j, e);
          v4f x{all[e], all[e + 1], all[e + 2], all[e + 3]};
          if (flushed) {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] += o[here + k * T];
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) o[here + k * T] = x[k];
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    flushed = true;
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): so that the loop's own loads are counted as without this
  };
  // the largest magnitude of the wave's sums
  auto largest = [&]() __attribute__((always_inline)) {
    int high = 0, low = 0;
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) {
        const v16i x = acc[i][j];
#pragma unroll
        for (int e = 0; e < 16; ++e) high = max(high, x[e]), low = min(low, x[e]);
        __builtin_amdgcn_sched_barrier(0);
      }
    high = max(high, -low);  // less than 2^31
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) high = max(high, __shfl_xor(high, o));
    return static_cast<uint64_t>(uniform(high));
  };
  using Pitch = std::conditional_t<COLS == kAny, uint64_t, unsigned>;
  const Pitch pitch = static_cast<Pitch>(d.ldq);
  if (steps) {
    const KG char* const q0 = uniform(reinterpret_cast<const KG char*>(gp(d.q)) + r_begin * d.ldq);
    unsigned some[kFactorAhead][G];  // of what the registers hold: ~0, or 0 for no row
    // this thread's rows of a step (none: row 0, and `some` is 0), by what list.step says of it
    auto rows_of = [&](uint32_t said, int (&r)[G], unsigned (&some)[G]) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        some[i] = static_cast<unsigned>((row[i] - static_cast<int>(said & 127)) >> 31);
        r[i] = static_cast<int>(list.idx[(said >> 7) + row[i]] & some[i]);
      }
    };
    auto fetch = [&](auto set, int k, const int (&r)[G]) {  // 2 G loads
      const int i = k / 2;
      const KG char* from = q0 + uint64_t(unsigned(r[i])) * pitch;
      if constexpr (COLS == kAny) {
        if (k & 1) araw[set][i].load(from + a_col[i], a_cut[i], narrow);
        else if (!same) braw[set][i].load(from + b_col[i], b_cut[i], narrow);
      } else {
        if (k & 1) araw[set][i].load(from + a_col[i]);
        else braw[set][i].load(from + b_col[i]);
      }
    };
    auto place = [&](auto set, auto buf, int k) {
      const int i = k / 2;
      if (same && !(k & 1)) return;
      Raw& x = k & 1 ? araw[set][i] : braw[set][i];
      if constexpr (RAGGED)
        if (cuts) x.shift(k & 1 ? a_cut[i] : b_cut[i]);
      *reinterpret_cast<v4u*>((k & 1 ? abuf : bbuf) + buf * L::OPERAND + at[i]) = x.codes(k & 1 ? a_cut[i] : b_cut[i], narrow) & some[set][i];
    };
    v4i fa[2][F], fb[2][F];
    constexpr int R = 2 * F, MN = F * F;
    auto read = [&](auto buf, int ks, int set, int k) {
      if (k < F) fb[set][k] = operand(fb_at[k] + buf * L::OPERAND + 32 * ks * T);
      else fa[set][k - F] = operand(fa_at[k - F] + buf * L::OPERAND + 32 * ks * T);
    };
    auto mma = [&](int set, int n) {
      acc[n / F][n % F] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[set][n / F], fb[set][n % F], acc[n / F][n % F], 0, 0, 0);
    };
    auto add_up = [&](auto FIRST) {  // its groups of columns, FIRST, FIRST + 2, ..
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int set = 0; set < 2; ++set)
#pragma unroll
          for (int i = decltype(FIRST)::value; i < F; i += 2)
            isum[i] = __builtin_amdgcn_sdot4(fa[set][i][k], 0x01010101, isum[i], false);
    };
#define KFAC_AT(x) std::integral_constant<int, (x)>{}
    int r[G];
    auto first = [&](auto s) {
      rows_of(list.step[s], r, some[s]);
#pragma unroll
      for (int k = 0; k < 2 * G; ++k) fetch(s, k, r);
    };
    first(KFAC_AT(0));
    first(KFAC_AT(1));
    first(KFAC_AT(2));
    uint32_t said = list.step[kFactorAhead];
#pragma unroll
    for (int k = 0; k < 2 * G; ++k) place(KFAC_AT(0), KFAC_AT(0), k);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < R; ++k) read(KFAC_AT(0), 0, 0, k);
    bound = uint64_t(uniform(list.n[0])) << 14, bound_col = bound >> 7;
    int c = 0;
    bool edge = false;  // the next step's rows have another scale
    // One step, as in the weight gradient's kernel: the products of its first 32 rows, with the other rows'
    // operands read and the next step placed behind them; those of the other rows, with the next step's first
    // operands read and step c + 3 fetched. Behind the last step come steps of no rows.
    auto step = [&](auto S) __attribute__((always_inline)) {
      constexpr int s = decltype(S)::value;
      constexpr int K = R + 2 * G;
      float s_next = 0.f;
      unsigned fetched[G];
#pragma unroll
      for (int n = 0; n < MN; ++n) {
        mma(0, n);
        if (n == MN / 2) {
          s_next = list.s[c + 1];
          rows_of(said, r, fetched);
        }
#pragma unroll
        for (int k = n * K / MN; k < (n + 1) * K / MN; ++k) {
          if (k < R) read(KFAC_AT(s), 1, 1, k);
          else place(KFAC_AT((s + 1) % BUFS), KFAC_AT((s + 1) % BUFS), k - R);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (sums_at == 0) add_up(KFAC_AT(0));
      else if (sums_at == 1) add_up(KFAC_AT(1));
      __syncthreads();
#pragma unroll
      for (int n = 0; n < MN; ++n) {
        mma(1, n);
        if (n == MN / 2) said = list.step[min(c + 1 + kFactorAhead, steps + kFactorAhead)];
#pragma unroll
        for (int k = n * K / MN; k < (n + 1) * K / MN; ++k) {
          if (k < R) read(KFAC_AT((s + 1) % BUFS), 0, 0, k);
          else fetch(KFAC_AT(s), k - R, r);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < G; ++i) some[s][i] = fetched[i];
      ++c;
      edge = uniform(s_next) != s_here;
    };
    // from rows of one scale to those of the next: the sums times 4^by, or to fp32
    auto change = [&]() __attribute__((always_inline)) {
      const float s_next = uniform(list.s[c]);
      const int by = static_cast<int>(__float_as_uint(s_here) >> 23) - static_cast<int>(__float_as_uint(s_next) >> 23);
      const uint64_t rows = uint64_t(uniform(list.n[c])) << 14;
      auto fits_in = [&](uint64_t sums) {
        return by >= 0 && by < 16 && (sums << (2 * by)) + rows < (uint64_t(1) << 31) &&
               (bound_col << by) + (rows >> 7) < (uint64_t(1) << 31);
      };
      bool fits = fits_in(bound);
      if (!fits) {  // what the sums have come to, instead of what they might
        bound = largest();
        fits = fits_in(bound);
      }
      if (!fits) flush(s_here);
      const int keep = fits ? -1 : 0, up = fits ? by : 0;
      bound = (fits ? bound << (2 * by) : 0) + rows;
      bound_col = (fits ? bound_col << by : 0) + (rows >> 7);
#pragma unroll
      for (int i = 0; i < F; ++i) {
        isum[i] = (isum[i] & keep) << up;
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = (acc[i][j] & keep) << (2 * up);
      }
      s_here = s_next;
    };
    do {  // up to two of the steps are of no rows
      step(KFAC_AT(0));
      if (edge) change();
      step(KFAC_AT(1));
      if (edge) change();
      step(KFAC_AT(2));
      if (edge) change();
    } while (c < steps);
#undef KFAC_AT
  }

  const float back = 1.f / unit;  // exact: a power of two
  const float inv_r = counted ? 1.f / static_cast<float>(counted) : 0.f;
  const float rel = bad ? __uint_as_float(0x7fc00000u) : s_here * unit, rel2 = rel * rel;
  const PutFactor put = put_factor(d, counted);
  if (d.part_rows && tile == 0 && tid == 0) gp(d.part_rows)[split] = bad ? -counted : counted;  // somebody joins
  unsigned here = lane_at;
  asm volatile("" : "+v"(here));
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) {
      v16f x = __builtin_convertvector(acc[i][j], v16f) * rel2;
      KG float* const o = part + here + entry(i, j, 0);
      if (flushed) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] += o[entry(0, 0, e)];
      }
      x *= back;
      x *= back;
      if (d.splits > 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e) o[entry(0, 0, e)] = x[e];
      } else {
        const int c = tj * T + wn + 32 * j + (lane & 31);
        int rs[16], cs[16];
        bool live[16];
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          rs[e] = ti * T + wm + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3), cs[e] = c;
          live[e] = rs[e] <= c && c < d.n, v[e] = x[e] * inv_r;
        }
        put.all(rs, cs, live, v);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  if (!sums_here) return;
  KG float* const col = d.solo ? nullptr : gp(d.part_col) + int64_t(split) * (int64_t(d.mt) * T);
#pragma unroll
  for (int i = 0; i < F; ++i) {
    add_columns(i, rel);
    const float sum = sums[i] * back;
    const int c = ti * T + wm + 32 * i + lane;
    if ((i & 1) != sums_at || lane >= 32) continue;
    if (!d.solo) {
      col[c] = sum;
    } else if (c < d.m) {
      put(c, d.m, sum * inv_r);
      if (c == 0) put(d.m, d.m, corner(counted, bad));
    }
  }
}

template <int F, int COLS>
static kfac_status launch(const TnArgs<true>& a, hipStream_t s) {
  KFAC_LAUNCH(K_FACTOR_Q8, (factor_q8_kernel<F, COLS>), dim3(xcd_grid(a.items)), dim3(256), 0, s, a);
  KFAC_CHECK_LAUNCH("factor_q8_kernel");
  return KFAC_OK;
}

kfac_status launch_factor_tiles(const TnArgs<true>& a, int f, bool ragged, hipStream_t s) {
  if (a.j[0].any) return launch<1, kAny>(a, s);
  if (f == 1) return ragged ? launch<1, kRagged>(a, s) : launch<1, kWhole>(a, s);
  if (f == 2) return ragged ? launch<2, kRagged>(a, s) : launch<2, kWhole>(a, s);
  return ragged ? launch<3, kRagged>(a, s) : launch<3, kWhole>(a, s);
}

}  // namespace kfac
