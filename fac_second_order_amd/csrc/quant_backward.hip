// Weight gradients and Kronecker factors from rows in 8 bits: the plain kernel of gradients, what joins the parts of
// the tiles, and the entry points.
#include "q8_tn_kernel.hpp"

namespace kfac {

constexpr int kSmallList = 2048;

// Groups of 8 columns of a step's BK rows x TC columns, NT threads.
template <class E, int TC, int NT, int BK>
struct Stage {
  static constexpr int perRow = TC / 8, N = perRow * BK / NT;
  using Raw = std::conditional_t<std::is_same_v<E, int8_t>, v2u, std::conditional_t<std::is_same_v<E, float>, v8f, v8s>>;
  Raw v[N];

  static __device__ inline int row(int i) { return (threadIdx.x + i * NT) / perRow; }
  static __device__ inline int col(int i) { return (threadIdx.x + i * NT) % perRow * 8; }

  // rows l.idx[k0 ..] + r0 of src, columns c0 .. of cols
  template <int LIST>
  __device__ inline void load(const E* src, int64_t ld, int64_t r0, const RowList<LIST>& l, int k0, int c0, int cols) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint16_t r = l.idx[k0 + row(i)];
      const int c = c0 + col(i);
      const KG E* p = gp(src) + (r0 + (r & (kNone - 1))) * ld + c;
      if (r != kNone && c + 8 <= cols) {
        if constexpr (std::is_same_v<E, int8_t>) {
          v[i] = __builtin_bit_cast(Raw, *reinterpret_cast<const KG typename Pack<int8_t, 8>::vec*>(p));
        } else if constexpr (std::is_same_v<E, float>) {
          const v4f a = load_pack<false, float>(p), b = load_pack<false, float>(p + 4);
          v[i] = Raw{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        } else {
          v[i] = __builtin_bit_cast(Raw, load_pack<false, short>(reinterpret_cast<const KG short*>(p)));
        }
      } else {
        v[i] = Raw{};
        if (r != kNone)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k < cols) {
              if constexpr (std::is_same_v<E, int8_t>) v[i][k >> 2] |= unsigned(uint8_t(p[k])) << (8 * (k & 3));
              else if constexpr (std::is_same_v<E, float>) v[i][k] = p[k];
              else v[i][k] = reinterpret_cast<const KG short*>(p)[k];
            }
      }
    }
  }
};

// The plain kernel: any sizes and pitches, tiles of 128 x 128, a step's rows staged and then multiplied. For
// operands of fewer than 8 columns, and rows 2^32 bytes and more apart.
template <class T>
__global__ void __launch_bounds__(256) q8_plain_kernel(TnJob d) {
  constexpr int TM = 128, TN = 128, NT = 256, BK = 32, PITCH = 128 + 32, P = kParts<T>;
  constexpr bool HALF = std::is_same_v<T, _Float16>;
  __shared__ __attribute__((aligned(16))) short lds[P + 1][BK][PITCH];
  __shared__ RowList<kSmallList> list;
  __shared__ float colsum[TM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tile = blockIdx.x % d.tiles, split = blockIdx.x / d.tiles;
  const int ti = tile / d.nt, tj = tile % d.nt;
  const int64_t r_begin = int64_t(split) * d.per_split;
  const int r_count = static_cast<int>(min(int64_t(d.per_split), d.rows - r_begin));
  const bool sums = d.bias && tj == 0;  // this block adds up the columns of its first operand
  if (tid < TM) colsum[tid] = 0.f;

  v16f acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  const float unit = HALF ? scale_unit<NT>(d.scale, r_begin, r_count, list.top) : 1.f;
  for (int base = 0; base < r_count; base += kSmallList) {
    const int64_t r0 = r_begin + base;
    const int n = list_rows<NT>(d.scale, r0, min(kSmallList, r_count - base), unit, list);
    for (int k0 = 0; k0 < n; k0 += BK) {
      Stage<T, TM, NT, BK> a;
      Stage<int8_t, TN, NT, BK> b;
      a.load(static_cast<const T*>(d.g), d.ldg, r0, list, k0, ti * TM, d.m);
      b.load(d.q, d.ldq, r0, list, k0, tj * TN, d.n);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < a.N; ++i) {
        const int r = a.row(i), c = a.col(i);
        if constexpr (P == 3) {
          v8s h[3];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            short p[3];
            cut3(a.v[i][k], p);
            h[0][k] = p[0], h[1][k] = p[1], h[2][k] = p[2];
          }
#pragma unroll
          for (int p = 0; p < 3; ++p) *reinterpret_cast<v8s*>(&lds[p][r][c]) = h[p];
        } else {
          *reinterpret_cast<v8s*>(&lds[0][r][c]) = a.v[i];
        }
      }
#pragma unroll
      for (int i = 0; i < b.N; ++i) {
        const int r = b.row(i), c = b.col(i);
        *reinterpret_cast<v8s*>(&lds[P][r][c]) = codes16<HALF>(b.v[i], list.s[k0 + r]);
      }
      __syncthreads();
      if (sums && tid < TM) {
        float sum = 0.f;
        for (int r = 0; r < BK; ++r)
#pragma unroll
          for (int p = P - 1; p >= 0; --p) {
            if (HALF) sum += static_cast<float>(__builtin_bit_cast(_Float16, lds[p][r][tid]));
            else sum += static_cast<float>(__builtin_bit_cast(__bf16, lds[p][r][tid]));
          }
        colsum[tid] += sum;
      }
      const int s16 = lane & 15, kk = 8 * (lane >> 5) + (s16 >> 2), cc = 16 * ((lane >> 4) & 1) + 4 * (s16 & 3);
      auto operand = [&](int p, int k, int c) {
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)&lds[p][k + kk][c + cc]);
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)&lds[p][k + kk + 4][c + cc]);
        return v8s{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      };
#pragma unroll
      for (int k = 0; k < BK; k += 16) {
        v8s vb[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) vb[j] = operand(P, k, (wave & 1) * 64 + 32 * j);
#pragma unroll
        for (int p = P - 1; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const v8s va = operand(p, k, (wave >> 1) * 64 + 32 * i);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if constexpr (HALF)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, va), __builtin_bit_cast(v8h, vb[j]), acc[i][j], 0, 0, 0);
              else
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, va), __builtin_bit_cast(v8b, vb[j]), acc[i][j], 0, 0, 0);
            }
          }
      }
    }
  }
  __syncthreads();
  const float back = 1.f / unit;  // exact: a power of two
  if (d.splits > 1) {
    KG float* part = gp(d.part) + (int64_t(split) * d.tiles + tile) * (TM * TN);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int r = (wave >> 1) * 64 + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
          const int c = (wave & 1) * 64 + 32 * j + (lane & 31);
          part[r * TN + c] = acc[i][j][e] * back;
        }
    if (sums && tid < TM) gp(d.part_col)[(int64_t(split) * d.mt + ti) * TM + tid] = colsum[tid];
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t r = int64_t(ti) * TM + (wave >> 1) * 64 + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        const int64_t c = int64_t(tj) * TN + (wave & 1) * 64 + 32 * j + (lane & 31);
        if (r < d.m && c < d.n) put_grad(gp(d.out) + r * d.ldo + c, acc[i][j][e] * back, d.accumulate);
      }
  if (!sums || tid >= TM) return;
  const int64_t r = int64_t(ti) * TM + tid;
  if (r < d.m) put_grad(gp(d.bias_out) + r * d.inc_b, colsum[tid], d.accumulate);
}

// ---- joining ------------------------------------------------------------------------

constexpr int kJoin = 1024;  // entries of a tile that a block joins

__host__ __device__ inline int tile_edge(const TnJob& d) { return d.f ? 64 * d.f : 128; }
__host__ __device__ inline int64_t join_tiles(const TnJob& d) {
  return d.splits > 1 ? int64_t(d.tiles) * (tile_edge(d) * tile_edge(d) / kJoin) : 0;
}
inline int64_t join_items(const TnJob& d) {
  return join_tiles(d) + (d.bias && (d.splits > 1 || (d.f && !d.solo)) ? (int64_t(d.m) + 63) / 64 : 0);
}

// The splits' parts of the outputs, and the shares of the column sums, added up in their order: a block joins
// 1024 entries of a tile, or 64 columns' sums, four threads each.
template <bool FACTOR>
__global__ void __launch_bounds__(256) q8_join_kernel(TnArgs<FACTOR> args) {
  const int tid = threadIdx.x;
  const TnJob& d = args.j[FACTOR ? args.owner(blockIdx.x, &TnJob::join_begin) : 0];
  const int T = tile_edge(d), item = blockIdx.x - d.join_begin, here = static_cast<int>(join_tiles(d));
  int counted = 0, bad = 0;
  if (FACTOR) {
    for (int s = tid & 63; s < d.splits; s += 64) {
      const int n = gp(d.part_rows)[s];
      counted += abs(n), bad |= n < 0;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) counted += __shfl_xor(counted, o), bad |= __shfl_xor(bad, o);
  }
  const float inv_r = counted ? 1.f / static_cast<float>(counted) : 0.f;
  const PutFactor put = put_factor(d, counted);
  if (item < here) {
    const int per = T * T / kJoin, tile = item / per, x = item % per * kJoin + 4 * tid;
    int ti, tj;
    if (FACTOR) factor_tile(tile, d.mt, ti, tj);
    else ti = tile / d.nt, tj = tile % d.nt;
    const int r = ti * T + x / T, c = tj * T + x % T;
    if (r >= d.m || c >= d.n || (FACTOR && r > c + 3)) return;
    const KG float* from = gp(d.part) + int64_t(tile) * (T * T) + x;
    const int64_t apart = int64_t(d.tiles) * (T * T);
    v4f sum = {0.f, 0.f, 0.f, 0.f};
    int s = 0;
    for (; s + 8 <= d.splits; s += 8) {
      v4f v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = *reinterpret_cast<const KG v4f*>(from + (s + k) * apart);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += v[k];
    }
    for (; s < d.splits; ++s) sum += *reinterpret_cast<const KG v4f*>(from + s * apart);
    if constexpr (FACTOR) {
      const int rs[4] = {r, r, r, r}, cs[4] = {c, c + 1, c + 2, c + 3};
      bool live[4];
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) live[k] = cs[k] < d.n && r <= cs[k], x[k] = sum[k] * inv_r;
      put.all(rs, cs, live, x);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + k < d.n) put_grad(gp(d.out) + int64_t(r) * d.ldo + c + k, sum[k], d.accumulate);
    }
    return;
  }
  __shared__ float part[4][64];
  const int c = (item - here) * 64 + (tid & 63);
  const int all = d.splits * d.shares;
  float sum = 0.f;
  if (c < d.m)
#pragma unroll 8
    for (int k = tid >> 6; k < all; k += 4) sum += gp(d.part_col)[int64_t(k) * (int64_t(d.mt) * T) + c];
  part[tid >> 6][tid & 63] = sum;
  __syncthreads();
  if (tid >= 64 || c >= d.m) return;
  sum = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
  if (FACTOR) {
    put(c, d.m, sum * inv_r);
    if (c == 0) put(d.m, d.m, corner(counted, bad));
  } else {
    put_grad(gp(d.bias_out) + c * d.inc_b, sum, d.accumulate);
  }
}

// ---- host -------------------------------------------------------------------

constexpr int kCus = 256;

static void set_tiles(TnJob& j, int f, bool factor) {
  j.f = f;
  const int T = tile_edge(j);
  j.mt = static_cast<int32_t>((int64_t(j.m) + T - 1) / T);
  j.nt = std::max(1, static_cast<int32_t>((int64_t(j.n) + T - 1) / T));  // a bias alone has its tiles too
  j.tiles = factor ? j.mt * (j.mt + 1) / 2 : j.mt * j.nt;
  j.shares = !f || factor ? 1 : 2 * j.nt;
}

// Tile edge and splits of the rows by what they are expected to take, in us, which is returned: rounds over the
// compute units of the steps of one tile (measured on full cards; a factor's scales add some), what a block
// spends before and after, and the parts' way through memory. `share`: the part of the card that the job has;
// `only`: this tile edge, unless 0. A factor of few columns or far rows has tiles of 64.
static double plan(TnJob& j, bool factor, kfac_dtype dtype, bool near, double share, int only) {
  const int64_t rows = std::max(j.rows, 1);
  const int least = factor ? 16 : 8, rows_a_step = factor ? 64 : kStep;
  double best = 0;
  const bool plain = !near || j.m < least || j.n < least;
  j.any = factor && plain;
  if (plain && !factor) {
    set_tiles(j, 0, factor);
    const int64_t splits = std::max<int64_t>(1, std::min<int64_t>((rows + 511) / 512, 512 / std::max(1, j.tiles)));
    j.per_split = static_cast<int32_t>((rows + splits - 1) / splits);
  } else {
    int best_f = 0;
    int64_t best_splits = 1;
    const int64_t steps = (rows + rows_a_step - 1) / rows_a_step;
    for (int f : {1, 2, 3, 4}) {
      if (factor ? f == 4 : f == 1 || f == 3 || (f == 4 && dtype == KFAC_F32)) continue;
      if (j.any ? f != 1 : only && f != only) continue;
      set_tiles(j, f, factor);
      const double entries = double(j.tiles) * tile_edge(j) * tile_edge(j);
      const double slots = std::max(1.0, kCus * share * (f == 1 ? 3 : f == 2 ? 2 : 1));
      const double step = factor ? (f == 1 ? 0.6 : 0.55) : f == 4 ? 0.95 : dtype == KFAC_F32 ? 2.0 : 0.6;
      const int64_t fewest = factor ? (rows + factor_rows(f) - 1) / factor_rows(f) : 1;
      for (int64_t s = fewest; s <= std::max<int64_t>(fewest, 128) && (s == fewest || steps / s >= 4); s += factor ? 1 + s / 8 : 1) {
        const double rounds = std::ceil(double(j.tiles) * s / slots), each = std::ceil(double(steps) / s);
        double us;
        if (factor) {
          us = rounds * (6 + 4 * f + (each + 4) * step);
          us += s > 1 ? 6 + 0.15 * s + entries * (10 + 2 * s) / (6e6 * share) : 2 * f * f;
        } else {
          us = rounds * (8 + each * step) + (s > 1 ? 4 + entries * (1 + s) / 1e6 : 0);
        }
        if (best == 0 || us < best) best = us, best_f = f, best_splits = s;
      }
    }
    set_tiles(j, best_f, factor);
    j.per_split = static_cast<int32_t>((steps + best_splits - 1) / best_splits * rows_a_step);
  }
  j.splits = static_cast<int32_t>((rows + j.per_split - 1) / j.per_split);
  // one tile's waves add up the columns alone where that saves a launch and takes little
  j.solo = j.f && j.splits == 1 && (factor || j.nt == 1 || rows <= 1024);
  return best;
}

// A factor's sums need room beside the splits' parts: where they leave 32 bits, which one row's cannot.
static void carve(TnJob& j, bool factor, Carver& cv) {
  const int T = tile_edge(j);
  if (j.splits > 1 || (factor && j.rows > 1)) j.part = cv.take<float>(size_t(j.splits) * j.tiles * T * T);
  if (j.splits == 1 && (!j.f || j.solo)) return;
  j.part_col = cv.take<float>(size_t(j.splits) * j.shares * j.mt * T);
  j.part_rows = cv.take<int32_t>(j.splits);
}

static kfac_status sizes_fit(int64_t rows, int64_t m, int64_t n) {
  if (rows < 0 || m < 0 || n < 0) return fail(KFAC_ERR_INVALID, "negative size");
  if (((m + 127) / 128) * ((n + 127) / 128) > (1 << 20)) return fail(KFAC_ERR_UNSUPPORTED, "more than 2^20 tiles of 128 x 128");
  return KFAC_OK;
}

template <class T>
static kfac_status launch_plain(const TnJob& j, hipStream_t s) {
  if (j.m == 0 || (j.n == 0 && !j.bias)) return KFAC_OK;
  KFAC_LAUNCH(K_GRAD_Q8, q8_plain_kernel<T>, dim3(j.tiles * j.splits), dim3(256), 0, s, j);
  KFAC_CHECK_LAUNCH("q8_plain_kernel");
  return KFAC_OK;
}

// Jobs of one kind (a gradient, or factors of one tile edge), and what joins their parts.
template <class T, bool FACTOR>
static kfac_status launch_jobs(TnJob* j, int n, bool ragged, hipStream_t s) {
  TnArgs<FACTOR> a = {};
  int64_t items = 0, joins = 0;
  for (int i = 0; i < n; ++i) {
    j[i].begin = static_cast<int32_t>(items), j[i].join_begin = static_cast<int32_t>(joins);
    items += int64_t(j[i].tiles) * j[i].splits;
    joins += join_items(j[i]);
    a.j[i] = j[i];
  }
  if (items > kMostBlocks || joins > kMostBlocks) return fail(KFAC_ERR_UNSUPPORTED, "too many tiles: more than a launch takes");
  a.n = n, a.items = static_cast<int32_t>(items), a.joins = static_cast<int32_t>(joins);
  const int f = j[0].f;
  kfac_status st = KFAC_OK;
  if constexpr (FACTOR) {
    st = launch_factor_tiles(a, f, ragged, s);
  } else {
    if (f == 0) st = launch_plain<T>(j[0], s);
    if (f == 2) st = ragged ? launch_grad_tiles<T, 2, true>(a, s) : launch_grad_tiles<T, 2, false>(a, s);
    if constexpr (!std::is_same_v<T, float>)
      if (f == 4) st = ragged ? launch_grad_tiles<T, 4, true>(a, s) : launch_grad_tiles<T, 4, false>(a, s);
  }
  if (st || !joins) return st;
  KFAC_LAUNCH(FACTOR ? K_FACTOR_Q8_JOIN : K_GRAD_Q8_JOIN, q8_join_kernel<FACTOR>, dim3(static_cast<unsigned>(joins)),
              dim3(256), 0, s, a);
  KFAC_CHECK_LAUNCH("q8_join_kernel");
  return KFAC_OK;
}

// near: rows lie less than 2^32 bytes apart.
static TnJob grad_job(int32_t rows, int32_t c_in, int32_t c_out, kfac_dtype dtype, bool bias, bool near) {
  TnJob j = {};
  j.rows = rows, j.m = c_out, j.n = c_in, j.bias = bias;
  plan(j, false, dtype, near, 1.0, 0);
  return j;
}

extern "C" kfac_status kfac_weight_grad_q8_workspace(int32_t rows, int32_t c_in, int32_t c_out, kfac_dtype dtype,
                                                     size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  if (!row_dtype(dtype)) return fail(KFAC_ERR_UNSUPPORTED, "dtype %d", dtype);
  kfac_status st = sizes_fit(rows, c_out, c_in);
  if (st) return st;
  *bytes = 0;
  for (bool near : {false, true}) {
    TnJob j = grad_job(rows, c_in, c_out, dtype, true, near);
    Carver cv;
    carve(j, false, cv);
    *bytes = std::max(*bytes, cv.used);
  }
  return KFAC_OK;
}

extern "C" kfac_status kfac_weight_grad_q8(int32_t rows, int32_t c_in, int32_t c_out, kfac_dtype dtype, const void* gout,
                                           int64_t ld_g, const int8_t* q, int64_t ld_q, const float* scale, float* dweight,
                                           int64_t ld_dw, float* dbias, int64_t inc_db, int32_t accumulate,
                                           void* workspace, size_t ws_bytes, void* stream) {
  if (!row_dtype(dtype)) return fail(KFAC_ERR_UNSUPPORTED, "dtype %d", dtype);
  kfac_status st = sizes_fit(rows, c_out, c_in);
  if (st) return st;
  if (accumulate != 0 && accumulate != 1) return fail(KFAC_ERR_INVALID, "accumulate must be 0 or 1");
  const RowsOf gs = {gout, rows, c_out, ld_g, dtype_bytes(dtype), "gout"}, qs = {q, rows, c_in, ld_q, 1, "q"},
               ss = {scale, c_out > 0 ? rows : 0, 1, 1, 4, "scale"}, ws = {dweight, c_out, c_in, ld_dw, 4, "dweight"},
               bs = {dbias, dbias ? c_out : 0, 1, inc_db, 4, "dbias"};
  for (const RowsOf* r : {&gs, &qs, &ss, &ws, &bs})
    if ((st = check_rows(*r))) return st;
  constexpr int64_t kFar = int64_t(1) << 32;  // bytes between rows, which the tile kernel holds in 32 bits
  const bool near = rows <= 1 || (ld_g < kFar / gs.size && ld_q < kFar);
  TnJob j = grad_job(rows, c_in, c_out, dtype, dbias != nullptr, near);
  Carver sizing, cv(workspace);
  carve(j, false, sizing);
  const RowsOf scr = scratch(workspace, sizing.used);
  if ((st = check_apart({&ws, &bs, &scr, &gs, &qs, &ss}, 3))) return st;
  if ((st = check_device())) return st;
  if ((st = check_workspace(workspace, ws_bytes, sizing.used))) return st;
  carve(j, false, cv);
  j.g = gout, j.q = q, j.scale = scale, j.out = dweight, j.bias_out = dbias;
  j.ldg = ld_g, j.ldq = ld_q, j.ldo = ld_dw, j.inc_b = inc_db, j.accumulate = accumulate;
  if (c_out == 0 || (c_in == 0 && !dbias)) return KFAC_OK;
  return with_row_type(dtype, [&](auto tag) {
    return launch_jobs<decltype(tag), false>(&j, 1, (c_in | c_out) & 7, static_cast<hipStream_t>(stream));
  });
}

static TnJob factor_job(int32_t rows, int32_t cols, int32_t bias, double share, int f, bool near, double* us) {
  TnJob j = {};
  j.rows = rows, j.m = j.n = cols, j.bias = bias;
  const double t = plan(j, true, KFAC_F16, near, share, f);
  if (us) *us = t;
  return j;
}

// The layers' jobs: near, if their rows lie less than 2^32 bytes apart, and far, if not.
static kfac_status factor_jobs(int32_t count, const int32_t* rows, const int32_t* cols, const int32_t* bias,
                               std::vector<TnJob>& near, std::vector<TnJob>& far) {
  if (count < 0) return fail(KFAC_ERR_INVALID, "negative count");
  if (count > 0 && (!rows || !cols || !bias)) return fail(KFAC_ERR_INVALID, "NULL array");
  double work = 0;
  auto work_of = [&](int i) { return double(std::max(rows[i], 256)) * (cols[i] + 128.0) * (cols[i] + 128.0); };
  for (int i = 0; i < count; ++i) {
    kfac_status st = sizes_fit(rows[i], cols[i], cols[i]);
    if (st) return st;
    if (cols[i] < 1) return fail(KFAC_ERR_INVALID, "layer %d: cols must be positive", i);
    if (bias[i] != 0 && bias[i] != 1) return fail(KFAC_ERR_INVALID, "layer %d: bias must be 0 or 1", i);
    work += work_of(i);
  }
  // one tile edge for all layers, so that they run side by side: the one whose slowest layer is soonest done
  double best = 0;
  for (int f : {1, 2, 3}) {
    std::vector<TnJob> jobs;
    double slowest = 0;
    for (int i = 0; i < count; ++i) {
      double us = 0;
      jobs.push_back(factor_job(rows[i], cols[i], bias[i], work_of(i) / work, f, true, &us));
      if (!jobs[i].any) slowest = std::max(slowest, us);
    }
    if (f == 1 || slowest < best) best = slowest, near = std::move(jobs);
  }
  for (int i = 0; i < count; ++i) far.push_back(factor_job(rows[i], cols[i], bias[i], 1.0, 0, false, nullptr));
  return KFAC_OK;
}

static size_t bytes_of(TnJob j) {
  Carver cv;
  carve(j, true, cv);
  return cv.used;
}

// Layers run side by side as long as their parts and sums fit here, and in launches one after another, which use the
// same room, where they do not: such layers fill the card each.
constexpr size_t kRoom = size_t(128) << 20;

// The workspace of a call, whichever of its jobs each layer turns out to have.
static size_t factors_room(const std::vector<TnJob>& near, const std::vector<TnJob>& far) {
  size_t all = 0, largest = 0;
  for (size_t i = 0; i < near.size(); ++i) {
    const size_t one = std::max(bytes_of(near[i]), bytes_of(far[i]));
    all += one, largest = std::max(largest, one);
  }
  return std::max(largest, std::min(all, kRoom));
}

extern "C" kfac_status kfac_factors_q8_workspace(int32_t count, const int32_t* rows, const int32_t* cols,
                                                 const int32_t* bias, size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  return guarded([&] {
    std::vector<TnJob> near, far;
    kfac_status st = factor_jobs(count, rows, cols, bias, near, far);
    if (st) return st;
    *bytes = factors_room(near, far);
    return KFAC_OK;
  });
}

static kfac_status factors_impl(int32_t count, const int32_t* rows, const int32_t* cols, const int32_t* bias,
                                const int8_t* const* q, const int64_t* ld_q, const float* const* scale,
                                float* const* A_packed, float* const* A_full, float ema_decay, void* workspace,
                                size_t ws_bytes, hipStream_t s) {
  if (!(ema_decay >= 0.f && ema_decay <= 1.f)) return fail(KFAC_ERR_INVALID, "ema_decay must be in [0, 1]");
  if (count > 0 && (!q || !ld_q || !scale || !A_packed)) return fail(KFAC_ERR_INVALID, "NULL array");
  std::vector<TnJob> jobs, far;
  kfac_status st = factor_jobs(count, rows, cols, bias, jobs, far);
  if (st) return st;
  const size_t need = factors_room(jobs, far);
  for (int i = 0; i < count; ++i)
    if (rows[i] > 1 && ld_q[i] >= (int64_t(1) << 32)) jobs[i] = far[i];
  auto left_out = [&](int i) { return !q[i] && !scale[i] && !A_packed[i]; };
  std::vector<RowsOf> all = {scratch(workspace, need)};
  for (int i = 0; i < count; ++i) {
    if (left_out(i)) continue;
    const int64_t d = cols[i] + bias[i];
    all.push_back({A_packed[i], 1, d * (d + 1) / 2, 0, 4, "A_packed"});
    if (A_full && A_full[i]) all.push_back({A_full[i], 1, d * d, 0, 4, "A_full"});
  }
  const int written = static_cast<int>(all.size());
  for (int i = 0; i < count; ++i) {
    if (left_out(i)) continue;
    all.push_back({q[i], rows[i], cols[i], ld_q[i], 1, "q"});
    all.push_back({scale[i], rows[i], 1, 1, 4, "scale"});
  }
  std::vector<const RowsOf*> each;
  for (const RowsOf& r : all) {
    if (&r != &all[0] && (st = check_rows(r))) return st;
    each.push_back(&r);
  }
  if ((st = check_apart(each.data(), static_cast<int>(each.size()), written))) return st;
  if ((st = check_device())) return st;
  if ((st = check_workspace(workspace, ws_bytes, need))) return st;
  for (int i = 0; i < count; ++i) {
    TnJob& j = jobs[i];
    j.q = q[i], j.scale = scale[i], j.ldq = ld_q[i], j.out = A_packed[i], j.full = A_full ? A_full[i] : nullptr;
    j.decay = ema_decay;
  }
  // layers in tiles of 64 go with those of few columns, if there are any: 4 of 20000 x 64 and one of 20000 x 8 24 us, in
  // two launches 40
  if (std::any_of(jobs.begin(), jobs.end(), [](const TnJob& j) { return j.any; }))
    for (TnJob& j : jobs) j.any = j.f == 1;
  jobs.erase(std::remove_if(jobs.begin(), jobs.end(), [](const TnJob& j) { return !j.out; }), jobs.end());
  // a launch for the layers of one kind, or several
  std::vector<TnJob> some;
  for (int kind = 0; kind < 7; ++kind) {
    const int f = 3 - kind / 2, any = kind == 6;
    const bool ragged = kind & 1;
    some.clear();
    for (const TnJob& j : jobs)
      if (any ? j.any : !j.any && j.f == f && bool(j.m & 15) == ragged) some.push_back(j);
    for (size_t i = 0, n; i < some.size(); i += n) {
      Carver cv(workspace);
      for (n = 0; n < kTnMany && i + n < some.size() && (n == 0 || cv.used + bytes_of(some[i + n]) <= kRoom); ++n)
        carve(some[i + n], true, cv);
      if ((st = launch_jobs<_Float16, true>(&some[i], static_cast<int>(n), ragged, s))) return st;
    }
  }
  return KFAC_OK;
}

extern "C" kfac_status kfac_factors_q8(int32_t count, const int32_t* rows, const int32_t* cols, const int32_t* bias,
                                       const int8_t* const* q, const int64_t* ld_q, const float* const* scale,
                                       float* const* A_packed, float* const* A_full, float ema_decay, void* workspace,
                                       size_t ws_bytes, void* stream) {
  return guarded([&] {
    return factors_impl(count, rows, cols, bias, q, ld_q, scale, A_packed, A_full, ema_decay, workspace, ws_bytes,
                        static_cast<hipStream_t>(stream));
  });
}

}  // namespace kfac
