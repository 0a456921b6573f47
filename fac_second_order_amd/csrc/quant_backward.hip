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
// formed in fp16.
//
// Rows with s_t = 0 are taken out of a list of the block's rows, before anything of them is
// read: their gradients may hold anything, and cost nothing.
#include "q8.hpp"

namespace kfac {

constexpr int LIST = 2048;  // rows that a list covers
constexpr uint16_t kNoRow = 0xffff;

struct TnJob {
  const void* g;  // gradients; the factor has none
  const int8_t* q;
  const float* scale;
  float* out;       // dW, or the packed factor
  float* full;      // the factor's upper triangle in a full matrix, or NULL
  float* bias_out;  // db, or NULL
  float* part;      // [splits][tiles][TM * TN], with splits > 1
  float* part_col;  // [splits][tile rows][TM]
  int32_t* part_rows;  // [splits]: rows that count
  int64_t ldg, ldq, ldo, inc_b;
  int32_t m, n, rows;  // columns of both operands
  int32_t mt, nt;      // tiles along them
  int32_t tiles, splits, per_split;
  int32_t bias, accumulate;
  float decay;
  int32_t begin;  // first work item
};

// fp16 gradients and the factor are formed in fp16, others in bf16; fp32 ones in three parts.
template <class T>
constexpr int kParts = std::is_same_v<T, float> ? 3 : 1;

template <bool HALF>
__device__ inline v8s codes16(v2u u, float s) {
  v8s out;
  if constexpr (HALF) {
    // 0x64 in front of a byte b is the fp16 number 1024 + b
    const v2h mid = {static_cast<_Float16>(1152.f), static_cast<_Float16>(1152.f)};
    const _Float16 sh = static_cast<_Float16>(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned w = u[i >> 1] ^ 0x80808080u;
      const unsigned b = __builtin_amdgcn_perm(0x64646464u, w, (i & 1) ? 0x04030402u : 0x04010400u);
      const v2h h = (__builtin_bit_cast(v2h, b) - mid) * v2h{sh, sh};
      const unsigned bits = __builtin_bit_cast(unsigned, h);
      out[2 * i] = static_cast<short>(bits);
      out[2 * i + 1] = static_cast<short>(bits >> 16);
    }
  } else {
    const float mid = -128.f * s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned w = u[i >> 2] ^ 0x80808080u;
      out[i] = __builtin_bit_cast(short, static_cast<__bf16>(fmaf(static_cast<float>((w >> (8 * (i & 3))) & 255u), s, mid)));
    }
  }
  return out;
}

// x = h[0] + h[1] + h[2], 8 bits of the significand each, cut and not rounded. An infinity stays one.
__device__ inline void cut3(float x, short (&h)[3]) {
  float r = x;
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const unsigned b = __float_as_uint(r) & 0xffff0000u;
    h[p] = static_cast<short>(b >> 16);
    const float top = __uint_as_float(b);
    r = r == top ? 0.f : r - top;
  }
}

struct RowList {
  uint16_t idx[LIST];
  float s[LIST];
  int32_t group[LIST / 64];
  float top[8];
};

// The rows of [r0, r0 + n) with a scale, in order, with their scales times `unit`; filled up to a
// multiple of 64 with none. Returns how many there are.
template <int NT>
__device__ inline int list_rows(const float* scale, int64_t r0, int n, float unit, RowList& l) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int PER = LIST / NT;
  float s[PER];
  unsigned long long b[PER];
  __syncthreads();  // the list before is done with
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = (wave + i * (NT / 64)) * 64 + lane;
    s[i] = r < n ? gp(scale)[r0 + r] : 0.f;
    b[i] = __ballot(s[i] != 0.f);
    if (lane == 0) l.group[wave + i * (NT / 64)] = __popcll(b[i]);
  }
  __syncthreads();
  int total = 0;
  for (int g = 0; g < LIST / 64; ++g) total += l.group[g];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int own = wave + i * (NT / 64);
    int at = __popcll(b[i] & ((1ull << lane) - 1));
    for (int g = 0; g < own; ++g) at += l.group[g];
    if (s[i] != 0.f) {
      l.idx[at] = static_cast<uint16_t>(own * 64 + lane);
      l.s[at] = s[i] * unit;
    }
  }
  const int whole = (total + 63) / 64 * 64;
  if (total + tid < whole) {
    l.idx[total + tid] = kNoRow;
    l.s[total + tid] = 0.f;
  }
  __syncthreads();
  return total;
}

// 2^k such that the largest finite scale of the rows times it is 2^5: relative to that, fp16 holds
// s q down to 2^-29 of the largest scale exactly (the sum with 1152 that makes a code stays finite).
template <int NT>
__device__ inline float scale_unit(const float* scale, int64_t r0, int n, RowList& l) {
  unsigned top = 0;
  for (int r = threadIdx.x; r < n; r += NT) {
    const unsigned b = __float_as_uint(gp(scale)[r0 + r]) & 0x7fffffffu;
    if (b < 0x7f800000u) top = max(top, b);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, __shfl_xor(top, o));
  if ((threadIdx.x & 63) == 0) l.top[threadIdx.x >> 6] = __uint_as_float(top);
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < NT / 64; ++i) t = fmaxf(t, l.top[i]);
  __syncthreads();
  int e = static_cast<int>(__float_as_uint(t) >> 23);  // 2^(e - 127) <= t
  e = 127 + 5 - (e - 127);                              // of 2^5 / 2^(e - 127)
  return __uint_as_float(static_cast<unsigned>(max(1, min(e, 253))) << 23);
}

// Groups of 8 columns of NU rows x TC columns a step, NT threads.
template <class E, int TC, int NT, int BK>
struct Stage {
  static constexpr int perRow = TC / 8, N = perRow * BK / NT;
  using Raw = std::conditional_t<std::is_same_v<E, int8_t>, v2u, std::conditional_t<std::is_same_v<E, float>, v8f, v8s>>;
  Raw v[N];

  static __device__ inline int row(int i) { return (threadIdx.x + i * NT) / perRow; }
  static __device__ inline int col(int i) { return (threadIdx.x + i * NT) % perRow * 8; }

  // rows l.idx[k0 ..] + r0 of src, columns c0 .. of cols
  __device__ inline void load(const E* src, int64_t ld, int64_t r0, const RowList& l, int k0, int c0, int cols) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint16_t r = l.idx[k0 + row(i)];
      const int c = c0 + col(i);
      const KG E* p = gp(src) + (r0 + r) * ld + c;
      if (r != kNoRow && c + 8 <= cols) {
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
        if (r != kNoRow)
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

// Work item = (job, split of the rows, tile of TM x TN). WM x WN waves of 64 x 64.
template <class T, bool FACTOR>
__global__ void __launch_bounds__(256) q8_tn_kernel(TnJob d) {
  constexpr int TM = 128, TN = 128, NT = 256, BK = 32, PITCH = 128 + 32, P = kParts<T>;
  constexpr bool HALF = std::is_same_v<T, _Float16>;
  using G = std::conditional_t<FACTOR, int8_t, T>;
  __shared__ __attribute__((aligned(16))) short lds[P + 1][BK][PITCH];
  __shared__ RowList list;
  __shared__ float colsum[TM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tile = blockIdx.x % d.tiles, split = blockIdx.x / d.tiles;
  int ti, tj;
  if (FACTOR) upper_tile(tile, d.mt, ti, tj);
  else ti = tile / d.nt, tj = tile % d.nt;
  const int64_t r_begin = int64_t(split) * d.per_split;
  const int r_count = static_cast<int>(min(int64_t(d.per_split), d.rows - r_begin));
  const bool sums = FACTOR ? ti == tj : d.bias && tj == 0;  // this block adds up the columns of its first operand
  if (tid < TM) colsum[tid] = 0.f;

  v16f acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  const float unit = HALF ? scale_unit<NT>(d.scale, r_begin, r_count, list) : 1.f;
  int counted = 0;
  for (int base = 0; base < r_count; base += LIST) {
    const int64_t r0 = r_begin + base;
    const int n = list_rows<NT>(d.scale, r0, min(LIST, r_count - base), unit, list);
    counted += n;
    for (int k0 = 0; k0 < n; k0 += BK) {
      Stage<G, TM, NT, BK> a;
      Stage<int8_t, TN, NT, BK> b;
      const G* src = FACTOR ? reinterpret_cast<const G*>(d.q) : static_cast<const G*>(d.g);
      a.load(src, FACTOR ? d.ldq : d.ldg, r0, list, k0, ti * TM, d.m);
      b.load(d.q, d.ldq, r0, list, k0, tj * TN, d.n);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < a.N; ++i) {
        const int r = a.row(i), c = a.col(i);
        if constexpr (FACTOR) {
          *reinterpret_cast<v8s*>(&lds[0][r][c]) = codes16<HALF>(a.v[i], list.s[k0 + r]);
        } else if constexpr (P == 3) {
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
  const float colback = FACTOR ? back : 1.f;
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
          part[r * TN + c] = FACTOR ? acc[i][j][e] * back * back : acc[i][j][e] * back;
        }
    if (sums && tid < TM) gp(d.part_col)[(int64_t(split) * d.mt + ti) * TM + tid] = colsum[tid] * colback;
    if (tile == 0 && tid == 0) gp(d.part_rows)[split] = counted;
    return;
  }
  const float inv_r = counted ? 1.f / static_cast<float>(counted) : 0.f;
  auto put = [&](int64_t o, int64_t f, float v) {
    if (d.decay != 0.f) {
      const float old = gp(d.out)[o];
      v = counted ? d.decay * old + (1.f - d.decay) * v : old;
    }
    gp(d.out)[o] = v;
    if (d.full) gp(d.full)[f] = v;
  };
  const int64_t order = d.m + d.bias;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t r = int64_t(ti) * TM + (wave >> 1) * 64 + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        const int64_t c = int64_t(tj) * TN + (wave & 1) * 64 + 32 * j + (lane & 31);
        if (FACTOR) {
          if (r <= c && c < d.n) put(packed_off(r, c, order), r * order + c, acc[i][j][e] * back * back * inv_r);
        } else if (r < d.m && c < d.n) {
          KG float* o = gp(d.out) + r * d.ldo + c;
          const float v = acc[i][j][e] * back;
          *o = d.accumulate ? *o + v : v;
        }
      }
  if (!d.bias || !sums || tid >= TM) return;
  const int64_t r = int64_t(ti) * TM + tid;
  if (FACTOR) {
    if (r < d.m) put(packed_off(r, d.m, order), r * order + d.m, colsum[tid] * colback * inv_r);
    if (tile == 0 && tid == 0) put(packed_off(d.m, d.m, order), d.m * order + d.m, counted ? 1.f : 0.f);
  } else if (r < d.m) {
    KG float* o = gp(d.bias_out) + r * d.inc_b;
    *o = d.accumulate ? *o + colsum[tid] : colsum[tid];
  }
}

// The splits' parts added up, a tile a block.
template <bool FACTOR>
__global__ void __launch_bounds__(256) q8_join_kernel(TnJob d) {
  constexpr int TM = 128, TN = 128;
  const int tid = threadIdx.x, tile = blockIdx.x;
  int ti, tj;
  if (FACTOR) upper_tile(tile, d.mt, ti, tj);
  else ti = tile / d.nt, tj = tile % d.nt;
  int counted = 0;
  for (int s = 0; s < d.splits; ++s) counted += gp(d.part_rows)[s];
  const float inv_r = counted ? 1.f / static_cast<float>(counted) : 0.f;
  auto put = [&](int64_t o, int64_t f, float v) {
    if (d.decay != 0.f) {
      const float old = gp(d.out)[o];
      v = counted ? d.decay * old + (1.f - d.decay) * v : old;
    }
    gp(d.out)[o] = v;
    if (d.full) gp(d.full)[f] = v;
  };
  const int64_t order = d.m + d.bias;
  for (int x = tid; x < TM * TN; x += 256) {
    const int64_t r = int64_t(ti) * TM + x / TN, c = int64_t(tj) * TN + x % TN;
    if (FACTOR ? r > c || c >= d.n : r >= d.m || c >= d.n) continue;
    float sum = 0.f;
    for (int s = 0; s < d.splits; ++s) sum += gp(d.part)[(int64_t(s) * d.tiles + tile) * (TM * TN) + x];
    if (FACTOR) {
      put(packed_off(r, c, order), r * order + c, sum * inv_r);
    } else {
      KG float* o = gp(d.out) + r * d.ldo + c;
      *o = d.accumulate ? *o + sum : sum;
    }
  }
  if (!d.bias || tid >= TM || (FACTOR ? ti != tj : tj != 0)) return;
  const int64_t r = int64_t(ti) * TM + tid;
  if (r >= d.m) return;
  float sum = 0.f;
  for (int s = 0; s < d.splits; ++s) sum += gp(d.part_col)[(int64_t(s) * d.mt + ti) * TM + tid];
  if (FACTOR) {
    put(packed_off(r, d.m, order), r * order + d.m, sum * inv_r);
    if (r == 0) put(packed_off(d.m, d.m, order), d.m * order + d.m, counted ? 1.f : 0.f);
  } else {
    KG float* o = gp(d.bias_out) + r * d.inc_b;
    *o = d.accumulate ? *o + sum : sum;
  }
}

// ---- host -------------------------------------------------------------------

constexpr int TILE = 128;

// Tiles and splits of a job's m x n outputs over its rows: enough items to fill the 256 compute units
// twice, no fewer than 512 rows each.
static void plan(TnJob& j, bool factor) {
  j.mt = (j.m + TILE - 1) / TILE;
  j.nt = std::max(1, (j.n + TILE - 1) / TILE);  // a bias alone has its tiles too
  const int64_t tiles = factor ? int64_t(j.mt) * (j.mt + 1) / 2 : int64_t(j.mt) * j.nt;
  j.tiles = static_cast<int32_t>(std::min<int64_t>(tiles, INT32_MAX));
  int64_t splits = std::min<int64_t>((j.rows + 511) / 512, 512 / std::max<int64_t>(1, tiles));
  splits = std::max<int64_t>(1, splits);
  j.per_split = static_cast<int32_t>((std::max(j.rows, 1) + splits - 1) / splits);
  j.splits = std::max(1, (j.rows + j.per_split - 1) / j.per_split);
}

static void carve(TnJob& j, Carver& cv) {
  if (j.splits == 1) return;
  j.part = cv.take<float>(size_t(j.splits) * j.tiles * TILE * TILE);
  j.part_col = cv.take<float>(size_t(j.splits) * j.mt * TILE);
  j.part_rows = cv.take<int32_t>(j.splits);
}

static kfac_status sizes_fit(int64_t rows, int64_t m, int64_t n) {
  if (rows < 0 || m < 0 || n < 0) return fail(KFAC_ERR_INVALID, "negative size");
  if (((m + TILE - 1) / TILE) * ((n + TILE - 1) / TILE) > (1 << 22)) return fail(KFAC_ERR_UNSUPPORTED, "more than 2^22 tiles");
  return KFAC_OK;
}

template <class T, bool FACTOR>
static kfac_status launch_tn(const TnJob& j, hipStream_t s) {
  if (j.m == 0 || (j.n == 0 && !j.bias)) return KFAC_OK;
  KFAC_LAUNCH(FACTOR ? K_FACTOR_Q8 : K_GRAD_Q8, (q8_tn_kernel<T, FACTOR>), dim3(j.tiles * j.splits), dim3(256), 0, s, j);
  KFAC_CHECK_LAUNCH("q8_tn_kernel");
  if (j.splits > 1) {
    KFAC_LAUNCH(FACTOR ? K_FACTOR_Q8_JOIN : K_GRAD_Q8_JOIN, q8_join_kernel<FACTOR>, dim3(j.tiles), dim3(256), 0, s, j);
    KFAC_CHECK_LAUNCH("q8_join_kernel");
  }
  return KFAC_OK;
}

static TnJob grad_job(int32_t rows, int32_t c_in, int32_t c_out) {
  TnJob j = {};
  j.rows = rows, j.m = c_out, j.n = c_in;
  plan(j, false);
  return j;
}

extern "C" kfac_status kfac_weight_grad_q8_workspace(int32_t rows, int32_t c_in, int32_t c_out, kfac_dtype dtype,
                                                     size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  if (!row_dtype(dtype)) return fail(KFAC_ERR_UNSUPPORTED, "dtype %d", dtype);
  kfac_status st = sizes_fit(rows, c_out, c_in);
  if (st) return st;
  TnJob j = grad_job(rows, c_in, c_out);
  Carver cv;
  carve(j, cv);
  *bytes = cv.used;
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
  TnJob j = grad_job(rows, c_in, c_out);
  Carver sizing, cv(workspace);
  carve(j, sizing);
  const RowsOf scr = scratch(workspace, sizing.used);
  if ((st = check_apart({&ws, &bs, &scr, &gs, &qs, &ss}, 3))) return st;
  if ((st = check_device())) return st;
  if ((st = check_workspace(workspace, ws_bytes, sizing.used))) return st;
  carve(j, cv);
  j.g = gout, j.q = q, j.scale = scale, j.out = dweight, j.bias_out = dbias;
  j.ldg = ld_g, j.ldq = ld_q, j.ldo = ld_dw, j.inc_b = inc_db, j.bias = dbias != nullptr, j.accumulate = accumulate;
  return with_row_type(dtype, [&](auto tag) { return launch_tn<decltype(tag), false>(j, static_cast<hipStream_t>(stream)); });
}

static kfac_status factor_jobs(int32_t count, const int32_t* rows, const int32_t* cols, const int32_t* bias,
                               std::vector<TnJob>& jobs, Carver& cv) {
  if (count < 0) return fail(KFAC_ERR_INVALID, "negative count");
  if (count > 0 && (!rows || !cols || !bias)) return fail(KFAC_ERR_INVALID, "NULL array");
  for (int i = 0; i < count; ++i) {
    kfac_status st = sizes_fit(rows[i], cols[i], cols[i]);
    if (st) return st;
    if (cols[i] < 1) return fail(KFAC_ERR_INVALID, "layer %d: cols must be positive", i);
    if (bias[i] != 0 && bias[i] != 1) return fail(KFAC_ERR_INVALID, "layer %d: bias must be 0 or 1", i);
    TnJob j = {};
    j.rows = rows[i], j.m = j.n = cols[i], j.bias = bias[i];
    plan(j, true);
    carve(j, cv);
    jobs.push_back(j);
  }
  return KFAC_OK;
}

extern "C" kfac_status kfac_factors_q8_workspace(int32_t count, const int32_t* rows, const int32_t* cols,
                                                 const int32_t* bias, size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  return guarded([&] {
    std::vector<TnJob> jobs;
    Carver cv;
    kfac_status st = factor_jobs(count, rows, cols, bias, jobs, cv);
    if (!st) *bytes = cv.used;
    return st;
  });
}

static kfac_status factors_impl(int32_t count, const int32_t* rows, const int32_t* cols, const int32_t* bias,
                                const int8_t* const* q, const int64_t* ld_q, const float* const* scale,
                                float* const* A_packed, float* const* A_full, float ema_decay, void* workspace,
                                size_t ws_bytes, hipStream_t s) {
  if (!(ema_decay >= 0.f && ema_decay <= 1.f)) return fail(KFAC_ERR_INVALID, "ema_decay must be in [0, 1]");
  std::vector<TnJob> jobs;
  Carver sizing;
  kfac_status st = factor_jobs(count, rows, cols, bias, jobs, sizing);
  if (st) return st;
  if (count > 0 && (!q || !ld_q || !scale || !A_packed)) return fail(KFAC_ERR_INVALID, "NULL array");
  std::vector<RowsOf> all = {scratch(workspace, sizing.used)};
  for (int i = 0; i < count; ++i) {
    const int64_t d = cols[i] + bias[i];
    all.push_back({A_packed[i], 1, d * (d + 1) / 2, 0, 4, "A_packed"});
    if (A_full && A_full[i]) all.push_back({A_full[i], 1, d * d, 0, 4, "A_full"});
  }
  const int written = static_cast<int>(all.size());
  for (int i = 0; i < count; ++i) {
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
  if ((st = check_workspace(workspace, ws_bytes, sizing.used))) return st;
  Carver cv(workspace);
  for (int i = 0; i < count; ++i) {
    TnJob& j = jobs[i];
    carve(j, cv);
    j.q = q[i], j.scale = scale[i], j.ldq = ld_q[i], j.out = A_packed[i], j.full = A_full ? A_full[i] : nullptr;
    j.decay = ema_decay;
    if ((st = launch_tn<_Float16, true>(j, s))) return st;
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
