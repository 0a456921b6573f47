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

constexpr int kSmallList = 2048, kBigList = 8192;  // rows that a list covers

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
  int32_t big;    // 256 x 256 tiles
};

// fp16 gradients and the factor are formed in fp16, others in bf16; fp32 ones in three parts.
template <class T>
constexpr int kParts = std::is_same_v<T, float> ? 3 : 1;

// Codes 2 h and 2 h + 1 of four, times s, as two 16-bit numbers.
template <bool HALF>
__device__ inline unsigned two_codes(unsigned four, int h, float s) {
  const unsigned w = four ^ 0x80808080u;  // code + 128
  if constexpr (HALF) {
    // 0x64 in front of a byte b is the fp16 number 1024 + b
    const v2h mid = {static_cast<_Float16>(1152.f), static_cast<_Float16>(1152.f)};
    const _Float16 sh = static_cast<_Float16>(s);
    const unsigned b = __builtin_amdgcn_perm(0x64646464u, w, h ? 0x04030402u : 0x04010400u);
    return __builtin_bit_cast(unsigned, (__builtin_bit_cast(v2h, b) - mid) * v2h{sh, sh});
  } else {
    const float mid = -128.f * s;
    const v2bf out = {static_cast<__bf16>(fmaf(static_cast<float>((w >> (16 * h)) & 255u), s, mid)),
                      static_cast<__bf16>(fmaf(static_cast<float>((w >> (16 * h + 8)) & 255u), s, mid))};
    return __builtin_bit_cast(unsigned, out);
  }
}

template <bool HALF>
__device__ inline v8s codes16(v2u u, float s) {
  return __builtin_bit_cast(v8s, v4u{two_codes<HALF>(u[0], 0, s), two_codes<HALF>(u[0], 1, s),
                                     two_codes<HALF>(u[1], 0, s), two_codes<HALF>(u[1], 1, s)});
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

// The rows of a stretch that take part, with their scales times a unit; behind them rows that are none.
template <int LIST>
struct RowList {
  __attribute__((aligned(16))) uint16_t idx[LIST + 64];  // or kNone: none (and row 0)
  __attribute__((aligned(16))) float s[LIST + 64];
  int32_t group[LIST / 64];
  float top[8];
};
constexpr uint16_t kNone = 0x8000;

// The rows of [r0, r0 + n) with a scale, in order; filled up to a multiple of 64. Returns how many there are.
// SHUFFLED: within 32 rows, row 8 i + j lies at 4 j + i.
template <int NT, bool SHUFFLED, int LIST>
__device__ inline int list_rows(const float* scale, int64_t r0, int n, float unit, RowList<LIST>& l) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int PER = LIST / NT;
  float s[PER];
  unsigned long long b[PER];
  __syncthreads();  // the list before is done with
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = (wave + i * (NT / 64)) * 64 + lane;
    s[i] = r < n ? gp(scale)[r0 + r] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    b[i] = __ballot(s[i] != 0.f);
    if (lane == 0) l.group[wave + i * (NT / 64)] = __popcll(b[i]);
  }
  __syncthreads();
  // rows before each group of 64: lane g adds up the groups below g, 64 groups at a time
  int total = 0, before[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) before[i] = 0;
#pragma unroll
  for (int g0 = 0; g0 < LIST / 64; g0 += 64) {
    int own = g0 + lane < LIST / 64 ? l.group[g0 + lane] : 0, sum = own;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int up = __shfl_up(sum, o);
      if (lane >= o) sum += up;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int g = wave + i * (NT / 64);
      if (g >= g0 && g < g0 + 64) before[i] = total + __shfl(sum - own, g - g0);
    }
    total += __shfl(sum, 63);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = before[i] + __popcll(b[i] & ((1ull << lane) - 1));
    if (s[i] != 0.f) {
      const int to = SHUFFLED ? (at & ~31) | ((at & 7) << 2) | ((at >> 3) & 3) : at;
      l.idx[to] = static_cast<uint16_t>((wave + i * (NT / 64)) * 64 + lane);
      l.s[to] = s[i] * unit;
    }
  }
  const int whole = (total + 63) / 64 * 64;
  if (total + tid < whole) {
    const int at = total + tid, to = SHUFFLED ? (at & ~31) | ((at & 7) << 2) | ((at >> 3) & 3) : at;
    l.idx[to] = kNone;
    l.s[to] = 0.f;
  }
  __syncthreads();
  return total;
}

// 2^k such that the largest finite scale of the rows times it is 2^5: relative to that, fp16 holds
// s q down to 2^-29 of the largest scale exactly (the sum with 1152 that makes a code stays finite).
template <int NT, int LIST>
__device__ inline float scale_unit(const float* scale, int64_t r0, int n, RowList<LIST>& l) {
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

// Work item = (job, split of the rows, tile of TM x TN). WM x WN waves of 64 x 64.
template <class T, bool FACTOR>
__global__ void __launch_bounds__(256) q8_tn_kernel(TnJob d) {
  constexpr int TM = 128, TN = 128, NT = 256, BK = 32, PITCH = 128 + 32, P = kParts<T>;
  constexpr bool HALF = std::is_same_v<T, _Float16>;
  using G = std::conditional_t<FACTOR, int8_t, T>;
  __shared__ __attribute__((aligned(16))) short lds[P + 1][BK][PITCH];
  __shared__ RowList<kSmallList> list;
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
  for (int base = 0; base < r_count; base += kSmallList) {
    const int64_t r0 = r_begin + base;
    const int n = list_rows<NT, false>(d.scale, r0, min(kSmallList, r_count - base), unit, list);
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

// ---- 256 x 256 tiles of the weight gradient ------------------------------------------

// Four waves of 128 x 128, steps of 32 rows, which go from memory into registers four steps ahead and
// from there into LDS one step ahead, the codes with their scales. Both operands lie in LDS a row a line of 512
// bytes, its groups of 16 bytes moved by 64 bytes a row, so that the 4 rows that 16 lanes of a
// transposing load meet lie in different banks. (Gradients sent from memory into LDS directly were
// slower: the compiler has every transposing load wait for all that is on its way there.)
//
// For outputs and inputs in whole groups of 8. Groups past the last column are the first one again:
// what they give is not stored.
constexpr int BT = 256, BROWS = 32, BSTAGE = BROWS * BT * 2, BAHEAD = 4;

template <class T>
__global__ void __launch_bounds__(256) grad_big_kernel(TnJob d) {
  constexpr bool HALF = std::is_same_v<T, _Float16>;
  __shared__ __attribute__((aligned(16))) char lds[4 * BSTAGE];
  __shared__ RowList<kBigList> list;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int v = xcd_virtual(blockIdx.x, gridDim.x, d.tiles * d.splits);
  if (v < 0) return;
  const int split = v / d.tiles, tile = v - split * d.tiles;
  // bands of 4 tiles of outputs, so that the tiles that run at a time on an XCD share both operands
  const int band = tile / (4 * d.nt), in = tile - band * 4 * d.nt, high = min(4, d.mt - 4 * band);
  const int ti = band * 4 + in % high, tj = in / high;
  const int o0 = ti * BT, k0 = tj * BT;
  const int64_t r_begin = int64_t(split) * d.per_split;
  const int r_count = static_cast<int>(min(int64_t(d.per_split), d.rows - r_begin));

  // this thread's group of 8 columns, and its rows 8 i + row of a step
  const int col = tid % 32, row = tid / 32, slot = col ^ (4 * (row & 3));
  const int g_col = o0 + 8 * col < d.m ? 8 * col : 0, q_col = k0 + 8 * col < d.n ? 8 * col : 0;
  const unsigned q_pitch = static_cast<unsigned>(d.ldq), g_pitch = static_cast<unsigned>(d.ldg) * 2;
  char* const gbuf = lds;
  char* const qbuf = lds + 2 * BSTAGE;
  v2u qraw[BAHEAD][4];
  v4u graw[BAHEAD][4];

  const int wm = (wave >> 1) * 128, wn = (wave & 1) * 128;
  v16f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  // Column sums of the gradients: the tiles along the inputs, and a tile's two waves that hold the same
  // outputs, take turns, a step each. A lane adds up its column of the operands.
  float sums[4] = {0.f, 0.f, 0.f, 0.f};
  const int turn = d.bias ? 2 * tj + (wave & 1) : INT32_MAX, turns = 2 * d.nt;
  auto add_up = [&](const v8s (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (HALF) sums[i] += static_cast<float>(__builtin_bit_cast(v8h, f[i])[k]);
        else sums[i] += __uint_as_float(unsigned(static_cast<unsigned short>(f[i][k])) << 16);
      }
  };
  const int s16 = lane & 15, kk = 8 * (lane >> 5) + (s16 >> 2), cc = 16 * ((lane >> 4) & 1) + 4 * (s16 & 3);
  // where this lane's loads of the wave's four groups of 32 columns begin in a buffer
  const char* ga[4];
  const char* qa[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = kk * 512 + ((cc >> 3) | ((i ^ (kk & 3)) << 2)) * 16 + (cc & 7) * 2;
    ga[i] = gbuf + 2 * wm + at;
    qa[i] = qbuf + 2 * wn + at;
  }
  auto operand = [&](const char* from) {  // 8 rows of a column each lane
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)from);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(from + 4 * 512));
    return v8s{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  auto mma1 = [&](v8s a, v8s b, v16f c) {
    if constexpr (HALF) return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
  };
  const float unit = HALF ? scale_unit<256>(d.scale, r_begin, r_count, list) : 1.f;
  for (int base = 0; base < r_count; base += kBigList) {
    const int64_t r0 = r_begin + base;
    const int n = list_rows<256, true>(d.scale, r0, min(kBigList, r_count - base), unit, list);
    const int steps = (n + BROWS - 1) / BROWS;
    if (!steps) continue;
    const KG char* const g0 = reinterpret_cast<const KG char*>(gp(static_cast<const T*>(d.g)) + r0 * d.ldg + o0 + g_col);
    const KG int8_t* const q0 = gp(d.q) + r0 * d.ldq + k0 + q_col;
    // this thread's four rows of step c, and their scales
    auto rows_of = [&](int c) { return *reinterpret_cast<const v4us*>(&list.idx[c * BROWS + 4 * row]); };
    auto scales_of = [&](int c) { return *reinterpret_cast<const v4f*>(&list.s[c * BROWS + 4 * row]); };
    // row i into registers
    auto fetch_q = [&](unsigned short r, auto set, int i) {
      qraw[set][i] = __builtin_bit_cast(v2u, *reinterpret_cast<const KG typename Pack<int8_t, 8>::vec*>(q0 + uint64_t(r & (kNone - 1)) * q_pitch));
    };
    auto fetch_g = [&](unsigned short r, auto set, int i) {
      graw[set][i] = __builtin_bit_cast(v4u, load_pack<false, T>(reinterpret_cast<const KG T*>(g0 + uint64_t(r & (kNone - 1)) * g_pitch)));
    };
    // row i from registers into LDS: the gradients, and the codes, two at a time; whole: it is no row that is none
    auto place_g = [&](auto set, auto buf, int i, bool whole, float s) {
      v4u x = graw[set][i];
      if (!whole && s == 0.f) x = v4u{0, 0, 0, 0};
      *reinterpret_cast<v4u*>(gbuf + buf * BSTAGE + (8 * i + row) * 512 + 16 * slot) = x;
    };
    v4u placed;
    auto place2 = [&](auto set, auto buf, int i, int h, float s) {
      placed[h] = two_codes<HALF>(qraw[set][i][h >> 1], h & 1, s);
      if (h == 3) *reinterpret_cast<v4u*>(qbuf + buf * BSTAGE + (8 * i + row) * 512 + 16 * slot) = placed;
    };
    v8s fa[2][4], fb[2][4];
    auto read1 = [&](auto buf, int ks, int set, int n) {
      if (n & 1) fb[set][n / 2] = operand(qa[n / 2] + buf * BSTAGE + 16 * ks * 512);
      else fa[set][n / 2] = operand(ga[n / 2] + buf * BSTAGE + 16 * ks * 512);
    };
#define KFAC_AT(x) std::integral_constant<int, (x)>{}
    auto first = [&](auto s) {
      if (s < steps) {
        const v4us r = rows_of(s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          fetch_q(r[i], s, i);
          fetch_g(r[i], s, i);
        }
      }
    };
    first(KFAC_AT(0));
    first(KFAC_AT(1));
    first(KFAC_AT(2));
    first(KFAC_AT(3));
    v4f sc = scales_of(0);
    auto place = [&](auto set, int i) {
      place_g(set, set, i, false, sc[i]);
#pragma unroll
      for (int h = 0; h < 4; ++h) place2(set, set, i, h, sc[i]);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) place(KFAC_AT(0), i);
    if (1 < steps) {
      sc = scales_of(1);
#pragma unroll
      for (int i = 0; i < 2; ++i) place(KFAC_AT(1), i);
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 8; ++n) read1(KFAC_AT(0), 0, 0, n);

    // One step: 16 products of its rows' first half, in whose shade the second half's operands are read and
    // the next step's last two rows of codes placed; then, when everyone has read this step's
    // operands and the next step's are there, 16 products of the second half, with the next step's
    // first operands read, the first two rows of the step after that placed, and step c + 4 fetched.
    int next = turn;
    auto step = [&](int c, auto S, auto ALL) {
      constexpr int s = decltype(S)::value;
      constexpr bool all = decltype(ALL)::value;
      v4us r = {0, 0, 0, 0};
      v4f sn = {0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        acc[n / 4][n % 4] = mma1(fa[0][n / 4], fb[0][n % 4], acc[n / 4][n % 4]);
        if (n < 8) read1(KFAC_AT(s & 1), 1, 1, n);
        if (n == 8 && (all || c + BAHEAD < steps)) r = rows_of(c + BAHEAD);
        if (n == 8 && (all || c + 2 < steps)) sn = scales_of(c + 2);
        if (all || c + 1 < steps) {
          if (n >= 8) place2(KFAC_AT((s + 1) & 3), KFAC_AT((s + 1) & 1), n / 4, n % 4, sc[n / 4]);
          if (n == 5 || n == 7) place_g(KFAC_AT((s + 1) & 3), KFAC_AT((s + 1) & 1), n / 2, all, sc[n / 2]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (c == next) {
        add_up(fa[0]);
        add_up(fa[1]);
        next += turns;
      }
      __syncthreads();
      sc = sn;
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        acc[n / 4][n % 4] = mma1(fa[1][n / 4], fb[1][n % 4], acc[n / 4][n % 4]);
        if (n < 8) read1(KFAC_AT((s + 1) & 1), 0, 0, n);
        if (n % 2 && (all || c + 2 < steps)) {
          place2(KFAC_AT((s + 2) & 3), KFAC_AT(s & 1), n / 8, n / 2 % 4, sc[n / 8]);
          if (n == 9 || n == 11) place_g(KFAC_AT((s + 2) & 3), KFAC_AT(s & 1), n / 2 - 4, all, sc[n / 2 - 4]);
        }
        if (n >= 8 && n < 12 && (all || c + BAHEAD < steps)) fetch_q(r[n - 8], KFAC_AT(s), n - 8);
        if (n >= 12 && (all || c + BAHEAD < steps)) fetch_g(r[n - 12], KFAC_AT(s), n - 12);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int c = 0;
    for (; (c + 4 + BAHEAD) * BROWS <= n; c += 4) {
      step(c, KFAC_AT(0), std::true_type{});
      step(c + 1, KFAC_AT(1), std::true_type{});
      step(c + 2, KFAC_AT(2), std::true_type{});
      step(c + 3, KFAC_AT(3), std::true_type{});
    }
    for (; c < steps; c += 4) {
      step(c, KFAC_AT(0), std::false_type{});
      if (c + 1 < steps) step(c + 1, KFAC_AT(1), std::false_type{});
      if (c + 2 < steps) step(c + 2, KFAC_AT(2), std::false_type{});
      if (c + 3 < steps) step(c + 3, KFAC_AT(3), std::false_type{});
    }
#undef KFAC_AT
  }
  const float back = 1.f / unit;  // exact: a power of two
  if (d.splits > 1) {
    KG float* part = gp(d.part) + (int64_t(split) * d.tiles + ti * d.nt + tj) * (BT * BT);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        KG float* o = part + (wm + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * BT + wn + (lane & 31);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[32 * j] = acc[i][j][e] * back;
      }
  } else {
    const int c = k0 + wn + (lane & 31);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int r = o0 + wm + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        KG float* o = gp(d.out) + int64_t(r) * d.ldo + c;
        if (r < d.m) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + 32 * j < d.n) {
              const float x = acc[i][j][e] * back;
              o[32 * j] = d.accumulate ? o[32 * j] + x : x;
            }
        }
      }
  }
  if (d.bias) {
    KG float* part = gp(d.part_col) + ((int64_t(split) * d.nt + tj) * 2 + (wave & 1)) * (int64_t(d.mt) * BT) + o0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = sums[i] + __shfl_xor(sums[i], 32);
      if (lane < 32) part[wm + 32 * i + lane] = x;
    }
  }
}

// What the splits and the shares of the column sums left, added up in their order. Blocks of 256 outputs; the
// last ones do the bias.
__global__ void __launch_bounds__(256) grad_join_kernel(TnJob d, int64_t groups) {
  const int64_t b = blockIdx.x;
  if (b < groups) {
    const int per_row = (d.n + 255) / 256;
    const int64_t r = b / per_row;
    const int c = static_cast<int>(b - r * per_row) * 256 + threadIdx.x;
    if (c >= d.n) return;
    const int64_t at = (r / BT * d.nt + c / BT) * (BT * BT) + (r % BT) * BT + c % BT;
    float sum = 0.f;
    for (int s = 0; s < d.splits; ++s) sum += gp(d.part)[int64_t(s) * d.tiles * (BT * BT) + at];
    KG float* o = gp(d.out) + r * d.ldo + c;
    *o = d.accumulate ? *o + sum : sum;
    return;
  }
  const int64_t r = (b - groups) * 256 + threadIdx.x;
  if (r >= d.m) return;
  float sum = 0.f;
  for (int s = 0; s < d.splits * d.nt * 2; ++s) sum += gp(d.part_col)[int64_t(s) * d.mt * BT + r];
  KG float* o = gp(d.bias_out) + r * d.inc_b;
  *o = d.accumulate ? *o + sum : sum;
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

// near: rows lie less than 2^32 bytes apart.
static TnJob grad_job(int32_t rows, int32_t c_in, int32_t c_out, kfac_dtype dtype, bool near) {
  TnJob j = {};
  j.rows = rows, j.m = c_out, j.n = c_in;
  plan(j, false);
  const int64_t mt = (int64_t(c_out) + BT - 1) / BT, nt = (int64_t(c_in) + BT - 1) / BT;
  if (dtype == KFAC_F32 || !near || c_in % 8 || c_out % 8 || mt * nt < 64 || rows < 256) return j;
  j.big = true;
  j.mt = static_cast<int32_t>(mt), j.nt = static_cast<int32_t>(nt), j.tiles = static_cast<int32_t>(mt * nt);
  j.per_split = rows, j.splits = 1;
  return j;
}

static void carve_grad(TnJob& j, Carver& cv) {
  if (!j.big) return carve(j, cv);
  if (j.splits > 1) j.part = cv.take<float>(size_t(j.splits) * j.tiles * BT * BT);
  j.part_col = cv.take<float>(size_t(j.splits) * j.nt * 2 * j.mt * BT);
}

template <class T>
static kfac_status launch_grad(const TnJob& j, hipStream_t s) {
  if constexpr (!std::is_same_v<T, float>) {
    if (j.big) {
      KFAC_LAUNCH(K_GRAD_Q8, grad_big_kernel<T>, dim3(xcd_grid(int64_t(j.tiles) * j.splits)), dim3(256), 0, s, j);
      KFAC_CHECK_LAUNCH("grad_big_kernel");
      const int64_t groups = j.splits > 1 ? int64_t(j.m) * ((j.n + 255) / 256) : 0;
      const int64_t all = groups + (j.bias ? (j.m + 255) / 256 : 0);
      if (all) {
        KFAC_LAUNCH(K_GRAD_Q8_JOIN, grad_join_kernel, dim3(static_cast<unsigned>(all)), dim3(256), 0, s, j, groups);
        KFAC_CHECK_LAUNCH("grad_join_kernel");
      }
      return KFAC_OK;
    }
  }
  return launch_tn<T, false>(j, s);
}

extern "C" kfac_status kfac_weight_grad_q8_workspace(int32_t rows, int32_t c_in, int32_t c_out, kfac_dtype dtype,
                                                     size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  if (!row_dtype(dtype)) return fail(KFAC_ERR_UNSUPPORTED, "dtype %d", dtype);
  kfac_status st = sizes_fit(rows, c_out, c_in);
  if (st) return st;
  *bytes = 0;
  for (bool near : {false, true}) {
    TnJob j = grad_job(rows, c_in, c_out, dtype, near);
    Carver cv;
    carve_grad(j, cv);
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
  const bool near = rows <= 1 || (ld_g < (int64_t(1) << 31) && ld_q < (int64_t(1) << 32));
  TnJob j = grad_job(rows, c_in, c_out, dtype, near);
  Carver sizing, cv(workspace);
  carve_grad(j, sizing);
  const RowsOf scr = scratch(workspace, sizing.used);
  if ((st = check_apart({&ws, &bs, &scr, &gs, &qs, &ss}, 3))) return st;
  if ((st = check_device())) return st;
  if ((st = check_workspace(workspace, ws_bytes, sizing.used))) return st;
  carve_grad(j, cv);
  j.g = gout, j.q = q, j.scale = scale, j.out = dweight, j.bias_out = dbias;
  j.ldg = ld_g, j.ldq = ld_q, j.ldo = ld_dw, j.inc_b = inc_db, j.bias = dbias != nullptr, j.accumulate = accumulate;
  return with_row_type(dtype, [&](auto tag) { return launch_grad<decltype(tag)>(j, static_cast<hipStream_t>(stream)); });
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
