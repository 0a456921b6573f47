// The kernels of q8_tn.hpp, for the files that instantiate them.
#pragma once
#include "q8_tn.hpp"

namespace kfac {

// fp32 gradients are formed in three bf16 parts.
template <class T>
constexpr int kParts = std::is_same_v<T, float> ? 3 : 1;

// Codes 2 h and 2 h + 1 of four, times s, as two 16-bit numbers.
template <bool HALF>
__device__ inline unsigned two_codes(unsigned four, int h, float s) {
  if constexpr (HALF) {
    // code + 128 = b, and 0x64 in front of b is the fp16 number 1024 + b
    const v2h mid = {static_cast<_Float16>(1152.f), static_cast<_Float16>(1152.f)};
    const _Float16 sh = static_cast<_Float16>(s);
    const unsigned b = __builtin_amdgcn_perm(0x64646464u, four ^ 0x80808080u, h ? 0x04030402u : 0x04010400u);
    return __builtin_bit_cast(unsigned, (__builtin_bit_cast(v2h, b) - mid) * v2h{sh, sh});
  } else {  // the code itself times s: its own byte's conversion and a product, finite wherever s q is
    auto code = [&](int k) { return static_cast<float>(static_cast<int8_t>(four >> (8 * k))); };
    const v2bf out = {static_cast<__bf16>(code(2 * h) * s), static_cast<__bf16>(code(2 * h + 1) * s)};
    return __builtin_bit_cast(unsigned, out);
  }
}

template <bool HALF>
__device__ inline v8s codes16(v2u u, float s) {
  return __builtin_bit_cast(v8s, v4u{two_codes<HALF>(u[0], 0, s), two_codes<HALF>(u[0], 1, s),
                                     two_codes<HALF>(u[1], 0, s), two_codes<HALF>(u[1], 1, s)});
}

// What all lanes share, in scalar registers.
__device__ inline int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ inline float uniform(float x) { return __uint_as_float(uniform(static_cast<int>(__float_as_uint(x)))); }
template <typename P>
__device__ inline KG P* uniform(KG P* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint64_t lo = static_cast<unsigned>(uniform(static_cast<int>(a)));
  const uint64_t hi = static_cast<unsigned>(uniform(static_cast<int>(a >> 32)));
  return reinterpret_cast<KG P*>(hi << 32 | lo);
}

// x = h[0] + h[1] + h[2], 8 bits of the significand each, cut and not rounded. An infinity stays one.
__device__ inline void cut3(float x, short (&h)[3]) {
  float r = x;
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const unsigned b = __float_as_uint(r) & 0xffff0000u;
    h[p] = static_cast<short>(b >> 16);
    const float top = __uint_as_float(b);
    r = p == 0 && r == top ? 0.f : r - top;  // what is left of the first cut is finite, or NaN
  }
}
// The same of two numbers, each part's two 16 bits in one register.
__device__ inline void cut3(float x, float y, unsigned (&h)[3]) {
  float r[2] = {x, y};
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const unsigned b[2] = {__float_as_uint(r[0]), __float_as_uint(r[1])};
    h[p] = __builtin_amdgcn_perm(b[1], b[0], 0x07060302u);  // the upper halves
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float top = __uint_as_float(b[k] & 0xffff0000u);
      r[k] = p == 0 && r[k] == top ? 0.f : r[k] - top;
    }
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
template <int NT, int LIST>
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
      l.idx[at] = static_cast<uint16_t>((wave + i * (NT / 64)) * 64 + lane);
      const float scaled = s[i] * unit;
      l.s[at] = scaled == 0.f ? 1.17549435e-38f : scaled;  // 0 stands for no row: one far below the unit is none of those
    }
  }
  const int whole = (total + 63) / 64 * 64;
  if (total + tid < whole) {
    l.idx[total + tid] = kNone;
    l.s[total + tid] = 0.f;
  }
  __syncthreads();
  return total;
}

// 2^k such that the largest finite scale of the rows times it is 2^5: relative to that, fp16 holds
// s q down to 2^-29 of the largest scale exactly (the sum with 1152 that makes a code stays finite).
// scratch: NT / 64 floats.
template <int NT>
__device__ inline float scale_unit(const float* scale, int64_t r0, int n, float* scratch) {
  unsigned top = 0;
  for (int r = threadIdx.x; r < n; r += NT) {
    const unsigned b = __float_as_uint(gp(scale)[r0 + r]) & 0x7fffffffu;
    if (b < 0x7f800000u) top = max(top, b);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, __shfl_xor(top, o));
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = __uint_as_float(top);
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < NT / 64; ++i) t = fmaxf(t, scratch[i]);
  __syncthreads();
  int e = static_cast<int>(__float_as_uint(t) >> 23);  // 2^(e - 127) <= t
  e = 127 + 5 - (e - 127);                              // of 2^5 / 2^(e - 127)
  return __uint_as_float(static_cast<unsigned>(max(1, min(e, 253))) << 23);
}


// Tiles of T x T, T = 64 F, four waves of 32 F x 32 F, steps of 32 rows, which go from memory into registers AHEAD
// steps ahead and from there into LDS one step ahead, the codes with their scales and fp32 gradients cut
// into their parts. An operand lies in LDS a row a line of T 16-bit numbers, its groups of 8 moved by 4 in
// turn, so that the 4 rows that 16 lanes of a transposing load meet lie in different banks. (Gradients
// sent from memory into LDS directly were slower: the compiler has every transposing load wait for
// all that is on its way there.)
//
// 8192 x 4096 x 4096 bf16, 5570 rows of which count: 179 us, 1.04e15 operations a second, with tiles of 256 (128: 282); the
// library's product of 16-bit operands that lie so runs at 1.16e15. What is left is a block's start and end, 25 us,
// and the steps' one barrier. 4099 x 1001 x 777 fp32, three products: 39 us, bound by the cutting (250 vector
// instructions a thread and step).
//
// A thread holds F groups of 8 columns of each operand a step. RAGGED: the last group of a row that has
// no 8 columns left is read from 8 columns before the row's end, and shifted. Groups past the end are the
// first one again: what they give is not stored.
constexpr int kStep = 32;

template <int F>
struct Tile {
  static constexpr int T = 64 * F, LINE = 2 * T, OPERAND = kStep * LINE, GROUPS = T / 8, LIST = F == 2 ? 2048 : 8192;
  // by how many groups a row's line is moved
  static __device__ inline int moved(int row) { return (row & 3) << 2; }
};

// What a thread reads of a group of 8, as it comes from memory.
template <class E>
struct Raw8 {  // 16-bit elements
  v4u w;
  __device__ inline void load(const KG char* p) { w = __builtin_bit_cast(v4u, load_pack<false, short>(reinterpret_cast<const KG short*>(p))); }
  __device__ inline void shift(int k) {  // drops the first k elements
    uint64_t lo = uint64_t(w[1]) << 32 | w[0], hi = uint64_t(w[3]) << 32 | w[2];
    const int b = 16 * (k & 3);
    if (k & 4) lo = hi, hi = 0;
    lo = lo >> b | (b ? hi << (64 - b) : 0);
    hi >>= b;
    w = v4u{unsigned(lo), unsigned(lo >> 32), unsigned(hi), unsigned(hi >> 32)};
  }
};
template <>
struct Raw8<float> {
  float x[8];
  __device__ inline void load(const KG char* p) {
    const KG float* f = reinterpret_cast<const KG float*>(p);
    const v4f a = load_pack<false, float>(f), b = load_pack<false, float>(f + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = a[k], x[4 + k] = b[k];
  }
  __device__ inline void shift(int k) {
#pragma unroll
    for (int b = 1; b < 8; b *= 2)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = k & b ? (i + b < 8 ? x[i + b] : 0.f) : x[i];
  }
};
template <>
struct Raw8<int8_t> {
  v2u w;
  __device__ inline void load(const KG char* p) { w = __builtin_bit_cast(v2u, *reinterpret_cast<const KG typename Pack<int8_t, 8>::vec*>(reinterpret_cast<const KG int8_t*>(p))); }
  __device__ inline void shift(int k) { w = __builtin_bit_cast(v2u, (uint64_t(w[1]) << 32 | w[0]) >> (8 * k)); }
};

// An entry of a factor: blended with the stored one, also into the full matrix.
struct PutFactor {
  KG float* out;
  KG float* full;
  float decay;
  bool any;  // rows that count
  int64_t order;
  __device__ inline void operator()(int64_t r, int64_t c, float v) const {
    const int64_t o = packed_off(r, c, order);
    if (decay != 0.f) {
      const float old = out[o];
      v = any ? decay * old + (1.f - decay) * v : old;
    }
    out[o] = v;
    if (full) full[r * order + c] = v;
  }
  // N entries (r[k], c[k]) at a time, of which `live` are written: the stored ones are on their way together
  template <int N>
  __device__ inline void all(const int (&r)[N], const int (&c)[N], const bool (&live)[N], float (&v)[N]) const {
    int64_t o[N];
#pragma unroll
    for (int k = 0; k < N; ++k) o[k] = live[k] ? packed_off(r[k], c[k], order) : 0;
    if (decay != 0.f) {
      float old[N];
#pragma unroll
      for (int k = 0; k < N; ++k) old[k] = out[o[k]];
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = any ? decay * old[k] + (1.f - decay) * v[k] : old[k];
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (live[k]) out[o[k]] = v[k];
    if (!full) return;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (live[k]) full[r[k] * order + c[k]] = v[k];
  }
};
__device__ inline PutFactor put_factor(const TnJob& d, int counted) {
  return {gp(d.out), gp(d.full), d.decay, counted > 0, int64_t(d.m) + d.bias};
}
// The bias column's own entry: the rows' ones, NaN as all of the factor if one of them has a scale that is none.
__device__ inline float corner(int counted, bool bad) {
  return bad ? __uint_as_float(0x7fc00000u) : counted ? 1.f : 0.f;
}
__device__ inline void put_grad(KG float* o, float v, int accumulate) { *o = accumulate ? *o + v : v; }

template <class E, int F, bool RAGGED>
__global__ void __launch_bounds__(256, F == 2 ? 2 : 1) grad_tile_kernel(TnArgs<false> args) {
  using L = Tile<F>;
  constexpr int T = L::T, P = kParts<E>, W = 32 * F;
  constexpr bool HALF = std::is_same_v<E, _Float16>;
  __shared__ __attribute__((aligned(16))) char lds[2 * (P + 1) * L::OPERAND];
  __shared__ RowList<L::LIST> list;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int v = xcd_virtual(blockIdx.x, gridDim.x, args.items);
  if (v < 0) return;
  const TnJob& d = args.j[0];
  const int item = v - d.begin, split = item / d.tiles, tile = item - split * d.tiles;
  // bands of 4 tiles of outputs, so that the tiles that run at a time on an XCD share both operands
  const int band = tile / (4 * d.nt), in = tile - band * 4 * d.nt, high = min(4, d.mt - 4 * band);
  const int ti = band * 4 + in % high, tj = in / high;
  const int o0 = ti * T, k0 = tj * T;
  const int64_t r_begin = int64_t(split) * d.per_split;
  const int r_count = static_cast<int>(min(int64_t(d.per_split), d.rows - r_begin));
  char* const abuf = lds;
  char* const bbuf = lds + 2 * P * L::OPERAND;

  // this thread's groups: row of a step, place in its line, byte offset in its rows, elements to shift out
  int row[F], at[F], a_col[F], b_col[F], a_cut[F], b_cut[F];
#pragma unroll
  for (int i = 0; i < F; ++i) {
    const int u = tid + 256 * i, c = 8 * (u % L::GROUPS);
    row[i] = u / L::GROUPS;
    at[i] = row[i] * L::LINE + 16 * ((u % L::GROUPS) ^ L::moved(row[i]));
    auto column = [&](int c, int end, int& off, int& cut) {
      off = c + 8 <= end ? c : RAGGED && c < end ? end - 8 : 0;
      cut = RAGGED && c < end && c + 8 > end ? c + 8 - end : 0;
    };
    column(o0 + c, d.m, a_col[i], a_cut[i]);
    column(k0 + c, d.n, b_col[i], b_cut[i]);
    a_col[i] *= sizeof(E);
  }
  bool cuts = false;  // of the wave: only the last tiles of ragged operands have any
  if constexpr (RAGGED) {
#pragma unroll
    for (int i = 0; i < F; ++i) cuts |= (a_cut[i] | b_cut[i]) != 0;
    cuts = __any(cuts);
  }
  // steps fetched ahead (three of fp32: a fourth's registers spill, 43.6 against 39.3 us for 4099 x 1001 x 777), and the
  // steps after which registers and buffers come round
  constexpr int AHEAD = P == 3 ? 3 : 4, ROUND = P == 3 ? 6 : 4;
  Raw8<E> araw[AHEAD][F];
  Raw8<int8_t> braw[AHEAD][F];

  const int wm = (wave >> 1) * W, wn = (wave & 1) * W;
  v16f acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  // Column sums of the first operand: the tiles of a row of tiles, and a tile's two waves that hold the same
  // columns, take turns, a step each; or the row's first tile does all. A lane adds up its column.
  const bool sums_here = d.bias && (!d.solo || tj == 0);
  float sums[F];
#pragma unroll
  for (int i = 0; i < F; ++i) sums[i] = 0.f;
  const int turns = d.solo ? 2 : 2 * d.nt, turn = (d.solo ? 0 : 2 * tj) + (wave & 1);
  const int s16 = lane & 15, kk = 8 * (lane >> 5) + (s16 >> 2), cc = 16 * ((lane >> 4) & 1) + 4 * (s16 & 3);
  // where this lane's loads of the wave's groups of 32 columns begin in a buffer
  const char* fa_at[F];
  const char* fb_at[F];
#pragma unroll
  for (int i = 0; i < F; ++i) {
    auto place = [&](int c) { return kk * L::LINE + 16 * (((c + cc) >> 3) ^ L::moved(kk)) + (cc & 7) * 2; };
    fa_at[i] = abuf + place(wm + 32 * i);
    fb_at[i] = bbuf + place(wn + 32 * i);
  }
  auto operand = [&](const char* from) {  // 8 rows of a column each lane
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)from);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(from + 4 * L::LINE));
    return v8s{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  const float unit = HALF ? scale_unit<256>(d.scale, r_begin, r_count, list.top) : 1.f;
  const unsigned a_pitch = static_cast<unsigned>(d.ldg * int64_t(sizeof(E))), b_pitch = static_cast<unsigned>(d.ldq);
  for (int base = 0; base < r_count; base += L::LIST) {
    const int64_t r0 = r_begin + base;
    const int n = list_rows<256>(d.scale, r0, min(L::LIST, r_count - base), unit, list);
    const int steps = (n + kStep - 1) / kStep;
    if (!steps) continue;
    const KG char* const b0 = uniform(reinterpret_cast<const KG char*>(gp(d.q)) + r0 * d.ldq);
    const KG char* const a0 = uniform(gp(static_cast<const char*>(d.g)) + r0 * d.ldg * int64_t(sizeof(E)));
    // rows of a step from the list, and their scales
    auto rows_of = [&](int c, int (&r)[F]) {
#pragma unroll
      for (int i = 0; i < F; ++i) r[i] = list.idx[c * kStep + row[i]] & (kNone - 1);
    };
    auto scales_of = [&](int c, float (&s)[F]) {
#pragma unroll
      for (int i = 0; i < F; ++i) s[i] = list.s[c * kStep + row[i]];
    };
    auto fetch = [&](auto set, int k, const int (&r)[F]) {  // 2 F loads
      const int i = k / 2;
      if (k & 1) araw[set][i].load(a0 + uint64_t(unsigned(r[i])) * a_pitch + a_col[i]);
      else braw[set][i].load(b0 + uint64_t(unsigned(r[i])) * b_pitch + b_col[i]);
    };
    // A group's way from registers into LDS, in 8 parts: two codes each, or two gradients each of fp32, or all of
    // the 16-bit ones at the first. whole: the row is no row that is none.
    v4u made, parts[P == 3 ? 3 : 1];
    auto place = [&](auto set, auto buf, int k, bool whole, const float (&s)[F]) {
      const int i = k / 8, h = k % 4;
      if (k % 8 < 4) {
        if constexpr (RAGGED)
          if (h == 0 && cuts) braw[set][i].shift(b_cut[i]);
        made[h] = two_codes<HALF>(braw[set][i].w[h >> 1], h & 1, s[i]);
        if (h == 3) *reinterpret_cast<v4u*>(bbuf + buf * L::OPERAND + at[i]) = made;
        return;
      }
      if constexpr (RAGGED)
        if (h == 0 && cuts) araw[set][i].shift(a_cut[i]);
      char* const to = abuf + buf * P * L::OPERAND + at[i];
      if constexpr (P == 1) {
        if (h == 0) {
          v4u x = araw[set][i].w;
          if (!whole && s[i] == 0.f) x = v4u{0, 0, 0, 0};
          *reinterpret_cast<v4u*>(to) = x;
        }
      } else {
        unsigned two[3];
        float x0 = araw[set][i].x[2 * h], x1 = araw[set][i].x[2 * h + 1];
        if (!whole && s[i] == 0.f) x0 = x1 = 0.f;
        cut3(x0, x1, two);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          parts[p][h] = two[p];
          if (h == 3) *reinterpret_cast<v4u*>(to + p * L::OPERAND) = parts[p];
        }
      }
    };
    v8s fa[2][P][F], fb[2][F];
    constexpr int R = (P + 1) * F, N = P * F * F;  // operands and products of 16 rows
    auto read = [&](auto buf, int ks, int set, int k) {
      if (k < F) fb[set][k] = operand(fb_at[k] + buf * L::OPERAND + 16 * ks * L::LINE);
      else fa[set][k / F - 1][k % F] = operand(fa_at[k % F] + (buf * P + k / F - 1) * L::OPERAND + 16 * ks * L::LINE);
    };
    auto mma = [&](int set, int n) {  // smallest parts first
      const int p = P - 1 - n / (F * F), i = n / F % F, j = n % F;
      if constexpr (HALF) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, fa[set][p][i]), __builtin_bit_cast(v8h, fb[set][j]), acc[i][j], 0, 0, 0);
      else acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, fa[set][p][i]), __builtin_bit_cast(v8b, fb[set][j]), acc[i][j], 0, 0, 0);
    };
    auto add_up = [&](int set) {
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int p = P - 1; p >= 0; --p) {
            if constexpr (HALF) sums[i] += static_cast<float>(__builtin_bit_cast(v8h, fa[set][p][i])[k]);
            else sums[i] += __uint_as_float(unsigned(static_cast<unsigned short>(fa[set][p][i][k])) << 16);
          }
    };
#define KFAC_AT(x) std::integral_constant<int, (x)>{}
    int r[F];
    float sc[F], sn[F];
    auto first = [&](auto s) {
      if (s < steps) {
        rows_of(s, r);
#pragma unroll
        for (int k = 0; k < 2 * F; ++k) fetch(s, k, r);
      }
    };
    first(KFAC_AT(0));
    first(KFAC_AT(1));
    first(KFAC_AT(2));
    if constexpr (AHEAD == 4) first(KFAC_AT(3));
    constexpr int EARLY = F / 2;  // groups that are placed two steps ahead, the others one
    scales_of(0, sc);
#pragma unroll
    for (int k = 0; k < 8 * F; ++k) place(KFAC_AT(0), KFAC_AT(0), k, false, sc);
    if (1 < steps) {
      scales_of(1, sc);
#pragma unroll
      for (int k = 0; k < 8 * EARLY; ++k) place(KFAC_AT(1), KFAC_AT(1), k, false, sc);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < R; ++k) read(KFAC_AT(0), 0, 0, k);

    // One step: the products of its first 16 rows, in whose shade the other 16 rows' operands are read and the
    // next step's last groups placed; then, when everyone has read this step's operands and the
    // next step's are there, the products of the other rows, with the next step's first operands read, the first
    // groups of the step after that placed, and step c + AHEAD fetched.
    int next = sums_here ? turn : INT32_MAX;
    auto step = [&](int c, auto S, auto ALL) {
      constexpr int s = decltype(S)::value;
      constexpr bool all = decltype(ALL)::value;
      constexpr int K1 = R + 8 * (F - EARLY), K2 = R + 8 * EARLY + 2 * F;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        mma(0, n);
        if (n == N / 2 && (all || c + AHEAD < steps)) rows_of(c + AHEAD, r);
        if (n == N / 2 && (all || c + 2 < steps)) scales_of(c + 2, sn);
#pragma unroll
        for (int k = n * K1 / N; k < (n + 1) * K1 / N; ++k) {
          if (k < R) read(KFAC_AT(s & 1), 1, 1, k);
          else if (all || c + 1 < steps) place(KFAC_AT((s + 1) % AHEAD), KFAC_AT((s + 1) & 1), 8 * EARLY + k - R, all, sc);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (c == next) {
        add_up(0);
        add_up(1);
        next += turns;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < F; ++i) sc[i] = sn[i];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        mma(1, n);
#pragma unroll
        for (int k = n * K2 / N; k < (n + 1) * K2 / N; ++k) {
          if (k < R) read(KFAC_AT((s + 1) & 1), 0, 0, k);
          else if (k < R + 8 * EARLY) {
            if (all || c + 2 < steps) place(KFAC_AT((s + 2) % AHEAD), KFAC_AT(s & 1), k - R, all, sc);
          } else if (all || c + AHEAD < steps) {
            fetch(KFAC_AT(s % AHEAD), k - R - 8 * EARLY, r);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int c = 0;
    for (; (c + ROUND + AHEAD) * kStep <= n; c += ROUND) {
      step(c, KFAC_AT(0), std::true_type{});
      step(c + 1, KFAC_AT(1), std::true_type{});
      step(c + 2, KFAC_AT(2), std::true_type{});
      step(c + 3, KFAC_AT(3), std::true_type{});
      if constexpr (ROUND == 6) {
        step(c + 4, KFAC_AT(4), std::true_type{});
        step(c + 5, KFAC_AT(5), std::true_type{});
      }
    }
    for (; c < steps; c += ROUND) {
      step(c, KFAC_AT(0), std::false_type{});
      if (c + 1 < steps) step(c + 1, KFAC_AT(1), std::false_type{});
      if (c + 2 < steps) step(c + 2, KFAC_AT(2), std::false_type{});
      if (c + 3 < steps) step(c + 3, KFAC_AT(3), std::false_type{});
      if constexpr (ROUND == 6) {
        if (c + 4 < steps) step(c + 4, KFAC_AT(4), std::false_type{});
        if (c + 5 < steps) step(c + 5, KFAC_AT(5), std::false_type{});
      }
    }
#undef KFAC_AT
  }

  // a lane's accumulators: column lane % 32, rows 8 (e / 4) + 4 (lane / 32) + e % 4
  const float back = 1.f / unit;  // exact: a power of two
  if (d.splits > 1) {
    KG float* part = gp(d.part) + (int64_t(split) * d.tiles + ti * d.nt + tj) * (T * T);
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        KG float* o = part + (wm + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * T + wn + (lane & 31);
#pragma unroll
        for (int j = 0; j < F; ++j) o[32 * j] = acc[i][j][e] * back;
        __builtin_amdgcn_sched_barrier(0);
      }
  } else {
    const int c = k0 + wn + (lane & 31);
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int rr = o0 + wm + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
        if (rr < d.m) {
          KG float* o = gp(d.out) + int64_t(rr) * d.ldo + c;
#pragma unroll
          for (int j = 0; j < F; ++j)
            if (c + 32 * j < d.n) put_grad(o + 32 * j, acc[i][j][e] * back, d.accumulate);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
  }
  if (!sums_here) return;
#pragma unroll
  for (int i = 0; i < F; ++i) sums[i] += __shfl_xor(sums[i], 32);
  if (!d.solo) {
    KG float* part = gp(d.part_col) + (int64_t(split) * d.shares + turn) * (int64_t(d.mt) * T) + o0;
#pragma unroll
    for (int i = 0; i < F; ++i)
      if (lane < 32) part[wm + 32 * i + lane] = sums[i];
    return;
  }
  float* const other = reinterpret_cast<float*>(lds);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < F; ++i)
    if ((wave & 1) && lane < 32) other[wm + 32 * i + lane] = sums[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < F; ++i) {
    const int c = o0 + wm + 32 * i + lane;
    if ((wave & 1) || lane >= 32 || c >= d.m) continue;
    put_grad(gp(d.bias_out) + c * d.inc_b, sums[i] + other[wm + 32 * i + lane], d.accumulate);
  }
}

template <class T, int F, bool RAGGED>
kfac_status launch_grad_tiles(const TnArgs<false>& a, hipStream_t s) {
  KFAC_LAUNCH(K_GRAD_Q8, (grad_tile_kernel<T, F, RAGGED>), dim3(xcd_grid(a.items)), dim3(256), 0, s, a);
  KFAC_CHECK_LAUNCH("grad_tile_kernel");
  return KFAC_OK;
}

}  // namespace kfac
