// Rows in 8 bits: quantising, reading back, and the product in 8-bit integers.
//
// A row x with m = max |x| becomes q = round half to even (x / s), s the smallest power of two
// >= m / 127 (or, for weights, m / 127 rounded to fp32). The power of two costs up to one of the
// eight bits and makes s q a bf16 exactly, so that what is summed over the rows later (weight
// gradients, Kronecker factors) takes it as a matrix instruction's operand with no rounding.
// Both divisions are exact decisions: by a power of two nothing is rounded before the whole
// number is; otherwise the candidate of an fp32 product is put right by its exact remainder.
#include "q8.hpp"

namespace kfac {

constexpr float kMinScale = 1.17549435e-38f;  // 2^-126

// The smallest power of two >= amax / 127, of amax's bits (finite); at least 2^-126.
__device__ inline unsigned pow2_scale_bits(unsigned amax) {
  // 127 = 1.984375 * 2^6: a significand up to that needs 2^(E-6), a larger one 2^(E-5)
  const int e = static_cast<int>(amax >> 23) - 6 + ((amax & 0x7fffff) > 0x7e0000);
  return static_cast<unsigned>(max(e, 1)) << 23;
}

// Scale of a row whose largest magnitude has the bits `amax` (integers order non-negative floats, and
// put infinities and NaN on top).
template <bool POW2>
__device__ inline float row_scale(unsigned amax) {
  if (amax >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  if (amax == 0) return 1.f;
  if (POW2) return __uint_as_float(pow2_scale_bits(amax));
  return fmaxf(__uint_as_float(amax) / 127.f, kMinScale);
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a sum with it holds the rounded whole number in its low bits

// How a row of largest magnitude `amax` (its bits) is written: a scale, its reciprocal, and the largest code.
struct RowCode {
  float s, inv;
  int most;  // 127; 63 where 64 s would be infinite; 0 in a row with an infinity or a NaN
};

template <bool POW2>
__device__ inline RowCode row_code(unsigned amax) {
  RowCode c;
  c.s = row_scale<POW2>(amax);
  c.inv = 1.f / c.s;
  c.most = amax >= 0x7f800000u ? 0 : POW2 && c.s >= 5.316911983139664e36f ? 63 : 127;  // 2^122
  return c;
}

// The code of one element in the low 8 bits.
template <bool POW2>
__device__ inline unsigned code_of(float x, const RowCode& c) {
  const float m = fmaf(x, c.inv, kMagic);  // by a power of two exact but for this one rounding
  if constexpr (POW2) {
    return __float_as_uint(m);
  } else {
    // x - t s is exact (below a step, and a multiple of the smaller of both last places): put
    // right what the rounded reciprocal decided next to a half, ties to the even side
    float t = m - kMagic;
    // (against twice it: half the smallest scales is no float)
    const float d = fmaf(-t, c.s, x);
    const float twice = 2.f * fabsf(d);
    if (twice > c.s || (twice == c.s && (static_cast<int>(t) & 1))) t += copysignf(1.f, d);
    return static_cast<unsigned>(static_cast<int>(__builtin_amdgcn_fmed3f(t, -127.f, 127.f)));
  }
}

// 8 elements of a row in registers as they came, and as floats.
template <class T>
struct Eight {
  static constexpr int W = sizeof(T) * 2;  // words
  unsigned w[W];
  __device__ inline float get(int k) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[k]);
    else if constexpr (std::is_same_v<T, __bf16>) return __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
    else return static_cast<float>(__builtin_bit_cast(v2h, w[k / 2])[k & 1]);
  }
  __device__ inline void load(const KG T* p, int left) {  // `left` elements are the row's
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
    if (left >= 8) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const v4u v = __builtin_bit_cast(v4u, load_pack<false, T>(p + i * 4 / sizeof(T)));
        w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) {
          if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(p[k]);
          else w[k / 2] |= unsigned(__builtin_bit_cast(unsigned short, T(p[k]))) << (16 * (k & 1));
        }
    }
  }
  // bits of the largest magnitude (infinities and NaN are larger than every number)
  __device__ inline unsigned top(unsigned m) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(get(k)) & 0x7fffffffu);
    return m;
  }
  template <bool POW2>
  __device__ inline v2u coded(const RowCode& c) const {
    v2u out = {0, 0};
    if (c.most == 127) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unsigned b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = code_of<POW2>(get(4 * h + k), c);
        out[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u), __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
      }
    } else if (c.most) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int q = static_cast<int8_t>(code_of<POW2>(get(k), c));
        out[k / 4] |= unsigned(uint8_t(max(-c.most, min(c.most, q)))) << (8 * (k & 3));
      }
    }
    return out;
  }
  static __device__ inline void put(KG int8_t* p, int left, v2u out) {
    if (left >= 8) {
      *reinterpret_cast<KG typename Pack<int8_t, 8>::vec*>(p) = __builtin_bit_cast(typename Pack<int8_t, 8>::vec, out);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) p[k] = static_cast<int8_t>(out[k / 4] >> (8 * (k & 3)));
    }
  }
};

// TPR threads a row (a wave, or the block), each with U groups of 8 elements kept in registers between the
// largest magnitude and the codes; U = 0: rows of any length, read twice.
template <class T, bool POW2, int TPR, int U>
__global__ void __launch_bounds__(256) quantize_rows_kernel(int rows, int cols, const T* __restrict__ x, int64_t ld,
                                                            const uint8_t* __restrict__ mask, int8_t* __restrict__ q,
                                                            int64_t ldq, float* __restrict__ scale) {
  const int t = threadIdx.x % TPR;
  const int64_t row = int64_t(blockIdx.x) * (256 / TPR) + threadIdx.x / TPR;
  if (row >= rows) return;
  const KG T* xr = gp(x) + row * ld;
  KG int8_t* qr = gp(q) + row * ldq;
  const unsigned end = cols;  // unsigned: a column past the last may lie past the largest int
  if (mask && !gp(mask)[row]) {
    for (unsigned c = 8 * t; c < end; c += 8 * TPR) Eight<T>::put(qr + c, end - c, v2u{0, 0});
    if (t == 0) gp(scale)[row] = 0.f;
    return;
  }
  Eight<T> v[U ? U : 1];
  unsigned top = 0;
  if constexpr (U) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u].load(xr + 8 * (t + u * TPR), cols - 8 * (t + u * TPR));
#pragma unroll
    for (int u = 0; u < U; ++u) top = v[u].top(top);
  } else {
    for (unsigned c = 8 * t; c < end; c += 8 * TPR) {
      v[0].load(xr + c, end - c);
      top = v[0].top(top);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, __shfl_xor(top, o));
  if constexpr (TPR > 64) {
    __shared__ unsigned part[4];
    if ((t & 63) == 0) part[t >> 6] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
  }
  const RowCode code = row_code<POW2>(top);
  if constexpr (U) {
#pragma unroll
    for (int u = 0; u < U; ++u) Eight<T>::put(qr + 8 * (t + u * TPR), cols - 8 * (t + u * TPR), v[u].template coded<POW2>(code));
  } else {
    for (unsigned c = 8 * t; c < end; c += 8 * TPR) {
      v[0].load(xr + c, end - c);
      Eight<T>::put(qr + c, end - c, v[0].template coded<POW2>(code));
    }
  }
  if (t == 0) gp(scale)[row] = code.s;
}

template <class T>
__device__ inline T held(float v) {
  constexpr float most = std::is_same_v<T, _Float16> ? 65504.f
                         : std::is_same_v<T, float>  ? 3.4028234663852886e38f
                                                     : 3.3895313892515355e38f;
  if (fabsf(v) > most) v = copysignf(most, v);
  return static_cast<T>(v);
}

// 8192 x 4096 bf16: 16.5 us, 6.1 TB/s. Groups of 8 elements, numbered through the rows, one a thread.
template <class T>
__global__ void __launch_bounds__(256) dequantize_rows_kernel(int cols, unsigned per_row, unsigned groups,
                                                              const int8_t* __restrict__ q, int64_t ldq,
                                                              const float* __restrict__ scale, T* __restrict__ x,
                                                              int64_t ld) {
  const unsigned g = blockIdx.x * 256 + threadIdx.x;
  if (g >= groups) return;
  const int64_t row = g / per_row;
  const int c = static_cast<int>(g % per_row) * 8, left = cols - c;
  const float s = gp(scale)[row];
  const KG int8_t* from = gp(q) + row * ldq + c;
  KG T* to = gp(x) + row * ld + c;
  if (left >= 8) {
    const auto v = *reinterpret_cast<const KG typename Pack<int8_t, 8>::vec*>(from);
    constexpr int EV = 16 / sizeof(T);
#pragma unroll
    for (int k = 0; k < 8; k += EV) {
      typename Pack<T>::vec out;
#pragma unroll
      for (int e = 0; e < EV; ++e) out[e] = held<T>(static_cast<float>(v[k + e]) * s);
      store_pack<false, T>(to + k, out);
    }
  } else {
    for (int k = 0; k < left; ++k) to[k] = held<T>(static_cast<float>(from[k]) * s);
  }
}

// ---- y = fp32(sum of q w) s v + b ------------------------------------------------

struct LinearArgs {
  int rows, c_in, c_out;
  int8_t* q;
  const int8_t* w;
  float* scale;
  const float* w_scale;
  const void* bias;
  void* y;
  int64_t ldq, ldw, ldy;
};

// A row with scale 0 takes no part, whatever the channel's scale holds.
__device__ inline float entry(int sum, float s, float v, float b) {
  return s == 0.f ? b : static_cast<float>(sum) * s * v + b;
}

// 16 codes of a row at k0, zeros past its end; nothing behind the row is read.
__device__ inline v4i load_codes(const KG int8_t* row, int k0, int c_in) {
  if (k0 + 16 <= c_in) return __builtin_bit_cast(v4i, load_pack<false, int8_t>(row + k0));
  v4i v = {0, 0, 0, 0};
  for (int k = 0; k < 16 && k0 + k < c_in; ++k) {
    const int byte = int(uint8_t(row[k0 + k])) << (8 * (k & 3));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] |= (k >> 2) == i ? byte : 0;
  }
  return v;
}

// Tiles of 2 WT channels x 2 WT rows, four waves of WT x WT. The weights are the matrix instruction's
// first operand, so that a lane holds 4 neighbouring channels of one row. Both operands lie along
// the sum: 16 codes are 16 bytes of an LDS line, which holds the tile's rows of BK codes with their
// groups of 16 bytes swizzled, so that 16 lanes that read one group of 16 rows meet every bank once.
template <int WT>
struct LinearTile {
  static constexpr int T = 2 * WT, BK = 128, CPR = BK / 16, LOADS = 2 * T * CPR / 256, KS = BK / 32, F = WT / 32;
  static constexpr int STAGE = 2 * T * BK;  // bytes of both operands
  static constexpr int STAGES = WT == 32 ? 4 : 2;
  static __device__ inline int swizzle(int row) { return (row / (256 / BK)) & (CPR - 1); }
  static __device__ inline int at(int row, int chunk) { return row * BK + 16 * (chunk ^ swizzle(row)); }
};

// 8192 x 4096 x 8192 bf16: 259 us, 2.1e15 operations a second, of which the loop takes 200 (2.8e15) and the ends of the
// tiles, each a round of the compute units with its 8-bit rows' first loads and 16-bit stores, 60; the library's
// product of the same sizes without scales runs at 2.2e15. Steps of 64 codes took 290.
//
// DIRECT: rows at multiples of 16 bytes go from memory into LDS without registers, up to three steps
// ahead; others by registers, two ahead.
template <class T, int WT, bool DIRECT>
__global__ void __launch_bounds__(256) linear_q8_kernel(LinearArgs a, int across, int tiles) {
  using L = LinearTile<WT>;
  constexpr int kPitch = WT * sizeof(T) + 16, kRowsAt = sizeof(T) == 4 && L::F > 1 ? L::F / 2 : L::F;
  constexpr int kOut = 4 * 32 * kRowsAt * kPitch + 2 * L::T * sizeof(float), kIn = L::STAGE * (DIRECT ? L::STAGES : 2);
  __shared__ __attribute__((aligned(16))) char lds[kOut > kIn ? kOut : kIn];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int v = xcd_virtual(blockIdx.x, gridDim.x, tiles);
  if (v < 0) return;
  // bands of 8 tiles of rows, walked channel tile by channel tile: the tiles that run at a time on an XCD
  // share rows and weights in its L2
  const int down = tiles / across, band = v / (8 * across), in = v - band * 8 * across, high = min(8, down - 8 * band);
  const int o0 = in / high * L::T, r0 = (band * 8 + in % high) * L::T;

  // rows past the last are that one again: what they give is not stored
  const KG int8_t* const wb = gp(a.w) + o0 * a.ldw;
  const KG int8_t* const qb = gp(static_cast<const int8_t*>(a.q)) + r0 * a.ldq;
  const int slot = tid % L::CPR, chunk = slot ^ L::swizzle(tid / L::CPR);  // the same for all loads of a thread
  unsigned off[L::LOADS];
#pragma unroll
  for (int i = 0; i < L::LOADS; ++i) {
    const int row = (tid + 256 * i) / L::CPR;
    const bool is_w = 2 * i < L::LOADS;
    const int r = is_w ? min(row, a.c_out - 1 - o0) : min(row - L::T, a.rows - 1 - r0);
    off[i] = static_cast<unsigned>(r) * static_cast<unsigned>(is_w ? a.ldw : a.ldq) + 16 * chunk;
  }
  v4i st[L::LOADS];
  auto load = [&](int k0) {
#pragma unroll
    for (int i = 0; i < L::LOADS; ++i)
      st[i] = __builtin_bit_cast(v4i, load_pack<false, int8_t>((2 * i < L::LOADS ? wb : qb) + k0 + off[i]));
  };
  auto load_end = [&](int k0) {
#pragma unroll
    for (int i = 0; i < L::LOADS; ++i)
      st[i] = load_codes((2 * i < L::LOADS ? wb : qb) + (off[i] - 16 * chunk), k0 + 16 * chunk, a.c_in);
  };
  auto load_any = [&](int k0) {
    if (k0 + L::BK <= a.c_in) load(k0);
    else load_end(k0);
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < L::LOADS; ++i) *reinterpret_cast<v4i*>(lds + buf * L::STAGE + 16 * (tid + 256 * i)) = st[i];
  };
  auto send = [&](int k0, int buf, int i) {  // memory to LDS: a wave's 64 groups of 16 bytes side by side
    __builtin_amdgcn_global_load_lds((const KG void*)((2 * i < L::LOADS ? wb : qb) + k0 + off[i]),
                                     (__attribute__((address_space(3))) void*)(lds + buf * L::STAGE + 16 * (64 * wave + 256 * i)),
                                     16, 0, 0);
  };
  const int wo = (wave >> 1) * WT, wr = L::T + (wave & 1) * WT;
  auto frag = [&](int buf, int row, int ks) {
    return *reinterpret_cast<const v4i*>(lds + buf * L::STAGE + L::at(row + (lane & 31), 2 * ks + (lane >> 5)));
  };
  v16i acc[L::F][L::F];
#pragma unroll
  for (int i = 0; i < L::F; ++i)
#pragma unroll
    for (int j = 0; j < L::F; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  // what the end needs, on its way while the products are formed
  const int channel = min(o0 + tid % L::T, a.c_out - 1);
  const float channel_scale = gp(a.w_scale)[channel];
  const float channel_bias = a.bias ? static_cast<float>(gp(static_cast<const T*>(a.bias))[channel]) : 0.f;
  float row_scale[L::F];
#pragma unroll
  for (int j = 0; j < L::F; ++j) row_scale[j] = gp(a.scale)[min(r0 + wr - L::T + 32 * j + (lane & 31), a.rows - 1)];

  const int steps = (a.c_in + L::BK - 1) / L::BK;
  if (steps) {
    v4i fa[2][L::F], fb[2][L::F];
    auto read1 = [&](int buf, int ks, int set, int n) {  // operand n of 2 F
      if (n & 1) fb[set][n / 2] = frag(buf, wr + 32 * (n / 2), ks);
      else fa[set][n / 2] = frag(buf, wo + 32 * (n / 2), ks);
    };
    auto read = [&](int buf, int ks, int set) {
#pragma unroll
      for (int n = 0; n < 2 * L::F; ++n) read1(buf, ks, set, n);
    };
    // behind(n) is issued behind product n, while the matrix unit works on that
    auto mma = [&](int set, auto&& behind) {
#pragma unroll
      for (int n = 0; n < L::F * L::F; ++n) {
        const int i = n / L::F, j = n % L::F;
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[set][i], fb[set][j], acc[i][j], 0, 0, 0);
        behind(n);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // The operands of the next 32 codes are read while the matrix unit works on these. The barrier stands
    // before a step's last products, when its operands have all been read and the next step's have
    // arrived: those are read behind them, and the step's buffer is filled again.
    if constexpr (DIRECT) {
      auto send_any = [&](int c) {
        if ((c + 1) * L::BK <= a.c_in) {
#pragma unroll
          for (int i = 0; i < L::LOADS; ++i) send(c * L::BK, c % L::STAGES, i);
        } else if (c < steps) {
          load_end(c * L::BK);
          store(c % L::STAGES);
        }
      };
      for (int c = 0; c < L::STAGES - 1; ++c) send_any(c);
      if (steps < L::STAGES) arrive<0>();
      else arrive<(L::STAGES - 2) * L::LOADS>();
      send_any(L::STAGES - 1);
      read(0, 0, 0);
      constexpr int N = L::F * L::F, R = 2 * L::F, per = (R + N - 1) / N;  // products and operands of 32 codes
      constexpr int each = (L::LOADS + N - 1) / N, from = N - (L::LOADS + each - 1) / each;
      // the operands behind the first products, what fetch sends behind the last
      auto step = [&](int c, auto ahead, auto&& fetch) {
#pragma unroll
        for (int ks = 0; ks < L::KS; ++ks) {
          const bool last = ks + 1 == L::KS;
          // loads that may still be on their way when step c + 1's have arrived
          if (last) arrive<decltype(ahead)::value>();
          mma(ks & 1, [&](int n) {
#pragma unroll
            for (int k = n * per; k < n * per + per && k < R; ++k)
              last ? read1((c + 1) % L::STAGES, 0, 0, k) : read1(c % L::STAGES, ks + 1, (ks + 1) & 1, k);
#pragma unroll
            for (int i = (n - from) * each; i < (n - from + 1) * each && i < L::LOADS; ++i)
              if (last && i >= 0) fetch(i);
          });
        }
      };
      int c = 0;
      for (; (c + L::STAGES + 1) * L::BK <= a.c_in; ++c)
        step(c, std::integral_constant<int, (L::STAGES - 2) * L::LOADS>{},
             [&](int i) { send((c + L::STAGES) * L::BK, c % L::STAGES, i); });
      // the last steps: all that was sent is waited for
      for (; c < steps; ++c)
        step(c, std::integral_constant<int, 0>{}, [&](int i) {
          if (i == 0) send_any(c + L::STAGES);
        });
    } else {
      load_any(0);
      store(0);
      if (steps > 1) load_any(L::BK);
      __syncthreads();
      read(0, 0, 0);
      auto step = [&](int cur, bool next, auto&& fetch) {
        if (next) store(cur ^ 1);
        fetch();
#pragma unroll
        for (int ks = 0; ks < L::KS; ++ks) {
          if (ks + 1 < L::KS) {
            read(cur, ks + 1, (ks + 1) & 1);
          } else {
            __syncthreads();
            if (next) read(cur ^ 1, 0, 0);
          }
          mma(ks & 1, [](int) {});
        }
      };
      int c = 0;
      for (; (c + 3) * L::BK <= a.c_in; ++c) step(c & 1, true, [&] { load((c + 2) * L::BK); });
      for (; c < steps; ++c)
        step(c & 1, c + 1 < steps, [&] {
          if (c + 2 < steps) load_any((c + 2) * L::BK);
        });
    }
    __syncthreads();
  }

  // The channels' scales and biases go through LDS; then each wave brings its rows into LDS lines of their
  // channels (fp32: half of them at a time) and stores them 16 bytes a lane.
  float* const sv = reinterpret_cast<float*>(lds);
  float* const sb = sv + L::T;
  char* const mine = lds + 2 * L::T * sizeof(float) + wave * 32 * kRowsAt * kPitch;
  if (tid < L::T) sv[tid] = channel_scale, sb[tid] = channel_bias;
  __syncthreads();
  constexpr int EV = 16 / sizeof(T), LANES = WT / EV;
  const int wo0 = o0 + wo, wr0 = r0 + wr - L::T;
#pragma unroll
  for (int j0 = 0; j0 < L::F; j0 += kRowsAt) {
#pragma unroll
    for (int i = 0; i < L::F; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = 32 * i + 8 * g + 4 * (lane >> 5);
        const v4f v = *reinterpret_cast<const v4f*>(sv + wo + c), b = *reinterpret_cast<const v4f*>(sb + wo + c);
#pragma unroll
        for (int j = j0; j < j0 + kRowsAt; ++j) {
          typedef T vec4 __attribute__((ext_vector_type(4)));
          vec4 out;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            out[e] = static_cast<T>(entry(acc[i][j][4 * g + e], row_scale[j], v[e], b[e]));
          *reinterpret_cast<vec4*>(mine + (32 * (j - j0) + (lane & 31)) * kPitch + c * sizeof(T)) = out;
        }
      }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int n = 0; n < kRowsAt * 32 * LANES / 64; ++n) {
      const int u = n * 64 + lane, row = u / LANES, c = u % LANES * EV;
      const v4i raw = *reinterpret_cast<const v4i*>(mine + row * kPitch + c * sizeof(T));
      const auto out = __builtin_bit_cast(typename Pack<T>::vec, raw);
      const int64_t rr = wr0 + 32 * j0 + row;
      const int o = wo0 + c;
      if (rr < a.rows) {
        KG T* p = gp(static_cast<T*>(a.y)) + rr * a.ldy + o;
        if (o + EV <= a.c_out) {
          store_pack<false, T>(p, out);
        } else {
#pragma unroll
          for (int k = 0; k < EV; ++k)
            if (o + k < a.c_out) p[k] = out[k];
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Few rows: the weights' way from memory is what it takes. A block has 16 channels and all rows, 16 NB of them
// or fewer; its WAVES waves share the codes, 64 at a time, operands straight from memory into the
// matrix unit's layout (16 bytes a lane), DEPTH of them on their way; the waves' sums meet in LDS.
//
// FUSED: the block first quantises the rows itself, its first weights on their way meanwhile, which saves a
// launch; block 0 writes the checkpoint. For up to kFusedCodes codes, which each block has to form.
constexpr int kFewRows = 32, kFusedCodes = 16384, kFewChannels = 1 << 25;  // 1024 threads for 16 of them

template <class T, int NB, int WAVES, bool FUSED>
__global__ void __launch_bounds__(64 * WAVES) linear_few_kernel(LinearArgs a, const T* __restrict__ x, int64_t ldx,
                                                                const uint8_t* __restrict__ mask) {
  constexpr int NT = 64 * WAVES, DEPTH = 4, U = FUSED ? kFusedCodes / 8 / NT + 1 : 1;
  __shared__ __attribute__((aligned(16))) int sums[WAVES][NB][16][17];
  __shared__ __attribute__((aligned(16))) int8_t codes[FUSED ? kFusedCodes + 64 * 16 : 16];
  __shared__ float scales[16 * NB];
  __shared__ unsigned tops[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int o0 = blockIdx.x * 16, chunks = (a.c_in + 63) / 64;
  const KG int8_t* const w = gp(a.w) + int64_t(min(o0 + (lane & 15), a.c_out - 1)) * a.ldw;
  const int k_lane = 16 * (lane >> 4), pitch = (a.c_in + 15) / 16 * 16 + 16;  // of the codes in LDS
  auto load = [&](const KG int8_t* row, int c) {  // past the end: zeros
    if (64 * c + 64 <= a.c_in) return __builtin_bit_cast(v4i, load_pack<false, int8_t>(row + 64 * c + k_lane));
    return load_codes(row, 64 * c + k_lane, a.c_in);
  };
  const KG int8_t* q[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) q[b] = gp(static_cast<const int8_t*>(a.q)) + int64_t(min(16 * b + (lane & 15), a.rows - 1)) * a.ldq;
  v4i wv[DEPTH], qv[DEPTH][NB];
  auto load_all = [&](int d, int c) {
    wv[d] = load(w, c);
    if constexpr (!FUSED)
#pragma unroll
      for (int b = 0; b < NB; ++b) qv[d][b] = load(q[b], c);
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load_all(d, wave + d * WAVES);
  if constexpr (FUSED) {
    const int groups = pitch / 8, all = a.rows * groups;  // of 8 codes, with what is behind a row's end
    Eight<T> v[U];
    if (tid < 16) tops[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = tid + u * NT, r = g / groups, c = 8 * (g - r * groups);
      const bool take = g < all && c < a.c_in && (!mask || gp(mask)[r]);
      v[u].load(gp(x) + (take ? r * ldx + c : 0), take ? a.c_in - c : 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = tid + u * NT;
      if (g < all) atomicMax(&tops[g / groups], v[u].top(0));  // of whole numbers: any order
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = tid + u * NT, r = g / groups, c = 8 * (g - r * groups);
      if (g >= all) continue;
      RowCode code = row_code<true>(tops[r]);
      if (mask && !gp(mask)[r]) code.s = 0.f;
      const v2u out = v[u].template coded<true>(code);
      *reinterpret_cast<v2u*>(codes + r * pitch + c) = out;
      if (c == 0) scales[r] = code.s;
      if (blockIdx.x == 0) {
        if (c < a.c_in) Eight<T>::put(gp(a.q) + r * a.ldq + c, a.c_in - c, out);
        if (c == 0) gp(a.scale)[r] = code.s;
      }
    }
    __syncthreads();
  } else {
    if (tid < 16 * NB) scales[tid] = gp(a.scale)[min(tid, a.rows - 1)];
  }
  const int8_t* const mine = codes + min(lane & 15, a.rows - 1) * pitch;
  v4i acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = v4i{0, 0, 0, 0};
  for (int c = wave; c < chunks; c += WAVES * DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int at = c + d * WAVES;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        v4i v;
        // past the end the weights are 0
        if constexpr (FUSED) v = *reinterpret_cast<const v4i*>(mine + min(64 * at + k_lane, pitch - 16));
        else v = qv[d][b];
        acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[d], v, acc[b], 0, 0, 0);
      }
      load_all(d, at + DEPTH * WAVES);
    }
  }
  // a lane has row lane % 16 and channels 4 (lane / 16) ..
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[wave][b][lane & 15][4 * (lane >> 4) + e] = acc[b][e];
  __syncthreads();
  for (int u = tid; u < 256 * NB; u += NT) {
    const int r = u >> 4, o = o0 + (u & 15);
    if (r >= a.rows || o >= a.c_out) continue;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) sum += sums[i][r >> 4][r & 15][u & 15];
    const float b = a.bias ? static_cast<float>(gp(static_cast<const T*>(a.bias))[o]) : 0.f;
    gp(static_cast<T*>(a.y))[r * a.ldy + o] = static_cast<T>(entry(sum, scales[r], gp(a.w_scale)[o], b));
  }
}

// ---- host -------------------------------------------------------------------

static kfac_status sizes_ok(int32_t rows, int32_t cols, const char* what) {
  if (rows < 0 || cols < 0) return fail(KFAC_ERR_INVALID, "negative %s", what);
  return KFAC_OK;
}

template <class T, bool POW2>
static kfac_status launch_quantize(int32_t rows, int32_t cols, const void* x, int64_t ld, const uint8_t* mask,
                                   int8_t* q, int64_t ldq, float* scale, hipStream_t s) {
  auto go = [&](auto tpr, auto u) {
    constexpr int TPR = decltype(tpr)::value, PER = 256 / TPR;
    for (int64_t r = 0; r < rows; r += kMostBlocks * PER) {
      const int n = static_cast<int>(std::min<int64_t>(rows - r, kMostBlocks * PER));
      KFAC_LAUNCH(K_QUANTIZE, (quantize_rows_kernel<T, POW2, TPR, decltype(u)::value>), dim3((n + PER - 1) / PER), dim3(256),
                  0, s, n, cols, static_cast<const T*>(x) + r * ld, ld, mask ? mask + r : nullptr, q + r * ldq, ldq, scale + r);
      KFAC_CHECK_LAUNCH("quantize_rows_kernel");
    }
    return KFAC_OK;
  };
  constexpr std::integral_constant<int, 64> wave;
  constexpr std::integral_constant<int, 256> block;
  if (cols <= 512) return go(wave, std::integral_constant<int, 1>{});
  // a wave a row, if there are many: 8192 x 2048 bf16 11.0 us (a block a row: 11.7), 1024 x 2048 6.9 (6.5); but
  // 8192 x 4096, with 64 elements a lane, 25.8 (22.6: 4.5 TB/s)
  if (rows > 1024 && cols <= 2048) return go(wave, std::integral_constant<int, 4>{});
  if (cols <= 2048) return go(block, std::integral_constant<int, 1>{});
  if (cols <= 4096) return go(block, std::integral_constant<int, 2>{});
  if (cols <= 8192) return go(block, std::integral_constant<int, 4>{});
  if (cols <= 16384) return go(block, std::integral_constant<int, 8>{});
  return go(block, std::integral_constant<int, 0>{});
}

static kfac_status quantize_checks(int32_t rows, int32_t cols, kfac_dtype dtype, const RowsOf& x, const uint8_t* mask,
                                   const RowsOf& q, const RowsOf& scale) {
  kfac_status st;
  if (!row_dtype(dtype)) return fail(KFAC_ERR_UNSUPPORTED, "dtype %d", dtype);
  if ((st = sizes_ok(rows, cols, "rows or cols"))) return st;
  for (const RowsOf* r : {&x, &q, &scale})
    if ((st = check_rows(*r))) return st;
  const RowsOf m = {mask, mask ? rows : 0, 1, 1, 1, "mask"};
  return check_apart({&q, &scale, &x, &m}, 2);
}

extern "C" kfac_status kfac_quantize_rows(int32_t rows, int32_t cols, kfac_dtype dtype, const void* x, int64_t ld_x,
                                          const uint8_t* mask, int32_t pow2, int8_t* q, int64_t ld_q, float* scale,
                                          void* stream) {
  kfac_status st = quantize_checks(rows, cols, dtype, {x, rows, cols, ld_x, dtype_bytes(dtype), "x"}, mask,
                                   {q, rows, cols, ld_q, 1, "q"}, {scale, rows, 1, 1, 4, "scale"});
  if (st) return st;
  if (pow2 != 0 && pow2 != 1) return fail(KFAC_ERR_INVALID, "pow2 must be 0 or 1");
  if ((st = check_device())) return st;
  if (rows == 0) return KFAC_OK;
  return with_row_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return pow2 ? launch_quantize<T, true>(rows, cols, x, ld_x, mask, q, ld_q, scale, s)
                : launch_quantize<T, false>(rows, cols, x, ld_x, mask, q, ld_q, scale, s);
  });
}

extern "C" kfac_status kfac_dequantize_rows(int32_t rows, int32_t cols, const int8_t* q, int64_t ld_q,
                                            const float* scale, kfac_dtype dtype, void* x, int64_t ld_x, void* stream) {
  if (!row_dtype(dtype)) return fail(KFAC_ERR_UNSUPPORTED, "dtype %d", dtype);
  kfac_status st = sizes_ok(rows, cols, "rows or cols");
  if (st) return st;
  const RowsOf xs = {x, rows, cols, ld_x, dtype_bytes(dtype), "x"}, qs = {q, rows, cols, ld_q, 1, "q"},
               ss = {scale, cols > 0 ? rows : 0, 1, 1, 4, "scale"};
  for (const RowsOf* r : {&xs, &qs, &ss})
    if ((st = check_rows(*r))) return st;
  if ((st = check_apart({&xs, &qs, &ss}, 1))) return st;
  if ((st = check_device())) return st;
  if (xs.empty()) return KFAC_OK;
  return with_row_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    const unsigned per_row = static_cast<unsigned>((int64_t(cols) + 7) / 8);
    const int64_t most = kMostBlocks * 256 / per_row;  // rows a launch
    for (int64_t r = 0; r < rows; r += most) {
      const int64_t n = std::min(rows - r, most);
      const unsigned groups = static_cast<unsigned>(n * per_row);
      KFAC_LAUNCH(K_DEQUANTIZE, dequantize_rows_kernel<T>, dim3((groups + 255) / 256), dim3(256), 0,
                  static_cast<hipStream_t>(stream), cols, per_row, groups, q + r * ld_q, ld_q, scale + r,
                  static_cast<T*>(x) + r * ld_x, ld_x);
      KFAC_CHECK_LAUNCH("dequantize_rows_kernel");
    }
    return KFAC_OK;
  });
}

// 128^2 * (2^17 - 1) < 2^31: no sum leaves an int32, whatever the codes.
constexpr int32_t kMaxTerms = (1 << 17) - 1;
constexpr int64_t kMaxPitch = 1 << 23;  // 256 rows of a tile within 32-bit offsets

static kfac_status linear_sizes(int32_t rows, int32_t c_in, int32_t c_out) {
  if (rows < 0 || c_in < 0 || c_out < 0) return fail(KFAC_ERR_INVALID, "negative rows, c_in or c_out");
  if (c_in > kMaxTerms) return fail(KFAC_ERR_UNSUPPORTED, "c_in %d: a sum of more than %d products", c_in, kMaxTerms);
  // as many take tiles of 256
  if ((int64_t(rows) + 255) / 256 * ((int64_t(c_out) + 255) / 256) > kMostBlocks)
    return fail(KFAC_ERR_UNSUPPORTED, "%d x %d: more than 2^24 - 8 tiles of 256 x 256", rows, c_out);
  return KFAC_OK;
}

template <class T, int WT, bool DIRECT>
static kfac_status launch_linear(const LinearArgs& a, hipStream_t s) {
  using L = LinearTile<WT>;
  const int64_t across = (int64_t(a.c_out) + L::T - 1) / L::T, tiles = across * ((int64_t(a.rows) + L::T - 1) / L::T);
  KFAC_LAUNCH(K_LINEAR_Q8, (linear_q8_kernel<T, WT, DIRECT>), dim3(xcd_grid(tiles)), dim3(256), 0, s, a,
              static_cast<int>(across), static_cast<int>(tiles));
  KFAC_CHECK_LAUNCH("linear_q8_kernel");
  return KFAC_OK;
}

template <class T>
static kfac_status launch_few(const LinearArgs& a, const T* x, int64_t ldx, const uint8_t* mask, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>((int64_t(a.c_out) + 15) / 16);
  auto go = [&](auto nb, auto fused) {
    constexpr int W = 16;  // 4 or 8 waves: 10.7 us for one row of 4096 x 4096 instead of 10.2, 17.0 and 18.1 for 8192 x 8192 instead of 14.9
    KFAC_LAUNCH(K_LINEAR_Q8, (linear_few_kernel<T, decltype(nb)::value, W, decltype(fused)::value>), dim3(blocks),
                dim3(64 * W), 0, s, a, x, ldx, mask);
    KFAC_CHECK_LAUNCH("linear_few_kernel");
    return KFAC_OK;
  };
  if (x) return go(std::integral_constant<int, 1>{}, std::true_type{});
  if (a.rows <= 16) return go(std::integral_constant<int, 1>{}, std::false_type{});
  return go(std::integral_constant<int, 2>{}, std::false_type{});
}

static size_t linear_need(int32_t, int32_t, int32_t) { return 0; }

extern "C" kfac_status kfac_linear_q8_workspace(int32_t rows, int32_t c_in, int32_t c_out, size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  kfac_status st = linear_sizes(rows, c_in, c_out);
  if (st) return st;
  *bytes = linear_need(rows, c_in, c_out);
  return KFAC_OK;
}

extern "C" kfac_status kfac_linear_q8(int32_t rows, int32_t c_in, int32_t c_out, kfac_dtype dtype, const void* x,
                                      int64_t ld_x, const uint8_t* mask, int8_t* q, int64_t ld_q, float* scale,
                                      const int8_t* w, int64_t ld_w, const float* w_scale, const void* bias, void* y,
                                      int64_t ld_y, void* workspace, size_t ws_bytes, void* stream) {
  if (!row_dtype(dtype)) return fail(KFAC_ERR_UNSUPPORTED, "dtype %d", dtype);
  kfac_status st = linear_sizes(rows, c_in, c_out);
  if (st) return st;
  const int size = dtype_bytes(dtype);
  const RowsOf xs = {x, x ? rows : 0, c_in, ld_x, size, "x"}, qs = {q, rows, c_in, ld_q, 1, "q"},
               ss = {scale, rows, 1, 1, 4, "scale"}, ws = {w, c_out, c_in, ld_w, 1, "w"},
               vs = {w_scale, c_out, 1, 1, 4, "w_scale"}, bs = {bias, bias ? c_out : 0, 1, 1, size, "bias"},
               ys = {y, rows, c_out, ld_y, size, "y"}, ms = {mask, mask && x ? rows : 0, 1, 1, 1, "mask"};
  for (const RowsOf* r : {&xs, &qs, &ss, &ws, &vs, &bs, &ys})
    if ((st = check_rows(*r))) return st;
  if (mask && !x) return fail(KFAC_ERR_INVALID, "mask without x");
  for (const RowsOf* r : {&qs, &ws})
    if (r->rows > 1 && r->ld >= kMaxPitch) return fail(KFAC_ERR_UNSUPPORTED, "%s: rows of 2^23 bytes and more", r->name);
  const RowsOf scr = scratch(workspace, linear_need(rows, c_in, c_out));
  if (x) st = check_apart({&ys, &scr, &qs, &ss, &xs, &ws, &vs, &bs, &ms}, 4);
  else st = check_apart({&ys, &scr, &qs, &ss, &ws, &vs, &bs}, 2);
  if (st) return st;
  if ((st = check_device())) return st;
  if ((st = check_workspace(workspace, ws_bytes, scr.width))) return st;
  if (rows == 0) return KFAC_OK;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return with_row_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    const LinearArgs args = {rows, c_in, c_out, q, w, scale, w_scale, bias, y, ld_q, ld_w, ld_y};
    // Few rows, kernels by themselves, codes given, in us, in tiles in brackets: 1 x 4096 x 4096 bf16 5.9 (11.4), 16 x 1024 x
    // 4096 4.5 (5.0), 16 x 512 x 8192 4.5 (3.9). More than 16 rows: 32 x 4096 x 4096 9.1 (11.6), 17 x 2048 x 4096 6.3 (7.6), but
    // 17 x 1024 x 4096 5.4 (5.0), and with more channels than the card takes blocks for at a time, 17 x 1024 x 8192 9.4 (5.6),
    // 32 x 8192 x 8192 28.0 (21.0). Fused with the quantising, the whole call: 1 x 4096 x 4096 8.5, else 6.4 + 7.5, 16 x 1024 x
    // 4096 9.8, else 7.0 + 6.5: a launch less, 3 us a call
    const bool few = c_out > 0 && (rows <= 16 ? c_out <= kFewChannels : rows <= kFewRows && c_in > 1024 && c_out <= 4096);
    const bool fused = few && x && rows <= 16 && int64_t(rows) * c_in <= kFusedCodes;
    if (x && !fused) {
      kfac_status e = launch_quantize<T, true>(rows, c_in, x, ld_x, mask, q, ld_q, scale, s);
      if (e) return e;
    }
    if (c_out == 0) return KFAC_OK;
    if (few) return launch_few<T>(args, fused ? static_cast<const T*>(x) : nullptr, ld_x, mask, s);
    const int64_t big = (int64_t(c_out) + 255) / 256 * ((int64_t(rows) + 255) / 256);
    const int64_t mid = (int64_t(c_out) + 127) / 128 * ((int64_t(rows) + 127) / 128);
    const bool direct = !((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(w) | uintptr_t(ld_q) | uintptr_t(ld_w)) & 15);
    auto go = [&](auto wt) {
      return direct ? launch_linear<T, decltype(wt)::value, true>(args, s) : launch_linear<T, decltype(wt)::value, false>(args, s);
    };
    // tiles of 256, 128 or 64, so that there is a block for most compute units: 4096 x 4096 x 4096 bf16 (256 tiles of
    // 256) 63.5 us (tiles of 128: 70.7), 1024 x 4096 x 8192 (128) 52.5 (38.6); 1024 x 4096 x 3200 (200 of 128) 28.1
    // (tiles of 64: 30.9), 1024 x 4096 x 2048 (128) 25.9 (18.9)
    if (big >= 192) return go(std::integral_constant<int, 128>{});
    if (mid >= 160) return go(std::integral_constant<int, 64>{});
    return go(std::integral_constant<int, 32>{});
  });
}

}  // namespace kfac
