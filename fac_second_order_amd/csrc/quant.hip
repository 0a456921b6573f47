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

struct RowCode {
  float s, inv;
  int most;  // 127, or 63 where 64 s would be infinite
};

template <bool POW2>
__device__ inline RowCode row_code(unsigned amax) {
  RowCode c;
  c.s = row_scale<POW2>(amax);
  const bool bad = amax >= 0x7f800000u;
  c.inv = bad ? 0.f : 1.f / c.s;
  c.most = POW2 && !bad && c.s >= 5.3169119831396635e36f ? 63 : 127;  // 2^122
  return c;
}

// q of one element, as an integer. A row with an infinity or a NaN has none: all zeros.
template <bool POW2>
__device__ inline int code_of(float x, const RowCode& c) {
  if (c.inv == 0.f) return 0;
  float t = fmaf(x, c.inv, kMagic) - kMagic;
  if (!POW2) {
    // x - t s is exact (below a step, and a multiple of the smaller of both last places): put
    // right what the rounded reciprocal decided next to a half, ties to the even side
    const float d = fmaf(-t, c.s, x), h = 0.5f * c.s;
    const float a = fabsf(d);
    if (a > h || (a == h && (static_cast<int>(t) & 1))) t += copysignf(1.f, d);
  }
  const int q = static_cast<int>(t);
  return max(-c.most, min(c.most, q));
}

// A block per row: the largest magnitude, then the codes, the row's second reading from the caches.
template <class T, bool POW2>
__global__ void __launch_bounds__(256) quantize_rows_kernel(int cols, const T* __restrict__ x, int64_t ld,
                                                            const uint8_t* __restrict__ mask, int8_t* __restrict__ q,
                                                            int64_t ldq, float* __restrict__ scale) {
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const KG T* xr = gp(x) + row * ld;
  KG int8_t* qr = gp(q) + row * ldq;
  if (mask && !gp(mask)[row]) {
    for (int c = tid; c < cols; c += 256) qr[c] = 0;
    if (tid == 0) gp(scale)[row] = 0.f;
    return;
  }
  unsigned top = 0;
  for (int c = tid; c < cols; c += 256) top = max(top, __float_as_uint(static_cast<float>(xr[c])) & 0x7fffffffu);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = max(top, __shfl_xor(top, o));
  __shared__ unsigned part[4];
  if ((tid & 63) == 0) part[tid >> 6] = top;
  __syncthreads();
  const RowCode code = row_code<POW2>(max(max(part[0], part[1]), max(part[2], part[3])));
  for (int c = tid; c < cols; c += 256) qr[c] = static_cast<int8_t>(code_of<POW2>(static_cast<float>(xr[c]), code));
  if (tid == 0) gp(scale)[row] = code.s;
}

template <class T>
__device__ inline T held(float v) {
  constexpr float most = std::is_same_v<T, _Float16> ? 65504.f
                         : std::is_same_v<T, float>  ? 3.4028234663852886e38f
                                                     : 3.3895313892515355e38f;
  if (fabsf(v) > most) v = copysignf(most, v);
  return static_cast<T>(v);
}

template <class T>
__global__ void __launch_bounds__(256) dequantize_rows_kernel(int cols, const int8_t* __restrict__ q, int64_t ldq,
                                                              const float* __restrict__ scale, T* __restrict__ x,
                                                              int64_t ld) {
  const int64_t row = blockIdx.x;
  const float s = gp(scale)[row];
  for (int c = threadIdx.x; c < cols; c += 256)
    gp(x)[row * ld + c] = held<T>(static_cast<float>(gp(q)[row * ldq + c]) * s);
}

// y = fp32(sum of q w) s v + b, a tile of 64 x 64 a block: 4 waves of 32 x 32, 64 elements of the sum a step.
template <class T>
__global__ void __launch_bounds__(256) linear_q8_kernel(int rows, int c_in, int c_out, const int8_t* __restrict__ q,
                                                        int64_t ldq, const float* __restrict__ scale,
                                                        const int8_t* __restrict__ w, int64_t ldw,
                                                        const float* __restrict__ wscale, const T* __restrict__ bias,
                                                        T* __restrict__ y, int64_t ldy) {
  __shared__ __attribute__((aligned(16))) int8_t lds[2][64][80];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const unsigned across = (c_out + 63) / 64;
  const int64_t r0 = int64_t(blockIdx.x / across) * 64, o0 = int64_t(blockIdx.x % across) * 64;
  v16i acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0;
  for (int k0 = 0; k0 < c_in; k0 += 64) {
    for (int i = tid; i < 64 * 64; i += 256) {
      const int r = i >> 6, k = i & 63;
      lds[0][r][k] = r0 + r < rows && k0 + k < c_in ? gp(q)[(r0 + r) * ldq + k0 + k] : 0;
      lds[1][r][k] = o0 + r < c_out && k0 + k < c_in ? gp(w)[(o0 + r) * ldw + k0 + k] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = h * 32 + (lane >> 5) * 16;
      const v4i a = *reinterpret_cast<const v4i*>(&lds[0][(wave >> 1) * 32 + (lane & 31)][k]);
      const v4i b = *reinterpret_cast<const v4i*>(&lds[1][(wave & 1) * 32 + (lane & 31)][k]);
      acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, acc, 0, 0, 0);
    }
    __syncthreads();
  }
  const int64_t o = o0 + (wave & 1) * 32 + (lane & 31);
  if (o >= c_out) return;
  const float v = gp(wscale)[o], add = bias ? static_cast<float>(gp(bias)[o]) : 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int64_t r = r0 + (wave >> 1) * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
    if (r < rows) gp(y)[r * ldy + o] = static_cast<T>(static_cast<float>(acc[e]) * gp(scale)[r] * v + add);
  }
}

// ---- host -------------------------------------------------------------------

static kfac_status sizes_ok(int32_t rows, int32_t cols, const char* what) {
  if (rows < 0 || cols < 0) return fail(KFAC_ERR_INVALID, "negative %s", what);
  return KFAC_OK;
}

template <class T>
static kfac_status launch_quantize(int32_t rows, int32_t cols, const void* x, int64_t ld, const uint8_t* mask, bool pow2,
                                   int8_t* q, int64_t ldq, float* scale, hipStream_t s) {
  if (pow2) {
    KFAC_LAUNCH(K_QUANTIZE, (quantize_rows_kernel<T, true>), dim3(rows), dim3(256), 0, s, cols,
                static_cast<const T*>(x), ld, mask, q, ldq, scale);
  } else {
    KFAC_LAUNCH(K_QUANTIZE, (quantize_rows_kernel<T, false>), dim3(rows), dim3(256), 0, s, cols,
                static_cast<const T*>(x), ld, mask, q, ldq, scale);
  }
  KFAC_CHECK_LAUNCH("quantize_rows_kernel");
  return KFAC_OK;
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
    return launch_quantize<decltype(tag)>(rows, cols, x, ld_x, mask, pow2 == 1, q, ld_q, scale,
                                          static_cast<hipStream_t>(stream));
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
    KFAC_LAUNCH(K_DEQUANTIZE, dequantize_rows_kernel<T>, dim3(rows), dim3(256), 0, static_cast<hipStream_t>(stream), cols,
                q, ld_q, scale, static_cast<T*>(x), ld_x);
    KFAC_CHECK_LAUNCH("dequantize_rows_kernel");
    return KFAC_OK;
  });
}

// 128^2 * (2^17 - 1) < 2^31: no sum leaves an int32, whatever the codes.
constexpr int32_t kMaxTerms = (1 << 17) - 1;

static kfac_status linear_sizes(int32_t rows, int32_t c_in, int32_t c_out) {
  if (rows < 0 || c_in < 0 || c_out < 0) return fail(KFAC_ERR_INVALID, "negative rows, c_in or c_out");
  if (c_in > kMaxTerms) return fail(KFAC_ERR_UNSUPPORTED, "c_in %d: a sum of more than %d products", c_in, kMaxTerms);
  return KFAC_OK;
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
    if (x) {
      kfac_status e = launch_quantize<T>(rows, c_in, x, ld_x, mask, true, q, ld_q, scale, s);
      if (e) return e;
    }
    if (c_out == 0) return KFAC_OK;
    const int64_t tiles = (int64_t(c_out) + 63) / 64 * ((int64_t(rows) + 63) / 64);
    if (tiles > INT32_MAX) return fail(KFAC_ERR_UNSUPPORTED, "too many tiles");
    KFAC_LAUNCH(K_LINEAR_Q8, linear_q8_kernel<T>, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, rows, c_in,
                c_out, q, ld_q, scale, w, ld_w, w_scale, static_cast<const T*>(bias), static_cast<T*>(y), ld_y);
    KFAC_CHECK_LAUNCH("linear_q8_kernel");
    return KFAC_OK;
  });
}

}  // namespace kfac
