// Norms and updates over many tensors: the global gradient norm, clipping by it, and
// the update whose length is bounded by its predicted KL divergence.
//
// A tensor is cut into units of UNIT elements; a call's units are numbered through all
// tensors. A first launch sums over them, each block leaving one fp64 partial sum (a
// square of any fp32 value fits, and a multiply-add costs what an fp32 one costs); a second
// turns the sum into the factor; a third goes over the units again, last ones first, as the
// caches still hold those. Which block adds what depends on the sizes alone: results are
// deterministic. HBM-bound: the gradients are read twice, the result is written once.
//
// Measured: 54 fp32 tensors of ResNet-50 (102 MB) clipped in 52.8 us: 20.4 for the sum (5.0 TB/s),
// 4.6 for the factor, 29.7 for the second pass (6.9 TB/s, its reads from the last-level cache). A
// 111-tensor decoder, 1.7 GB in bf16 to fp32: 1.13 ms, 6.2 TB/s over both passes. The bounded update
// of ResNet-50 (409 MB moved): 82.7 us. (A copy kernel's best here is 6.15 TB/s, with one group of
// 16 bytes a thread in address order; a library copy does 4.95.)
#include <algorithm>
#include <type_traits>

#include "row_ops.hpp"

namespace kfac {

// Elements of a unit, and of the part of one that a block of the second pass takes: two groups of 16
// bytes a thread. A thread with one group copies fastest (6.15 TB/s, with four 5.7), but then finds
// its tensor for half as much.
constexpr int UNIT = 4096, PART = 2048;
constexpr int MAX_BLOCKS = 1024;   // partial sums
constexpr int GT = 256;            // threads per block
constexpr int ONE_THREADS = 1024;  // of the block that does a small call alone

// What a call does with its sum: the norm alone, clipping by it, or the bounded update.
enum Work { NORM, CLIP, TRUST };

// A tensor of a call: what the norm takes, and what the others need beside.
struct NormDesc {
  const void* grad;  // or the diagonal Fisher
  int64_t info;      // numel, and above it the types
  static constexpr int kType = 48, kWide = 50, kDiagonal = 51;
  __host__ __device__ int64_t numel() const { return info & ((int64_t(1) << kType) - 1); }
  __host__ __device__ int type() const { return static_cast<int>(info >> kType) & 3; }
  __host__ __device__ bool wide() const { return info >> kWide & 1; }  // out is fp32
  __host__ __device__ bool diagonal() const { return info >> kDiagonal & 1; }
};
struct ClipDesc : NormDesc {
  void* out;  // clipped gradient, or the weights of the update
};
struct TrustDesc : ClipDesc {
  const float* precond;
};
template <int W>
using DescOf = std::conditional_t<W == NORM, NormDesc, std::conditional_t<W == CLIP, ClipDesc, TrustDesc>>;

// The tables of a call: in the workspace, or where they fit in the kernel's arguments
// themselves, which saves the launches that send them (4.6 us each).
template <class D>
struct SentTables {
  const D* desc;
  const int32_t* begin;  // first unit of each tensor
};
template <class D>
struct InlineTables {
  static constexpr int most = 3888 / (sizeof(D) + 4);  // 194, 138 or 108: all arguments stay below 4 KB
  D desc[most];
  int32_t begin[most];
};

// The tensor that unit c lies in, by 64 begins at a time, one a lane: two loads side by side for up to
// 128 tensors (with one behind the other the second pass over 111 tensors took 4% longer), else steps
// of 64, 4096 and so on down to 1. Every tensor here has units, so the begins increase.
template <class TB>
__device__ inline int find_tensor(const TB& tb, int count, int c) {
  const int lane = threadIdx.x & 63;
  int p = 0;
  if (count <= 128) {
    bool before[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) before[k] = 64 * k + lane < count && tb.begin[64 * k + lane] <= c;
#pragma unroll
    for (int k = 0; k < 2; ++k) p += __popcll(__ballot(before[k]));
    return __builtin_amdgcn_readfirstlane(p - 1);
  }
  int step = 64;
  while (step < (count + 63) / 64) step *= 64;
  for (; step > 0; step /= 64) {
    const int i = p + lane * step;
    p += (__popcll(__ballot(i < count && tb.begin[i] <= c)) - 1) * step;
  }
  return __builtin_amdgcn_readfirstlane(p);
}

// f(type tag) with the type of a code.
template <class F>
__device__ inline void with_type(int code, F f) {
  if (code == KFAC_F32) f(float{});
  else if (code == KFAC_BF16) f(__bf16{});
  else f(_Float16{});
}

// n <= SIZE elements over NT threads in groups of EV: load(i, u) for all groups of a thread first,
// so that they are in flight together (a store could alias what is loaded next), one(i) for the
// last n % EV elements, use(i, u) for the groups. The groups come last: what runs behind a store
// and needs its registers waits until the store is done.
template <int SIZE, int NT, int EV>
constexpr int kTrips = (SIZE + NT * EV - 1) / (NT * EV);
template <int SIZE, int NT, int EV, class L, class U, class O>
__device__ inline void over(int n, L load, U use, O one) {
  const int tid = threadIdx.x, full = n / EV * EV;
#pragma unroll
  for (int u = 0; u < kTrips<SIZE, NT, EV>; ++u)
    if ((u * NT + tid) * EV < full) load((u * NT + tid) * EV, u);
  if (full + tid < n) one(full + tid);
#pragma unroll
  for (int u = 0; u < kTrips<SIZE, NT, EV>; ++u)
    if ((u * NT + tid) * EV < full) use((u * NT + tid) * EV, u);
}

template <int NT, bool LAST>
__device__ inline void add_squares(const NormDesc& d, int64_t e0, int n, double& acc) {
  with_type(d.type(), [&](auto tag) {
    using T = decltype(tag);
    constexpr int EV = Pack<T>::n;
    using V = typename Pack<T>::vec;
    const KG T* g = gp(static_cast<const T*>(d.grad)) + e0;
    V v[kTrips<UNIT, NT, EV>];
    over<UNIT, NT, EV>(
        n, [&](int i, int u) { v[u] = load_pack<LAST, T>(g + i); },
        [&](int, int u) {
#pragma unroll
          for (int k = 0; k < EV; ++k) {
            const double x = static_cast<float>(v[u][k]);
            acc = fma(x, x, acc);
          }
        },
        [&](int i) {
          const double x = static_cast<float>(g[i]);
          acc = fma(x, x, acc);
        });
  });
}

// What the second pass multiplies by, in two factors: their product may be too small for a float, as
// of a norm near the largest one, while its products with the gradients are not.
struct Factor {
  float f, pre;  // pre is 1 or a power of two
};

// out = coef * grad, coef in fp32, the product rounded once to the type of out.
template <int SIZE, int NT>
__device__ inline void scale_part(const ClipDesc& d, int64_t e0, int n, Factor c) {
  const auto times = [c](float g) { return g * c.pre * c.f; };
  with_type(d.type(), [&](auto tag) {
    using T = decltype(tag);
    const KG T* g = gp(static_cast<const T*>(d.grad)) + e0;
    const auto scale = [&](auto otag) {
      using O = decltype(otag);
      constexpr int EV = Pack<O>::n;  // a store of 16 bytes a lane, side by side
      using V = typename Pack<T, EV>::vec;
      using W = typename Pack<O, EV>::vec;
      KG O* o = gp(static_cast<O*>(d.out)) + e0;
      V v[kTrips<SIZE, NT, EV>];
      over<SIZE, NT, EV>(
          n, [&](int i, int u) { v[u] = load_pack<true, T, EV>(g + i); },
          [&](int i, int u) {
            W w;
#pragma unroll
            for (int k = 0; k < EV; ++k) w[k] = static_cast<O>(times(static_cast<float>(v[u][k])));
            store_pack<true, O>(o + i, w);
          },
          [&](int i) { o[i] = static_cast<O>(times(static_cast<float>(g[i]))); });
    };
    if (d.wide()) scale(float{});
    else scale(T{});
  });
}

// P * g, the preconditioned gradient against the gradient it came from.
template <int NT, bool LAST>
__device__ inline void add_products(const TrustDesc& d, int64_t e0, int n, float shift, double& acc) {
  const bool diagonal = d.diagonal();
  with_type(d.type(), [&](auto tag) {
    using T = decltype(tag);
    using V = Pack<float, 4>::vec;
    using W = typename Pack<T, 4>::vec;
    const KG float* p = gp(d.precond) + e0;
    const KG T* g = gp(static_cast<const T*>(d.grad)) + e0;
    V v[kTrips<UNIT, NT, 4>];
    W w[kTrips<UNIT, NT, 4>];
    const auto add = [&](float x, float y) {
      const double a = x, b = y;
      acc = fma(a, diagonal ? a * (b + shift) : b, acc);
    };
    over<UNIT, NT, 4>(
        n,
        [&](int i, int u) {
          v[u] = load_pack<LAST, float>(p + i);
          w[u] = load_pack<true, T, 4>(g + i);
        },
        [&](int, int u) {
#pragma unroll
          for (int k = 0; k < 4; ++k) add(v[u][k], static_cast<float>(w[u][k]));
        },
        [&](int i) { add(p[i], static_cast<float>(g[i])); });
  });
}

// w -= step * P.
template <int SIZE, int NT>
__device__ inline void apply_part(const TrustDesc& d, int64_t e0, int n, float step) {
  using V = Pack<float, 4>::vec;
  const KG float* p = gp(d.precond) + e0;
  KG float* w = gp(static_cast<float*>(d.out)) + e0;
  V v[kTrips<SIZE, NT, 4>], x[kTrips<SIZE, NT, 4>];
  over<SIZE, NT, 4>(
      n,
      [&](int i, int u) {
        v[u] = load_pack<true, float>(p + i);
        x[u] = load_pack<true, float>(w + i);
      },
      [&](int i, int u) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[u][k] = fmaf(-step, v[u][k], x[u][k]);
        store_pack<true, float>(w + i, x[u]);
      },
      [&](int i) { w[i] = fmaf(-step, p[i], w[i]); });
}

struct WorkArgs {
  float* result;  // norm; or step and q
  float a, b;     // max_norm; or lr and delta
  float shift;
};

// The factor of the second pass from the sum; `shown` writes the results.
template <int W>
__device__ inline Factor factor(double sum, const WorkArgs& k, bool shown) {
  if constexpr (W == TRUST) {
    const float q = static_cast<float>(sum);
    float step = 0.f;  // a q that is no finite float: no update, and q shows why
    if (q - q == 0) step = fmin(static_cast<double>(k.a), sqrt(2.0 * k.b / fabs(sum)));
    if (shown) {
      gp(k.result)[0] = step;
      gp(k.result)[1] = q;
    }
    return {step, 1.f};
  } else {
    const double root = sqrt(sum);
    const float norm = static_cast<float>(root);
    if (shown) gp(k.result)[0] = norm;
    // a norm that is no finite float: the gradients as they are
    if (W != CLIP || !(norm > k.a && norm <= 3.402823466e38f)) return {1.f, 1.f};
    const double c = k.a / root;
    return c >= 0x1p-126 ? Factor{static_cast<float>(c), 1.f} : Factor{static_cast<float>(c * 0x1p126), 0x1p-126f};
  }
}

template <int W, int NT, bool LAST, class D>
__device__ inline void sum_unit(const D& d, int64_t e0, int n, float shift, double& acc) {
  if constexpr (W == TRUST) add_products<NT, LAST>(d, e0, n, shift, acc);
  else add_squares<NT, LAST>(d, e0, n, acc);
}
template <int W, int SIZE, int NT, class D>
__device__ inline void second_part(const D& d, int64_t e0, int n, Factor f) {
  if constexpr (W == TRUST) {
    if (f.f != 0.f) apply_part<SIZE, NT>(d, e0, n, f.f);
  } else if constexpr (W == CLIP) {
    if (f.f != 1.f || f.pre != 1.f || d.out != d.grad) scale_part<SIZE, NT>(d, e0, n, f);
  }
}

// Sum of a block's per-thread values, in every thread (fixed order).
template <int NT>
__device__ inline double block_sum(double v, double* s) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0;
  for (int i = 0; i < NT / 64; ++i) t += s[i];
  return t;
}

// First pass: the block's units b, b + grid, ...
template <int W, bool LAST, class TB>
__global__ void __launch_bounds__(GT) grads_sum_kernel(TB tb, int count, int units, WorkArgs k,
                                                       double* __restrict__ partial) {
  __shared__ double s[GT / 64];
  double acc = 0;
  int p = find_tensor(tb, count, blockIdx.x);
  for (int c = blockIdx.x; c < units; c += gridDim.x) {
    if (p + 1 < count && tb.begin[p + 1] <= c) p = find_tensor(tb, count, c);
    const auto d = tb.desc[p];
    const int64_t e0 = int64_t(c - tb.begin[p]) * UNIT;
    sum_unit<W, GT, LAST>(d, e0, static_cast<int>(min(d.numel() - e0, int64_t(UNIT))), k.shift, acc);
  }
  acc = block_sum<GT>(acc, s);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

template <int W>
__global__ void __launch_bounds__(GT) grads_factor_kernel(const double* __restrict__ partial, int n, WorkArgs k,
                                                          Factor* __restrict__ out) {
  __shared__ double s[GT / 64];
  double v = 0;
  for (int i = threadIdx.x; i < n; i += GT) v += gp(partial)[i];
  const Factor f = factor<W>(block_sum<GT>(v, s), k, threadIdx.x == 0);
  if (threadIdx.x == 0) out[0] = f;
}

// Second pass, a part of a unit a block, the last first, up to the part `end`. No loop, and so no
// wait for a block's stores: with one the decoder's pass took 1137 us, without 857. Each part's block
// reads the factor that a launch of its own has formed: with the partial sums added up in every block
// the clipping of ResNet-50 took 55.5 us instead of 53.7.
constexpr int PARTS = UNIT / PART;
template <int W, class TB>
__global__ void __launch_bounds__(GT) grads_apply_kernel(TB tb, int count, int64_t end,
                                                         const Factor* __restrict__ f) {
  const int64_t at = end - 1 - blockIdx.x;
  const int c = static_cast<int>(at / PARTS);
  const int p = find_tensor(tb, count, c);
  const auto d = tb.desc[p];
  const int64_t e0 = int64_t(c - tb.begin[p]) * UNIT + at % PARTS * PART;
  const int64_t n = min(d.numel() - e0, int64_t(PART));
  if (n > 0) second_part<W, PART, GT>(d, e0, static_cast<int>(n), f[0]);
}

// A small call in one block: both passes, and no launch between them.
template <int W>
__global__ void __launch_bounds__(ONE_THREADS) grads_one_kernel(InlineTables<DescOf<W>> tb, int count,
                                                              WorkArgs k) {
  __shared__ double s[ONE_THREADS / 64];
  double acc = 0;
  for (int p = 0; p < count; ++p) {
    const auto d = tb.desc[p];
    for (int64_t e0 = 0; e0 < d.numel(); e0 += UNIT)
      sum_unit<W, ONE_THREADS, false>(d, e0, static_cast<int>(min(d.numel() - e0, int64_t(UNIT))), k.shift, acc);
  }
  const Factor f = factor<W>(block_sum<ONE_THREADS>(acc, s), k, threadIdx.x == 0);
  if constexpr (W != NORM)
    for (int p = 0; p < count; ++p) {
      const auto d = tb.desc[p];
      for (int64_t e0 = 0; e0 < d.numel(); e0 += UNIT)
        second_part<W, UNIT, ONE_THREADS>(d, e0, static_cast<int>(min(d.numel() - e0, int64_t(UNIT))), f);
    }
}

static size_t grads_need(int count) {
  return align256(sizeof(TrustDesc) * size_t(count)) + align256(sizeof(int32_t) * size_t(count)) +
         align256(sizeof(double) * MAX_BLOCKS) + 256;
}

}  // namespace kfac

using namespace kfac;

static bool known_dtype(kfac_dtype t) { return t == KFAC_F16 || t == KFAC_F32 || t == KFAC_BF16; }
static int dtype_size(kfac_dtype t) { return t == KFAC_F32 ? 4 : 2; }

static kfac_status sizes_validate(int32_t count, const int64_t* numel) {
  if (count < 0) return fail(KFAC_ERR_INVALID, "count must be >= 0");
  if (count > 0 && !numel) return fail(KFAC_ERR_INVALID, "numel is NULL");
  int64_t units = 0;
  for (int i = 0; i < count; ++i) {
    if (numel[i] < 0 || numel[i] > (int64_t(1) << 40))
      return fail(KFAC_ERR_INVALID, "numel[%d] = %lld out of range", i, static_cast<long long>(numel[i]));
    units += (numel[i] + UNIT - 1) / UNIT;
  }
  // a block's last step leads up to MAX_BLOCKS past them
  if (units > INT32_MAX - MAX_BLOCKS) return fail(KFAC_ERR_UNSUPPORTED, "too many elements in one call");
  return KFAC_OK;
}

// The buffers of a call: none that is written may share bytes with any other, apart
// from a read of the same tensor from the very same place.
struct Span {
  uintptr_t begin, end;
  int index;
  bool in_place;  // may be the written buffer of the same tensor, if it begins there
};

struct Spans {
  std::vector<Span> writes, reads;
  void write(const void* p, int64_t bytes, int i) { add(writes, p, bytes, i, false); }
  void read(const void* p, int64_t bytes, int i, bool in_place) { add(reads, p, bytes, i, in_place); }
  kfac_status check() {
    const auto before = [](const Span& a, const Span& b) { return a.begin < b.begin; };
    std::sort(writes.begin(), writes.end(), before);
    for (size_t a = 1; a < writes.size(); ++a)
      if (writes[a].begin < writes[a - 1].end)
        return fail(KFAC_ERR_INVALID, "tensors %d and %d: outputs overlap", writes[a - 1].index, writes[a].index);
    for (const Span& r : reads) {
      auto w = std::upper_bound(writes.begin(), writes.end(), r, before);
      if (w != writes.begin() && (w - 1)->end > r.begin) --w;
      for (; w != writes.end() && w->begin < r.end; ++w)
        if (!(r.in_place && w->index == r.index && w->begin == r.begin))
          return fail(KFAC_ERR_INVALID, "tensor %d: an input overlaps the output of tensor %d", r.index, w->index);
    }
    return KFAC_OK;
  }

 private:
  static void add(std::vector<Span>& v, const void* p, int64_t bytes, int i, bool in_place) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    v.push_back({a, a + static_cast<uintptr_t>(bytes), i, in_place});
  }
};

// The tensors that hold elements, as descriptors.
struct GradCall {
  std::vector<TrustDesc> desc;
  std::vector<int32_t> begin;
  Spans spans;
  int units = 0;
  int64_t read_bytes = 0;  // what the second pass reads again
  void add(const TrustDesc& d, int64_t bytes) {
    read_bytes += bytes;
    desc.push_back(d);
    begin.push_back(units);
    units += static_cast<int>((d.numel() + UNIT - 1) / UNIT);
  }
  static int64_t pack(int64_t numel, int type, bool wide, bool diagonal) {
    return numel | int64_t(type) << NormDesc::kType | int64_t(wide) << NormDesc::kWide |
           int64_t(diagonal) << NormDesc::kDiagonal;
  }
};

static kfac_status check_pointer(const void* p, int size, int i, const char* what) {
  if (!p) return fail(KFAC_ERR_INVALID, "tensor %d: %s is NULL", i, what);
  if (reinterpret_cast<uintptr_t>(p) % size) return fail(KFAC_ERR_INVALID, "tensor %d: %s is misaligned", i, what);
  return KFAC_OK;
}

// Calls of at most this many units go to one block, which takes less than the launches it saves: at
// 65536 elements the norm takes 11.1 us against 13.8, the clipping 14.2 against 19.9, the bounded
// update 17.3 against 22.9; at 131072 the clipping takes 25.5 against 20.6.
constexpr int ONE_UNITS = 16;
// The second pass finds what the first has read in the 256 MB last-level cache, if it fits (ResNet-50's
// 102 MB: second pass 29.7 us); beyond that the first pass does not keep it, and reads past the caches
// (streams of 2 GB: 7.2 TB/s against 6.4). The second pass always does, and writes past them too: lines
// left dirty there made the next call's sum take 36 us instead of 20.
constexpr int64_t CACHE_BYTES = int64_t(256) << 20;

template <int W, class TB>
static kfac_status launch_passes(const TB& tb, const GradCall& call, const WorkArgs& k, double* partial, Factor* f,
                                 hipStream_t s) {
  const int n = static_cast<int>(call.desc.size()), blocks = std::max(1, std::min(call.units, MAX_BLOCKS));
  constexpr int S = W == CLIP ? NORM : W;  // the same sum
  const int id = W == TRUST ? K_TRUST_SUM : K_NORM_SUM;
  if (call.read_bytes > CACHE_BYTES) {
    KFAC_LAUNCH(id, (grads_sum_kernel<S, true, TB>), dim3(blocks), dim3(GT), 0, s, tb, n, call.units, k, partial);
  } else {
    KFAC_LAUNCH(id, (grads_sum_kernel<S, false, TB>), dim3(blocks), dim3(GT), 0, s, tb, n, call.units, k, partial);
  }
  KFAC_CHECK_LAUNCH("grads_sum_kernel");
  KFAC_LAUNCH(K_GRADS_FACTOR, grads_factor_kernel<W>, dim3(1), dim3(GT), 0, s, partial, blocks, k, f);
  KFAC_CHECK_LAUNCH("grads_factor_kernel");
  if constexpr (W != NORM) {
    constexpr int64_t grid = int64_t(1) << 23;  // 2^31 threads
    for (int64_t end = int64_t(call.units) * PARTS; end > 0; end -= grid) {
      KFAC_LAUNCH(W == TRUST ? K_TRUST_APPLY : K_GRAD_SCALE, (grads_apply_kernel<W, TB>),
                  dim3(static_cast<unsigned>(std::min(end, grid))), dim3(GT), 0, s, tb, n, end, f);
      KFAC_CHECK_LAUNCH("grads_apply_kernel");
    }
  }
  return KFAC_OK;
}

template <int W>
static kfac_status launch_grads(const GradCall& call, int32_t count, const WorkArgs& k, void* workspace,
                                size_t ws_bytes, hipStream_t s) {
  kfac_status st = check_device();
  if (st) return st;
  st = check_workspace(workspace, ws_bytes, grads_need(count));
  if (st) return st;
  const int n = static_cast<int>(call.desc.size());
  using D = DescOf<W>;
  Carver cv(workspace);
  D* desc = cv.take<D>(count);
  int32_t* begin = cv.take<int32_t>(count);
  double* partial = cv.take<double>(MAX_BLOCKS);
  Factor* f = cv.take<Factor>(1);
  if (n <= InlineTables<D>::most) {
    InlineTables<D> tb;
    std::copy(call.desc.begin(), call.desc.end(), tb.desc);
    std::copy(call.begin.begin(), call.begin.end(), tb.begin);
    if (call.units > ONE_UNITS) return launch_passes<W>(tb, call, k, partial, f, s);
    KFAC_LAUNCH(K_GRADS_ONE, grads_one_kernel<W>, dim3(1), dim3(ONE_THREADS), 0, s, tb, n, k);
    KFAC_CHECK_LAUNCH("grads_one_kernel");
    return KFAC_OK;
  }
  const std::vector<D> sent(call.desc.begin(), call.desc.end());
  TableUpload tu;
  tu.add(desc, sent.data(), sizeof(D) * n);
  tu.add(begin, call.begin.data(), sizeof(int32_t) * n);
  if ((st = tu.flush(s))) return st;
  return launch_passes<W>(SentTables<D>{desc, begin}, call, k, partial, f, s);
}

extern "C" kfac_status kfac_grad_norm_workspace(int32_t count, const int64_t* numel, size_t* bytes) {
  if (!bytes) return fail(KFAC_ERR_INVALID, "bytes is NULL");
  kfac_status st = sizes_validate(count, numel);
  if (st) return st;
  *bytes = grads_need(count);
  return KFAC_OK;
}

static kfac_status grad_impl(int32_t count, const int64_t* numel, const kfac_dtype* dtype, const void* const* grad,
                             const kfac_dtype* out_dtype, void* const* out, bool clip, float max_norm, float* norm,
                             void* workspace, size_t ws_bytes, void* stream) {
  kfac_status st = sizes_validate(count, numel);
  if (st) return st;
  if (clip && !(max_norm > 0.f && max_norm - max_norm == 0.f))
    return fail(KFAC_ERR_INVALID, "max_norm must be positive and finite");
  if ((st = check_pointer(norm, 4, -1, "norm"))) return st;
  if (count > 0 && (!dtype || !grad || (clip && (!out_dtype || !out)))) return fail(KFAC_ERR_INVALID, "NULL array");
  GradCall call;
  for (int i = 0; i < count; ++i) {
    if (!known_dtype(dtype[i])) return fail(KFAC_ERR_UNSUPPORTED, "tensor %d: dtype %d", i, dtype[i]);
    if (clip && out_dtype[i] != dtype[i] && out_dtype[i] != KFAC_F32)
      return fail(KFAC_ERR_UNSUPPORTED, "tensor %d: out must have the gradient's type or fp32", i);
    if (numel[i] == 0) continue;
    if ((st = check_pointer(grad[i], dtype_size(dtype[i]), i, "grad"))) return st;
    TrustDesc d = {};
    d.grad = grad[i];
    d.info = GradCall::pack(numel[i], dtype[i], clip && out_dtype[i] == KFAC_F32, false);
    if (clip) {
      if ((st = check_pointer(out[i], dtype_size(out_dtype[i]), i, "out"))) return st;
      d.out = out[i];
      call.spans.write(out[i], numel[i] * dtype_size(out_dtype[i]), i);
      call.spans.read(grad[i], numel[i] * dtype_size(dtype[i]), i, out_dtype[i] == dtype[i]);
    }
    call.add(d, numel[i] * dtype_size(dtype[i]));
  }
  if (clip) {
    call.spans.write(norm, 4, -1);
    if ((st = call.spans.check())) return st;
  }
  const WorkArgs k = {norm, max_norm, 0.f, 0.f};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return clip ? launch_grads<CLIP>(call, count, k, workspace, ws_bytes, s)
              : launch_grads<NORM>(call, count, k, workspace, ws_bytes, s);
}

static kfac_status trust_impl(int32_t count, const int64_t* numel, const float* const* precond,
                              const kfac_dtype* grad_dtype, const void* const* grad, const float* const* fisher,
                              float shift, float* const* w, float lr, float delta, float* step, void* workspace,
                              size_t ws_bytes, void* stream) {
  kfac_status st = sizes_validate(count, numel);
  if (st) return st;
  if (!(lr >= 0.f && lr - lr == 0.f)) return fail(KFAC_ERR_INVALID, "lr must be finite and >= 0");
  if (!(delta > 0.f && delta - delta == 0.f)) return fail(KFAC_ERR_INVALID, "delta must be positive and finite");
  if (!(shift - shift == 0.f)) return fail(KFAC_ERR_INVALID, "shift must be finite");
  if ((st = check_pointer(step, 4, -1, "step"))) return st;
  if (count > 0 && (!precond || !grad_dtype || !grad || !w)) return fail(KFAC_ERR_INVALID, "NULL array");
  GradCall call;
  for (int i = 0; i < count; ++i) {
    if (numel[i] == 0) continue;
    if ((st = check_pointer(precond[i], 4, i, "precond"))) return st;
    if ((st = check_pointer(w[i], 4, i, "w"))) return st;
    TrustDesc d = {};
    d.grad = grad[i];
    d.precond = precond[i];
    d.out = w[i];
    d.info = GradCall::pack(numel[i], grad_dtype[i] & 3, true, false);
    if (grad[i]) {
      if (!known_dtype(grad_dtype[i])) return fail(KFAC_ERR_UNSUPPORTED, "tensor %d: dtype %d", i, grad_dtype[i]);
      if ((st = check_pointer(grad[i], dtype_size(grad_dtype[i]), i, "grad"))) return st;
      call.spans.read(grad[i], dtype_size(grad_dtype[i]) * numel[i], i, false);
    } else {
      if ((st = check_pointer(fisher ? fisher[i] : nullptr, 4, i, "fisher (and grad)"))) return st;
      d.grad = fisher[i];
      d.info = GradCall::pack(numel[i], KFAC_F32, true, true);
      call.spans.read(fisher[i], 4 * numel[i], i, false);
    }
    call.spans.read(precond[i], 4 * numel[i], i, false);
    call.spans.write(w[i], 4 * numel[i], i);
    call.add(d, numel[i] * 4);
  }
  call.spans.write(step, 8, -1);
  if ((st = call.spans.check())) return st;
  return launch_grads<TRUST>(call, count, WorkArgs{step, lr, delta, shift}, workspace, ws_bytes,
                             static_cast<hipStream_t>(stream));
}

extern "C" kfac_status kfac_grad_norm(int32_t count, const int64_t* numel, const kfac_dtype* dtype,
                                      const void* const* grad, float* norm, void* workspace, size_t ws_bytes,
                                      void* stream) {
  return guarded([&] {
    return grad_impl(count, numel, dtype, grad, nullptr, nullptr, false, 0.f, norm, workspace, ws_bytes, stream);
  });
}

extern "C" kfac_status kfac_grad_clip(int32_t count, const int64_t* numel, const kfac_dtype* dtype,
                                      const void* const* grad, const kfac_dtype* out_dtype, void* const* out,
                                      float max_norm, float* norm, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&] {
    return grad_impl(count, numel, dtype, grad, out_dtype, out, true, max_norm, norm, workspace, ws_bytes, stream);
  });
}

extern "C" kfac_status kfac_trust_update(int32_t count, const int64_t* numel, const float* const* precond,
                                         const kfac_dtype* grad_dtype, const void* const* grad,
                                         const float* const* fisher, float shift, float* const* w, float lr,
                                         float delta, float* step, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&] {
    return trust_impl(count, numel, precond, grad_dtype, grad, fisher, shift, w, lr, delta, step, workspace, ws_bytes,
                      stream);
  });
}
