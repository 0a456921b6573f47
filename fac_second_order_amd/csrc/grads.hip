// Norms and updates over many tensors: the global gradient norm, clipping by it, and
// the update whose length is bounded by its predicted KL divergence.
//
// A tensor is cut into chunks of CHUNK elements; a call's chunks are numbered through
// all tensors and dealt to the blocks in contiguous ranges, so the order of every sum
// depends on the sizes alone and results are deterministic. Sums are kept in fp64 (a
// square of any fp32 value fits, and a multiply-add costs what an fp32 one costs);
// each block leaves one partial sum, and the blocks of the next launch add them all.
// HBM-bound: one read of the gradients for the norm, a second read and the write for
// the result.
#include <algorithm>

#include "row_ops.hpp"

namespace kfac {

constexpr int CHUNK = 16384;       // elements of a work item
constexpr int MAX_BLOCKS = 2048;   // 8 blocks of 4 waves for each of 256 compute units
constexpr int GT = 256;            // threads per block

struct GradDesc {
  const void* grad;  // NULL: the Fisher is diagonal, g = P (fisher + shift)
  const float* fisher;
  const float* precond;
  void* out;         // clipped gradient, or the weights of the update
  int64_t numel;
  int32_t grad_dtype, out_dtype;
};

// Sum of a block's per-thread values, in every thread (fixed order).
__device__ inline double block_sum(double v, double* s) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0;
  for (int i = 0; i < GT / 64; ++i) t += s[i];
  return t;
}

__device__ inline double partial_total(const double* partial, int n, double* s) {
  double v = 0;
  for (int i = threadIdx.x; i < n; i += GT) v += gp(partial)[i];
  return block_sum(v, s);
}

// f(tensor, first element, one past the last) for each of this block's chunks.
template <class F>
__device__ inline void for_chunks(const GradDesc* desc, const int32_t* begin, int count, int total, bool reverse, F f) {
  const int b = reverse ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  const int c0 = static_cast<int>(int64_t(total) * b / gridDim.x);
  const int c1 = static_cast<int>(int64_t(total) * (b + 1) / gridDim.x);
  if (c0 >= c1) return;
  int p = find_problem(begin, count, c0);
  for (int c = c0; c < c1; ++c) {
    while (p + 1 < count && begin[p + 1] <= c) ++p;
    const GradDesc d = desc[p];
    const int64_t e0 = int64_t(c - begin[p]) * CHUNK;
    f(d, e0, min(d.numel, e0 + CHUNK));
  }
}

// f(dtype tag) with the type of a code.
template <class F>
__device__ inline void with_type(int32_t code, F f) {
  if (code == KFAC_F32) f(float{});
  else if (code == KFAC_BF16) f(__bf16{});
  else f(_Float16{});
}

__global__ void __launch_bounds__(GT) norm_partial_kernel(const GradDesc* __restrict__ desc,
                                                          const int32_t* __restrict__ begin, int count, int total,
                                                          double* __restrict__ partial) {
  __shared__ double s[GT / 64];
  double acc = 0;
  for_chunks(desc, begin, count, total, false, [&](const GradDesc& d, int64_t e0, int64_t e1) {
    with_type(d.grad_dtype, [&](auto tag) {
      using T = decltype(tag);
      using C = Chunk16<T>;
      const KG T* g = gp(static_cast<const T*>(d.grad));
      const int64_t full = e0 + (e1 - e0) / C::ev * C::ev;
      for (int64_t i = e0 + int64_t(threadIdx.x) * C::ev; i < full; i += GT * C::ev) {
        const typename C::vec v = *reinterpret_cast<const KG typename C::vec*>(g + i);
#pragma unroll
        for (int u = 0; u < C::ev; ++u) {
          const double x = static_cast<float>(v[u]);
          acc = fma(x, x, acc);
        }
      }
      const int64_t i = full + threadIdx.x;
      if (i < e1) {
        const double x = static_cast<float>(g[i]);
        acc = fma(x, x, acc);
      }
    });
  });
  acc = block_sum(acc, s);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

__global__ void __launch_bounds__(GT) norm_finish_kernel(const double* __restrict__ partial, int n, float* norm) {
  __shared__ double s[GT / 64];
  const double q = partial_total(partial, n, s);
  if (threadIdx.x == 0) norm[0] = static_cast<float>(sqrt(q));
}

// out = coef * grad, coef in fp32, the product rounded once to the type of out.
__global__ void __launch_bounds__(GT) grad_scale_kernel(const GradDesc* __restrict__ desc,
                                                        const int32_t* __restrict__ begin, int count, int total,
                                                        const double* __restrict__ partial, int n, float max_norm,
                                                        float* norm) {
  __shared__ double s[GT / 64];
  const double root = sqrt(partial_total(partial, n, s));
  const float shown = static_cast<float>(root);
  const float coef = shown > max_norm && shown <= 3.402823466e38f ? static_cast<float>(max_norm / root) : 1.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) norm[0] = shown;
  for_chunks(desc, begin, count, total, true, [&](const GradDesc& d, int64_t e0, int64_t e1) {
    if (coef == 1.f && d.out == d.grad) return;
    with_type(d.grad_dtype, [&](auto tag) {
      using T = decltype(tag);
      const auto scale = [&](auto otag) {
        using O = decltype(otag);
        constexpr int ev = Chunk16<T>::ev;
        typedef O ovec __attribute__((ext_vector_type(ev), aligned(sizeof(O))));
        using V = typename Chunk16<T>::vec;
        const KG T* g = gp(static_cast<const T*>(d.grad));
        KG O* o = gp(static_cast<O*>(d.out));
        const int64_t full = e0 + (e1 - e0) / ev * ev;
        for (int64_t i = e0 + int64_t(threadIdx.x) * ev; i < full; i += GT * ev) {
          const V v = *reinterpret_cast<const KG V*>(g + i);
          ovec w;
#pragma unroll
          for (int u = 0; u < ev; ++u) w[u] = static_cast<O>(static_cast<float>(v[u]) * coef);
          *reinterpret_cast<KG ovec*>(o + i) = w;
        }
        const int64_t i = full + threadIdx.x;
        if (i < e1) o[i] = static_cast<O>(static_cast<float>(g[i]) * coef);
      };
      if (d.out_dtype == KFAC_F32) scale(float{});
      else scale(T{});
    });
  });
}

// q = sum of P * g, the preconditioned gradient against the gradient it came from.
__global__ void __launch_bounds__(GT) trust_partial_kernel(const GradDesc* __restrict__ desc,
                                                           const int32_t* __restrict__ begin, int count, int total,
                                                           float shift, double* __restrict__ partial) {
  __shared__ double s[GT / 64];
  double acc = 0;
  for_chunks(desc, begin, count, total, false, [&](const GradDesc& d, int64_t e0, int64_t e1) {
    const KG float* p = gp(d.precond);
    if (!d.grad) {
      for (int64_t i = e0 + threadIdx.x; i < e1; i += GT) {
        const double x = p[i];
        acc = fma(x * x, static_cast<double>(gp(d.fisher)[i]) + shift, acc);
      }
      return;
    }
    with_type(d.grad_dtype, [&](auto tag) {
      using T = decltype(tag);
      typedef T gvec __attribute__((ext_vector_type(4), aligned(sizeof(T))));
      using V = Chunk16<float>::vec;
      const KG T* g = gp(static_cast<const T*>(d.grad));
      const int64_t full = e0 + (e1 - e0) / 4 * 4;
      for (int64_t i = e0 + int64_t(threadIdx.x) * 4; i < full; i += GT * 4) {
        const V v = *reinterpret_cast<const KG V*>(p + i);
        const gvec w = *reinterpret_cast<const KG gvec*>(g + i);
#pragma unroll
        for (int u = 0; u < 4; ++u) acc = fma(static_cast<double>(v[u]), static_cast<double>(static_cast<float>(w[u])), acc);
      }
      const int64_t i = full + threadIdx.x;
      if (i < e1) acc = fma(static_cast<double>(p[i]), static_cast<double>(static_cast<float>(g[i])), acc);
    });
  });
  acc = block_sum(acc, s);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

// w -= step * P, step = min(lr, sqrt(2 delta / |q|)).
__global__ void __launch_bounds__(GT) trust_apply_kernel(const GradDesc* __restrict__ desc,
                                                         const int32_t* __restrict__ begin, int count, int total,
                                                         const double* __restrict__ partial, int n, float lr,
                                                         float delta, float* step_out) {
  __shared__ double s[GT / 64];
  const double q = partial_total(partial, n, s);
  float step = 0.f;  // q not finite: no update
  if (q - q == 0) step = fmin(static_cast<double>(lr), sqrt(2.0 * delta / fabs(q)));
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    step_out[0] = step;
    step_out[1] = static_cast<float>(q);
  }
  if (step == 0.f) return;
  for_chunks(desc, begin, count, total, true, [&](const GradDesc& d, int64_t e0, int64_t e1) {
    using V = Chunk16<float>::vec;
    const KG float* p = gp(d.precond);
    KG float* w = gp(static_cast<float*>(d.out));
    const int64_t full = e0 + (e1 - e0) / 4 * 4;
    for (int64_t i = e0 + int64_t(threadIdx.x) * 4; i < full; i += GT * 4) {
      const V v = *reinterpret_cast<const KG V*>(p + i);
      V x = *reinterpret_cast<const KG V*>(w + i);
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = fmaf(-step, v[u], x[u]);
      *reinterpret_cast<KG V*>(w + i) = x;
    }
    const int64_t i = full + threadIdx.x;
    if (i < e1) w[i] = fmaf(-step, p[i], w[i]);
  });
}

static size_t grads_need(int count) {
  return align256(sizeof(GradDesc) * size_t(count)) + align256(sizeof(int32_t) * size_t(count)) +
         align256(sizeof(double) * MAX_BLOCKS);
}

}  // namespace kfac

using namespace kfac;

static bool known_dtype(kfac_dtype t) { return t == KFAC_F16 || t == KFAC_F32 || t == KFAC_BF16; }
static int dtype_size(kfac_dtype t) { return t == KFAC_F32 ? 4 : 2; }

static kfac_status sizes_validate(int32_t count, const int64_t* numel) {
  if (count < 0) return fail(KFAC_ERR_INVALID, "count must be >= 0");
  if (count > 0 && !numel) return fail(KFAC_ERR_INVALID, "numel is NULL");
  int64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    if (numel[i] < 0 || numel[i] > (int64_t(1) << 40))
      return fail(KFAC_ERR_INVALID, "numel[%d] = %lld out of range", i, static_cast<long long>(numel[i]));
    chunks += (numel[i] + CHUNK - 1) / CHUNK;
  }
  if (chunks >= (int64_t(1) << 31)) return fail(KFAC_ERR_UNSUPPORTED, "too many elements in one call");
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
  std::vector<GradDesc> desc;
  std::vector<int32_t> begin;
  Spans spans;
  int total = 0;  // chunks
  void add(const GradDesc& d) {
    desc.push_back(d);
    begin.push_back(total);
    total += static_cast<int>((d.numel + CHUNK - 1) / CHUNK);
  }
  int blocks() const { return total < 1 ? 1 : total < MAX_BLOCKS ? total : MAX_BLOCKS; }
};

static kfac_status check_pointer(const void* p, int size, int i, const char* what) {
  if (!p) return fail(KFAC_ERR_INVALID, "tensor %d: %s is NULL", i, what);
  if (reinterpret_cast<uintptr_t>(p) % size) return fail(KFAC_ERR_INVALID, "tensor %d: %s is misaligned", i, what);
  return KFAC_OK;
}

struct GradTables {
  GradDesc* desc;
  int32_t* begin;
  double* partial;
};

static kfac_status send_tables(const GradCall& call, int32_t count, void* workspace, size_t ws_bytes, hipStream_t s,
                               GradTables* t) {
  kfac_status st = check_device();
  if (st) return st;
  st = check_workspace(workspace, ws_bytes, grads_need(count));
  if (st) return st;
  Carver cv(workspace);
  t->desc = cv.take<GradDesc>(count);
  t->begin = cv.take<int32_t>(count);
  t->partial = cv.take<double>(MAX_BLOCKS);
  TableUpload tu;
  tu.add(t->desc, call.desc.data(), sizeof(GradDesc) * call.desc.size());
  tu.add(t->begin, call.begin.data(), sizeof(int32_t) * call.begin.size());
  return tu.flush(s);
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
    GradDesc d = {grad[i], nullptr, nullptr, nullptr, numel[i], dtype[i], dtype[i]};
    if (clip) {
      if ((st = check_pointer(out[i], dtype_size(out_dtype[i]), i, "out"))) return st;
      d.out = out[i];
      d.out_dtype = out_dtype[i];
      call.spans.write(d.out, d.numel * dtype_size(d.out_dtype), i);
      call.spans.read(d.grad, d.numel * dtype_size(d.grad_dtype), i, d.out_dtype == d.grad_dtype);
    }
    call.add(d);
  }
  if (clip) {
    call.spans.write(norm, 4, -1);
    if ((st = call.spans.check())) return st;
  }
  GradTables t;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = send_tables(call, count, workspace, ws_bytes, s, &t))) return st;
  const int n = static_cast<int>(call.desc.size()), blocks = call.blocks();
  KFAC_LAUNCH(K_NORM_PARTIAL, norm_partial_kernel, dim3(blocks), dim3(GT), 0, s, t.desc, t.begin, n, call.total,
              t.partial);
  KFAC_CHECK_LAUNCH("norm_partial_kernel");
  if (clip) {
    KFAC_LAUNCH(K_GRAD_SCALE, grad_scale_kernel, dim3(blocks), dim3(GT), 0, s, t.desc, t.begin, n, call.total,
                t.partial, blocks, max_norm, norm);
    KFAC_CHECK_LAUNCH("grad_scale_kernel");
  } else {
    KFAC_LAUNCH(K_NORM_FINISH, norm_finish_kernel, dim3(1), dim3(GT), 0, s, t.partial, blocks, norm);
    KFAC_CHECK_LAUNCH("norm_finish_kernel");
  }
  return KFAC_OK;
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
    GradDesc d = {grad[i], nullptr, precond[i], w[i], numel[i], grad_dtype[i], KFAC_F32};
    if (grad[i]) {
      if (!known_dtype(grad_dtype[i])) return fail(KFAC_ERR_UNSUPPORTED, "tensor %d: dtype %d", i, grad_dtype[i]);
      if ((st = check_pointer(grad[i], dtype_size(grad_dtype[i]), i, "grad"))) return st;
      call.spans.read(grad[i], dtype_size(grad_dtype[i]) * numel[i], i, false);
    } else {
      if ((st = check_pointer(fisher ? fisher[i] : nullptr, 4, i, "fisher (and grad)"))) return st;
      d.fisher = fisher[i];
      call.spans.read(fisher[i], 4 * numel[i], i, false);
    }
    call.spans.read(precond[i], 4 * numel[i], i, false);
    call.spans.write(w[i], 4 * numel[i], i);
    call.add(d);
  }
  call.spans.write(step, 8, -1);
  if ((st = call.spans.check())) return st;
  GradTables t;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if ((st = send_tables(call, count, workspace, ws_bytes, s, &t))) return st;
  const int n = static_cast<int>(call.desc.size()), blocks = call.blocks();
  KFAC_LAUNCH(K_TRUST_PARTIAL, trust_partial_kernel, dim3(blocks), dim3(GT), 0, s, t.desc, t.begin, n, call.total,
              shift, t.partial);
  KFAC_CHECK_LAUNCH("trust_partial_kernel");
  KFAC_LAUNCH(K_TRUST_APPLY, trust_apply_kernel, dim3(blocks), dim3(GT), 0, s, t.desc, t.begin, n, call.total,
              t.partial, blocks, lr, delta, step);
  KFAC_CHECK_LAUNCH("trust_apply_kernel");
  return KFAC_OK;
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
