// Kernel ids of the loss, clipping and bounded-update kernels, numbered on from those of
// common.hpp (the recorded HBM traffic of the inverse's update kernel holds for common.hpp
// as it is), and the 16-byte groups these kernels move.
#pragma once
#include <new>

#include "common.hpp"

namespace kfac {

enum RowKernelId {
  K_NORM_SUM = K_COUNT,  // grads_sum_kernel of the norm and the clipping
  K_TRUST_SUM,           // grads_sum_kernel of the bounded update
  K_GRADS_FACTOR,
  K_GRAD_SCALE,          // grads_apply_kernel of the clipping
  K_TRUST_APPLY,         // grads_apply_kernel of the bounded update
  K_GRADS_ONE,
  K_LOSS_COUNT,
  K_LOSS_NONEMPTY,
  K_POLICY_ROWS,
  K_POLICY_TERMS,
  K_POLICY_FINISH,
  K_POLICY_PART,
  K_POLICY_JOIN,
  K_PREF_ROWS,
  K_PREF_PAIRS,
  K_PREF_FINISH,
  K_PREF_GRAD,
  K_QUANTIZE,
  K_DEQUANTIZE,
  K_LINEAR_Q8,
  K_GRAD_Q8,           // q8_tn_kernel of the weight gradient
  K_GRAD_Q8_JOIN,
  K_FACTOR_Q8,         // q8_tn_kernel of the factors
  K_FACTOR_Q8_JOIN,
  K_TOTAL
};

// N elements at any address that is a multiple of an element's size: global memory takes up to
// 16 bytes as one access, aligned or not.
template <class T, int N = 16 / sizeof(T)>
struct Pack {
  static constexpr int n = N;
  typedef T vec __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

// Loads and stores of a pack; PAST: nothing looks at it again before the caches have turned over,
// so it passes them by. (The element type and the length are named, not the vector: a template
// argument would lose its alignment. PAST is no run-time choice: the compiler would make one
// plain access of both.)
template <bool PAST, class T, int N = 16 / sizeof(T)>
__device__ inline typename Pack<T, N>::vec load_pack(const KG T* p) {
  const auto from = reinterpret_cast<const KG typename Pack<T, N>::vec*>(p);
  if constexpr (PAST) return __builtin_nontemporal_load(from);
  else return *from;
}
template <bool PAST, class T, int N = 16 / sizeof(T)>
__device__ inline void store_pack(KG T* p, typename Pack<T, N>::vec v) {
  const auto to = reinterpret_cast<KG typename Pack<T, N>::vec*>(p);
  if constexpr (PAST) __builtin_nontemporal_store(v, to);
  else *to = v;
}

// Host tables are vectors: a failed allocation leaves an entry point as a status, not as
// an exception.
template <class F>
static kfac_status guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(KFAC_ERR_INVALID, "out of host memory for the call's tables");
  }
}

}  // namespace kfac
