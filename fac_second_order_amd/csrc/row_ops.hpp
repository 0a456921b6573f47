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
  K_POLICY_ROWS,
  K_POLICY_FINISH,
  K_PREF_ROWS,
  K_PREF_PAIRS,
  K_PREF_FINISH,
  K_PREF_GRAD,
  K_TOTAL
};

// 16 bytes of T at any address that is a multiple of its size: global memory takes them
// as one access, aligned or not.
template <class T>
struct Chunk16 {
  static constexpr int ev = 16 / sizeof(T);
  typedef T vec __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
};

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
