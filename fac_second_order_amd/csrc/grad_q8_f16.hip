// Weight gradients from fp16 gradients and rows in 8 bits.
#include "q8_tn_kernel.hpp"

namespace kfac {

template kfac_status launch_grad_tiles<_Float16, 2, false>(const TnArgs<false>&, hipStream_t);
template kfac_status launch_grad_tiles<_Float16, 2, true>(const TnArgs<false>&, hipStream_t);
template kfac_status launch_grad_tiles<_Float16, 4, false>(const TnArgs<false>&, hipStream_t);
template kfac_status launch_grad_tiles<_Float16, 4, true>(const TnArgs<false>&, hipStream_t);

}  // namespace kfac
