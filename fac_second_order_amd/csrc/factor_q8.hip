// Kronecker factors from rows in 8 bits.
#include "q8_tn_kernel.hpp"

namespace kfac {

template kfac_status launch_tiles<_Float16, true, 2, false>(const TnArgs<true>&, hipStream_t);
template kfac_status launch_tiles<_Float16, true, 2, true>(const TnArgs<true>&, hipStream_t);
template kfac_status launch_tiles<_Float16, true, 3, false>(const TnArgs<true>&, hipStream_t);
template kfac_status launch_tiles<_Float16, true, 3, true>(const TnArgs<true>&, hipStream_t);
template kfac_status launch_tiles<_Float16, true, 4, false>(const TnArgs<true>&, hipStream_t);
template kfac_status launch_tiles<_Float16, true, 4, true>(const TnArgs<true>&, hipStream_t);

}  // namespace kfac
