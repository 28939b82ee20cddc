// The INT4 kernels of rq_halves_impl.h: n = 28672 in two halves.
#include "rq_halves_impl.h"

namespace signrot {

hipError_t launch_rq_halves(const RqArgs& a, hipStream_t stream) { return launch_halves<false>(a, stream); }

}  // namespace signrot
