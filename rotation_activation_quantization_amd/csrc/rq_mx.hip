// The fast kernels (rq_fast_impl.h, rq_halves_impl.h) with MXFP4 output, d given as
// (c, sigma).  A block of 32 channels lies in one to four lanes after the transform, so
// no row maximum is exchanged between waves; but every wave stores scales beside its
// codes: 8192 x 14336 takes 71.6 us (INT4 66.7), with the producer 115 (107), 8192 x 28672
// 136 (129).
#include "rq_fast_impl.h"
#include "rq_halves_impl.h"

namespace signrot {

hipError_t launch_rq_mx(const RqArgs& a, hipStream_t s) {
  if (a.m28) {
    switch (a.k) {
      case 7: return launch_shape<28, 7, true>(a, s);
      case 8: return launch_shape<28, 8, true>(a, s);
      case 9: return launch_shape<28, 9, true>(a, s);
      default: return launch_halves<true>(a, s);  // 28 * 2^10 as two halves of 28 * 2^9
    }
  }
  if (a.n == 4096) return launch_shape<32, 7, true>(a, s);
  if (a.n == 8192) return launch_shape<32, 8, true>(a, s);
  return launch_shape<32, 9, true>(a, s);
}

}  // namespace signrot
