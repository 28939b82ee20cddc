// The INT4 kernels of rq_fast_impl.h: n = 28 * 2^k, k = 7..9, and n = 2^12, 2^13,
// 2^14.
#include "rq_fast_impl.h"

namespace signrot {

bool rq_fast_supports(int n, int k, bool m28) {
  if (m28) return k >= 7 && k <= 10 && n == (28 << k);  // 3584, 7168, 14336, 28672
  return n == 4096 || n == 8192 || n == 16384;
}

hipError_t launch_rq_fast(const RqArgs& a, hipStream_t s) {
  if (a.mx_scale) return launch_rq_mx(a, s);
  if (a.m28) {
    switch (a.k) {
      case 7: return launch_shape<28, 7, false>(a, s);
      case 8: return launch_shape<28, 8, false>(a, s);
      case 9: return launch_shape<28, 9, false>(a, s);
      default: return launch_rq_halves(a, s);  // 28 * 2^10 as two halves of 28 * 2^9
    }
  }
  if (a.n == 4096) return launch_shape<32, 7, false>(a, s);
  if (a.n == 8192) return launch_shape<32, 8, false>(a, s);
  return launch_shape<32, 9, false>(a, s);
}

const char* rq_fast_name(int n) {
  if (n == 28672) return "rq_mfma28x2_w7";
  if (n % 28 == 0) return "rq_mfma28_w7";
  return "rq_mfma32_w8";
}

}  // namespace signrot
