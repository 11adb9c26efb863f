// The linear layer's tiles on E5M2 A and E4M3FN B.
#include "fp8q_linear.h"

namespace fp8q {

template <>
void launch_linear_tiles<FP8Q_E5M2, FP8Q_E4M3FN>(const Proj& p, const Epilogue& e, bool fast, bool low, const Split& t,
                                           hipStream_t st) {
  launch_out<FP8Q_E5M2, FP8Q_E4M3FN>(p, e, fast, low, t, st);
}

}  // namespace fp8q
