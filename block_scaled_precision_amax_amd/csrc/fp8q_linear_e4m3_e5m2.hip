// The linear layer's tiles on E4M3FN A and E5M2 B.
#include "fp8q_linear.h"

namespace fp8q {

template <>
void launch_linear_tiles<FP8Q_E4M3FN, FP8Q_E5M2>(const Proj& p, const Epilogue& e, bool fast, bool low, const Split& t,
                                           hipStream_t st) {
  launch_out<FP8Q_E4M3FN, FP8Q_E5M2>(p, e, fast, low, t, st);
}

}  // namespace fp8q
