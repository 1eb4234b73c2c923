// The vocabulary loss of include/tg_train.h for f16 inputs: its forward product and the piecewise gradient.
#include "tg_xent.hpp"

namespace tg {
tg_status xent_forward_f16(const XentCall& q) { return xent_forward<E_F16>(q); }
tg_status xent_backward_f16(const XentCall& q) { return xent_backward<E_F16>(q); }
}  // namespace tg
