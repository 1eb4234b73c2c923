// The vocabulary loss of include/tg_train.h for bf16 inputs: its forward product and the piecewise gradient.
#include "tg_xent.hpp"

namespace tg {
tg_status xent_forward_bf16(const XentCall& q) { return xent_forward<E_BF16>(q); }
tg_status xent_backward_bf16(const XentCall& q) { return xent_backward<E_BF16>(q); }
}  // namespace tg
