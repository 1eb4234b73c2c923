// The vocabulary loss of include/tg_train.h for bf16 inputs: the product dW = dt^T.x.
#include "tg_xent.hpp"

namespace tg {
template <>
tg_status xent_wgrad<E_BF16>(const TileArgs& t, int dtype, const float* factor, void* ws, hipStream_t s)
{
    if (dtype == TG_F32)
        return xent_product<E_BF16, O_F32, A_MCONTIG>(t, factor, nullptr, 0, ws, s);
    return xent_product<E_BF16, OutOf<E_BF16>::O, A_MCONTIG>(t, factor, nullptr, 0, ws, s);
}
}  // namespace tg
