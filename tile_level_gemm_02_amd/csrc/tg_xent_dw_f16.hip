// The vocabulary loss of include/tg_train.h for f16 inputs: the product dW = dt^T.x.
#include "tg_xent.hpp"

namespace tg {
template <>
tg_status xent_wgrad<E_F16>(const TileArgs& t, int dtype, const float* factor, void* ws, hipStream_t s)
{
    if (dtype == TG_F32)
        return xent_product<E_F16, O_F32, A_MCONTIG>(t, factor, nullptr, 0, ws, s);
    return xent_product<E_F16, OutOf<E_F16>::O, A_MCONTIG>(t, factor, nullptr, 0, ws, s);
}
}  // namespace tg
