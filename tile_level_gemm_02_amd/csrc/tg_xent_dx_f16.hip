// The vocabulary loss of include/tg_train.h for f16 inputs: the product dX = dt.W.
#include "tg_xent.hpp"

namespace tg {
template <>
tg_status xent_xgrad<E_F16>(const TileArgs& t, bool last, const float* factor, const float* R, int64_t ldr, void* ws, hipStream_t s)
{
    if (last)
        return xent_dx<E_F16, OutOf<E_F16>::O>(t, factor, R, ldr, ws, s);
    return xent_dx<E_F16, O_F32>(t, factor, R, ldr, ws, s);
}
}  // namespace tg
