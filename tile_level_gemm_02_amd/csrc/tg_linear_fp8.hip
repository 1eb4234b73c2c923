// The fused products of include/tg_ops.h for fp8 inputs: tg_linear.
#include "tg_fused.hpp"

namespace tg {
tg_status linear_fp8(const TileArgs& t, const EpiArgs& e, int y_dtype, void* ws, int64_t ws_bytes, void* stream)
{
    return linear_typed<E_FP8>(t, e, y_dtype, ws, ws_bytes, stream);
}
}  // namespace tg
