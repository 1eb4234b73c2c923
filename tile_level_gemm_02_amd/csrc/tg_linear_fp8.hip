// The fused products of include/tg_ops.h for fp8 inputs: tg_linear.
#include "tg_fused.hpp"

namespace tg {
tg_status linear_fp8(const TileArgs& t, const EpiArgs& e, int y_dtype, void* ws, int64_t ws_bytes, void* stream)
{
    return linear_typed<E_FP8>(t, e, y_dtype, ws, ws_bytes, stream);
}

int64_t linear_ws_bytes_fp8(int64_t M, int64_t N, int64_t K) { return linear_ws_bytes<E_FP8>(M, N, K); }
}  // namespace tg
