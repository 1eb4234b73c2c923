// The fused products of include/tg_ops.h for bf16 inputs: tg_linear.
#include "tg_fused.hpp"

namespace tg {
tg_status linear_bf16(const TileArgs& t, const EpiArgs& e, int y_dtype, void* ws, int64_t ws_bytes, void* stream)
{
    return linear_typed<E_BF16>(t, e, y_dtype, ws, ws_bytes, stream);
}

int64_t linear_ws_bytes_bf16(int64_t M, int64_t N, int64_t K) { return linear_ws_bytes<E_BF16>(M, N, K); }
}  // namespace tg
