// The fused products of include/tg_ops.h for fp16 inputs: tg_glu.
#include "tg_fused.hpp"

namespace tg {
tg_status glu_f16(const TileArgs& t, const EpiArgs& e, int h_dtype, void* ws, int64_t ws_bytes, void* stream)
{
    return glu_typed<E_F16>(t, e, h_dtype, ws, ws_bytes, stream);
}

int64_t glu_ws_bytes_f16(int64_t M, int64_t F, int64_t D) { return glu_ws_bytes<E_F16>(M, F, D); }
}  // namespace tg
