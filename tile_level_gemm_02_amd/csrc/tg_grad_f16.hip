// The fused products of include/tg_ops.h for fp16 inputs: the products of the backward passes.
#include "tg_fused.hpp"

namespace tg {
tg_status wgrad_f16(const TileArgs& t, int c_dtype, void* ws, int64_t ws_bytes, void* stream)
{
    return wgrad_typed<E_F16>(t, c_dtype, ws, ws_bytes, stream);
}

tg_status xgrad_f16(const TileArgs& t, void* ws, int64_t ws_bytes, void* stream)
{
    return xgrad_typed<E_F16>(t, ws, ws_bytes, stream);
}

tg_status group_f16(const TileArgs* t, int n, int w_dtype, void* ws, int64_t ws_bytes, void* stream, bool* taken)
{
    return group_typed<E_F16>(t, n, w_dtype, ws, ws_bytes, stream, taken);
}

int64_t group_ws_bytes_f16(const TileArgs* t, int n) { return group_ws_bytes<E_F16>(t, n); }

tg_status glu_dgu_f16(const TileArgs& t, const EpiArgs& e, void* ws, int64_t ws_bytes, void* stream)
{
    return glu_dgu_typed<E_F16>(t, e, ws, ws_bytes, stream);
}

tg_status dz_f16(const DzArgs& p, void* ws, int64_t ws_bytes, void* stream)
{
    return dz_typed<E_F16>(p, ws, ws_bytes, stream);
}

int64_t wgrad_ws_bytes_f16(int64_t N, int64_t K, int64_t M) { return wgrad_ws_bytes<E_F16>(N, K, M); }
}  // namespace tg
