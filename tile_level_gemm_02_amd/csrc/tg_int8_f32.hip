// tg_linear_i8 (include/tg_int8.h) with f32 outputs.
#include "tg_int8.hpp"

namespace tg {
tg_status i8_linear_f32(const TileArgs& t, const I8Epi& e, void* ws, int64_t ws_bytes, hipStream_t s)
{
    return i8_linear<O_F32>(t, e, ws, ws_bytes, s);
}
}  // namespace tg
