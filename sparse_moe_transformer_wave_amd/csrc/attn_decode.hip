// attn_decode.hip -- decode attention over the bf16 paged cache (attn_core.h).
#include "attn_core.h"

namespace flint {

size_t attn_decode_call_bytes(const Cache &c, int64_t B) { return call_bytes(c, B); }

size_t attn_decode_ws_bytes(const Cache &c, int64_t B) { return any_batch_bytes(c, B); }

hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t st)
{
    return a.c.D == 128 ? launch_d<128, false>(a, st) : launch_d<64, false>(a, st);
}

}  // namespace flint
