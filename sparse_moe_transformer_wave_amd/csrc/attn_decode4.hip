// attn_decode4.hip -- decode attention over the 4-bit paged cache (attn_core.h).
#include "attn_core.h"
#include "serve.h"

namespace flint {

size_t attn_decode4_call_bytes(const Cache &c, int64_t B) { return call_bytes(c, B); }

size_t attn_decode4_ws_bytes(const Cache &c, int64_t B) { return any_batch_bytes(c, B); }

hipError_t launch_attn_decode4(const AttnArgs &a, hipStream_t st)
{
    return a.c.D == 128 ? launch_d<128, true>(a, st) : launch_d<64, true>(a, st);
}

}  // namespace flint
