// gdn_attn_f16.hip -- softmax attention of f16 queries, keys and values (gdn_attn_prefill.h, gdn_attn_decode.h).
#include "gdn_attn_decode.h"

namespace gdn {

hipError_t launch_attn_prefill_f16(const AttnPrefillParams &p, unsigned grid, hipStream_t s)
{
    return attn::launch_prefill<DT_F16>(p, grid, s);
}

hipError_t launch_attn_decode_f16(const AttnDecodeParams &p, unsigned grid, hipStream_t s)
{
    return attn::launch_decode<DT_F16>(p, grid, s);
}

}  // namespace gdn
