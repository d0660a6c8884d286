// gdn_attn_bf16.hip -- softmax attention of bf16 queries, keys and values (gdn_attn_prefill.h, gdn_attn_decode.h).
#include "gdn_attn_decode.h"

namespace gdn {

hipError_t launch_attn_prefill_bf16(const AttnPrefillParams &p, unsigned grid, hipStream_t s)
{
    return attn::launch_prefill<DT_BF16>(p, grid, s);
}

hipError_t launch_attn_decode_bf16(const AttnDecodeParams &p, unsigned grid, hipStream_t s)
{
    return attn::launch_decode<DT_BF16>(p, grid, s);
}

}  // namespace gdn
