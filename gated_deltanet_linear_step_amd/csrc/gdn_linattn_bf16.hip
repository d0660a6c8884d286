// gdn_linattn_bf16.hip -- the chunked decayed linear attention for bf16 activations.

#include "gdn_linattn_chunk.h"

namespace gdn {

hipError_t launch_linattn_chunk_bf16(const LinattnParams &p, int64_t segments, bool second, hipStream_t s)
{
    return linattn::launch_chunk_for<DT_BF16>(p, segments, second, s);
}

}  // namespace gdn
