// gdn_linattn_f16.hip -- the chunked decayed linear attention for f16 activations.

#include "gdn_linattn_chunk.h"

namespace gdn {

hipError_t launch_linattn_chunk_f16(const LinattnParams &p, int64_t segments, bool second, hipStream_t s)
{
    return linattn::launch_chunk_for<DT_F16>(p, segments, second, s);
}

}  // namespace gdn
