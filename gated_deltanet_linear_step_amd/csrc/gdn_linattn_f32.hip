// gdn_linattn_f32.hip -- the chunked decayed linear attention for f32 activations.

#include "gdn_linattn_chunk.h"

namespace gdn {

hipError_t launch_linattn_chunk_f32(const LinattnParams &p, int64_t segments, bool second, hipStream_t s)
{
    return linattn::launch_chunk_for<DT_F32>(p, segments, second, s);
}

}  // namespace gdn
