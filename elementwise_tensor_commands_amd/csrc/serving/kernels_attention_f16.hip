// kernels_attention_f16.hip -- paged attention of one new token, f16 instances.
#include "ecmd_kern_attention.h"

namespace ecmd {

int launch_attention_f16(const AttnArgs &A, void *stream) { return launch_attn_type<S_F16>(A, stream); }
int launch_attention_join_f16(const AttnArgs &A, void *stream) { return launch_join_type<S_F16>(A, stream); }

}  // namespace ecmd
