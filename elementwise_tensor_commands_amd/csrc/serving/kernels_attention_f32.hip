// kernels_attention_f32.hip -- paged attention of one new token, f32 instances.
#include "ecmd_kern_attention.h"

namespace ecmd {

int launch_attention_f32(const AttnArgs &A, void *stream) { return launch_attn_type<S_F32>(A, stream); }
int launch_attention_join_f32(const AttnArgs &A, void *stream) { return launch_join_type<S_F32>(A, stream); }

}  // namespace ecmd
