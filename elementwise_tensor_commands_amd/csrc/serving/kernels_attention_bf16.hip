// kernels_attention_bf16.hip -- paged attention of one new token, bf16 instances.
#include "ecmd_kern_attention.h"

namespace ecmd {

int launch_attention_bf16(const AttnArgs &A, void *stream) { return launch_attn_type<S_BF16>(A, stream); }
int launch_attention_join_bf16(const AttnArgs &A, void *stream) { return launch_join_type<S_BF16>(A, stream); }

}  // namespace ecmd
