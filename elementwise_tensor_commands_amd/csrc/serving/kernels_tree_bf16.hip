// kernels_tree_bf16.hip -- attention for trees of drafted tokens, bf16 instances.
#include "ecmd_kern_tree.h"

namespace ecmd {

int launch_tree_bf16(const TreeArgs &A, void *stream) { return launch_tree_type<S_BF16>(A, stream); }

}  // namespace ecmd
