// kernels_tree_f16.hip -- attention for trees of drafted tokens, f16 instances.
#include "ecmd_kern_tree.h"

namespace ecmd {

int launch_tree_f16(const TreeArgs &A, void *stream) { return launch_tree_type<S_F16>(A, stream); }

}  // namespace ecmd
