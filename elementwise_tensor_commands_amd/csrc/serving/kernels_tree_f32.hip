// kernels_tree_f32.hip -- attention for trees of drafted tokens, f32 instances.
#include "ecmd_kern_tree.h"

namespace ecmd {

int launch_tree_f32(const TreeArgs &A, void *stream) { return launch_tree_type<S_F32>(A, stream); }

}  // namespace ecmd
