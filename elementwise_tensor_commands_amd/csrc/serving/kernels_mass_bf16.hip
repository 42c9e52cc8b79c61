// kernels_mass_bf16.hip -- the weight that attention gave to pages, bf16 instances.
#include "ecmd_kern_mass.h"

namespace ecmd {

int launch_mass_bf16(const MassArgs &A, void *stream) { return launch_mass_type<S_BF16>(A, stream); }

}  // namespace ecmd
