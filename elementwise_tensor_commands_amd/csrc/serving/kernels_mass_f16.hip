// kernels_mass_f16.hip -- the weight that attention gave to pages, f16 instances.
#include "ecmd_kern_mass.h"

namespace ecmd {

int launch_mass_f16(const MassArgs &A, void *stream) { return launch_mass_type<S_F16>(A, stream); }

}  // namespace ecmd
