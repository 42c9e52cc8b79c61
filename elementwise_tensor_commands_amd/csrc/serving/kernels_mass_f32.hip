// kernels_mass_f32.hip -- the weight that attention gave to pages, f32 instances.
#include "ecmd_kern_mass.h"

namespace ecmd {

int launch_mass_f32(const MassArgs &A, void *stream) { return launch_mass_type<S_F32>(A, stream); }

}  // namespace ecmd
