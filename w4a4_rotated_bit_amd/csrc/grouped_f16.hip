// grouped_f16.hip -- the group-scaled 4-bit linear for f16 x.
#include "grouped_kernel.h"

namespace convrot {

void launch_grouped_f16(const grouped::GroupedParams& p, int group, hipStream_t s) { grouped::launch_type<_Float16>(p, group, s); }

}  // namespace convrot
