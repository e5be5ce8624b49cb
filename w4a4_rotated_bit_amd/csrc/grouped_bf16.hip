// grouped_bf16.hip -- the group-scaled 4-bit linear for bf16 x.
#include "grouped_kernel.h"

namespace convrot {

void launch_grouped_bf16(const grouped::GroupedParams& p, int group, hipStream_t s) { grouped::launch_type<__bf16>(p, group, s); }

}  // namespace convrot
