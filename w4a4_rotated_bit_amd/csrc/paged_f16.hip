// paged_f16.hip -- paged_kernel.h for heads in binary16.
#include "paged_kernel.h"

namespace convrot {
template void launch_paged_typed<_Float16>(const convrot_attention_paged_args&, const PagedPlan&, float*, hipStream_t);
}
