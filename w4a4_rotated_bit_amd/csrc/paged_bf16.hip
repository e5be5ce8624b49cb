// paged_bf16.hip -- paged_kernel.h for heads in bfloat16.
#include "paged_kernel.h"

namespace convrot {
template void launch_paged_typed<__bf16>(const convrot_attention_paged_args&, const PagedPlan&, float*, hipStream_t);
}
