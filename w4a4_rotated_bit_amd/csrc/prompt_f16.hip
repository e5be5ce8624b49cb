// prompt_f16.hip -- prompt_kernel.h for heads in binary16.
#include "prompt_kernel.h"

namespace convrot {
template void launch_prompt_typed<_Float16>(const convrot_attention_args&, const PromptPlan&, float*, hipStream_t);
}
