// prompt_bf16.hip -- prompt_kernel.h for heads in bfloat16.
#include "prompt_kernel.h"

namespace convrot {
template void launch_prompt_typed<__bf16>(const convrot_attention_args&, const PromptPlan&, float*, hipStream_t);
}
