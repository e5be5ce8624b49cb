// attention_api.hip -- device entry points of attention and of the paged cache
// that it reads: checks on the host, launches on the caller's stream, no state.
#include <hip/hip_runtime.h>

#include "../../include/convrot.h"
#include "attention_ops.h"
#include "internal.h"
#include "kernels.h"

using namespace convrot;

namespace convrot {

void launch_attention_paged(const convrot_attention_paged_args& a, const PagedPlan& plan, float* partial, hipStream_t s)
{
    a.dtype == CONVROT_BF16 ? launch_paged_typed<__bf16>(a, plan, partial, s) : launch_paged_typed<_Float16>(a, plan, partial, s);
}

void launch_attention(const convrot_attention_args& a, const PromptPlan& plan, float* partial, hipStream_t s)
{
    a.dtype == CONVROT_BF16 ? launch_prompt_typed<__bf16>(a, plan, partial, s) : launch_prompt_typed<_Float16>(a, plan, partial, s);
}

}  // namespace convrot

extern "C" {

int convrot_cache_write(const convrot_cache_args* args, void* stream)
{
    int rc = convrot_validate_cache_write(args);
    if (rc || args->tokens == 0) return rc;
    if ((rc = check_device())) return rc;
    launch_cache(*args, true, (hipStream_t)stream);
    return launched();
}

int convrot_cache_read(const convrot_cache_args* args, void* stream)
{
    int rc = convrot_validate_cache_read(args);
    if (rc || args->tokens == 0) return rc;
    if ((rc = check_device())) return rc;
    launch_cache(*args, false, (hipStream_t)stream);
    return launched();
}

int convrot_attention_paged(const convrot_attention_paged_args* args, void* workspace, size_t ws_bytes, void* stream)
{
    int rc = convrot_validate_attention_paged(args, workspace, ws_bytes);
    if (rc || args->batch == 0) return rc;
    if ((rc = check_device())) return rc;
    launch_attention_paged(*args, paged_plan(*args), (float*)workspace, (hipStream_t)stream);
    return launched();
}

int convrot_attention(const convrot_attention_args* args, void* workspace, size_t ws_bytes, void* stream)
{
    int rc = convrot_validate_attention(args, workspace, ws_bytes);
    if (rc || args->batch == 0 || args->q_tokens == 0) return rc;
    if ((rc = check_device())) return rc;
    launch_attention(*args, prompt_plan(*args), (float*)workspace, (hipStream_t)stream);
    return launched();
}

}  // extern "C"
