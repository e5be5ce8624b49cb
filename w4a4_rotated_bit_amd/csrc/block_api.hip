// block_api.hip -- device entry points of the operators around a rotated
// linear: checks on the host, one launch on the caller's stream, no state.
#include <hip/hip_runtime.h>

#include "../../include/convrot.h"
#include "block_ops.h"
#include "internal.h"
#include "kernels.h"

using namespace convrot;

extern "C" {

int convrot_residual_norm(const convrot_residual_norm_args* args, void* stream)
{
    int rc = convrot_validate_residual_norm(args);
    if (rc || args->rows == 0) return rc;
    if ((rc = check_device())) return rc;
    launch_residual_norm(*args, (hipStream_t)stream);
    return launched();
}

int convrot_rope(const convrot_rope_args* args, void* stream)
{
    int rc = convrot_validate_rope(args);
    if (rc || args->batch == 0 || args->tokens == 0) return rc;
    if ((rc = check_device())) return rc;
    constexpr double kTurn = 6.283185307179586476925286766559;
    RopePlan plan{};
    for (int i = 0; i < args->pairs; ++i) {
        plan.turns[i] = args->freq_host[i] / kTurn;
        plan.axis[i] = (uint8_t)args->axis_host[i];
    }
    launch_rope(*args, plan, (hipStream_t)stream);
    return launched();
}

int convrot_linear_grouped(const convrot_grouped_args* args, void* stream)
{
    int rc = convrot_validate_linear_grouped(args);
    if (rc || args->M == 0 || args->N == 0) return rc;
    if ((rc = check_device())) return rc;
    launch_linear_grouped(*args, (hipStream_t)stream);
    return launched();
}

int convrot_quantize_weight_grouped(const void* W, int64_t N, int64_t K, int group, int dtype, uint8_t* codes,
                                    void* scales, uint8_t* zeros, void* stream)
{
    int rc = convrot_validate_quantize_weight_grouped(W, N, K, group, dtype, codes, scales, zeros);
    if (rc || N == 0) return rc;
    if ((rc = check_device())) return rc;
    launch_quantize_grouped(W, N, K, group, dtype, codes, scales, zeros, (hipStream_t)stream);
    return launched();
}

}  // extern "C"
