// spec_prompt_attention: the entry points.
#include "prompt.cuh"

#include <cmath>

#include "host_util.h"

namespace sv {

__global__ void __launch_bounds__(32) no_rows_kernel(const PromptParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    PromptWalk w;
    w.start();
    prompt_statuses(p, w, nullptr);   // no rows, no waits
}

}  // namespace sv

using namespace sv;

extern "C" int spec_prompt_attention(const spec_prompt_args* a, void* stream) {
    clear_error();
    const char* const who = "spec_prompt_attention";
    if (a == nullptr) return set_error(SPEC_ERR_ARG, "%s: args is NULL", who);
    if (!valid_dtype(a->dtype)) return set_error(SPEC_ERR_DTYPE, "%s: dtype %d", who, a->dtype);
    if (a->B < 0 || a->B > SPEC_MAX_STREAMS) return set_error(SPEC_ERR_SHAPE, "%s: B = %d", who, a->B);
    if (a->Hkv < 1 || a->Hq < 1 || a->Hq > 1024 || a->Hq % a->Hkv != 0 || a->Hq / a->Hkv > 128)
        return set_error(SPEC_ERR_SHAPE, "%s: Hq = %d, Hkv = %d", who, a->Hq, a->Hkv);
    if (a->D < 8 || a->D > (a->dtype == SPEC_DTYPE_F32 ? 128 : SPEC_MAX_HEAD) || a->D % 8 != 0)
        return set_error(SPEC_ERR_SHAPE, "%s: D = %d", who, a->D);
    if (a->window < 0 || a->sinks < 0) return set_error(SPEC_ERR_SHAPE, "%s: window = %d, sinks = %d", who, a->window, a->sinks);
    if (a->q_row_stride < (int64_t)a->Hq * a->D || a->k_row_stride < (int64_t)a->Hkv * a->D || a->v_row_stride < (int64_t)a->Hkv * a->D)
        return set_error(SPEC_ERR_SHAPE, "%s: a row stride is below its heads * D", who);
    if (a->rows < 0 || a->rows > INT32_MAX || (a->cu_rows == nullptr && a->B > 0 && a->rows % a->B != 0))
        return set_error(SPEC_ERR_SHAPE, "%s: rows = %lld", who, (long long)a->rows);
    if (a->B == 0) return SPEC_OK;
    if (a->status == nullptr || (a->rows > 0 && (a->q == nullptr || a->k == nullptr || a->v == nullptr || a->out == nullptr)))
        return set_error(SPEC_ERR_ARG, "%s: a required pointer is NULL", who);
    const int es = a->dtype == SPEC_DTYPE_F32 ? 4 : 2;
    if (((uintptr_t)a->q | (uintptr_t)a->k | (uintptr_t)a->v | (uintptr_t)a->out | (uintptr_t)(a->q_row_stride * es) |
         (uintptr_t)(a->k_row_stride * es) | (uintptr_t)(a->v_row_stride * es)) & 15)
        return set_error(SPEC_ERR_ARG, "%s: q, k, v, out or a row stride is not a multiple of 16 bytes", who);
    if (!std::isfinite(a->scale) || !std::isfinite((float)((double)a->scale * kLog2e)))   // scores are taken to base 2
        return set_error(SPEC_ERR_ARG, "%s: scale is not finite", who);
    int sms = 0;
    const int rc = sm_count(&sms, who);
    if (rc != SPEC_OK) return rc;
    PromptParams p = {};
    p.a = *a;
    p.G = a->Hq / a->Hkv;
    p.by_G = divisor(p.G);
    p.group = 128 / p.G;
    p.piece = p.group;
    p.rows_each = (int)(a->rows / a->B);
    // the kernels negate Q for a negative scale, and multiply masked scores of -inf by it
    p.scale_log2 = a->scale == 0.f ? 1e-30f : std::fabs((float)((double)a->scale * kLog2e));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->rows == 0 ? launch_after(no_rows_kernel, dim3((unsigned)((a->B + 31) / 32)), dim3(32), 0, s, p)
                          : a->dtype == SPEC_DTYPE_BF16 ? launch_prompt_tc(p, sms, s)
                                                        : launch_prompt_f32(p, sms, s);
    return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, who);
}

extern "C" int spec_prompt_mark_timeout(int32_t marked, void* stream) {
    clear_error();
    if ((marked & ~1) != 0) return set_error(SPEC_ERR_ARG, "spec_prompt_mark_timeout: marked = %d", marked);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = mark_prompt_tc(marked, s);
    if (e == cudaSuccess) e = mark_prompt_f32(marked, s);
    return e == cudaSuccess ? SPEC_OK : set_cuda_error(e, "spec_prompt_mark_timeout");
}
