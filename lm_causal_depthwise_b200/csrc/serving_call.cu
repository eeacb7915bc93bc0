// serving_call.cu -- the serving calls with their parameters in a block.
//
// An interpreter converts each argument of a foreign call by itself (ctypes: 0.25 us an argument, 22 of them for
// rglru_paged_append), and packs a struct in one call.  Host code only, and with it the serving operators' test hook.
#include "internal.h"

thread_local int rglru::debug_withheld = 0;

extern "C" RGLRU_API rglru_status rglru_debug_withhold(int unit)
{
    if (unit < -1) return RGLRU_ERR_INVALID_ARG;
    rglru::debug_withheld = unit + 1;
    return RGLRU_OK;
}

extern "C" RGLRU_API rglru_status rglru_serving_call(rglru_call call, const void *args)
{
    if (args == nullptr) return RGLRU_ERR_INVALID_ARG;
    switch (call) {
    case RGLRU_CALL_ADD_RMSNORM: {
        const auto &a = *static_cast<const rglru_add_rmsnorm_args *>(args);
        return rglru_add_rmsnorm(a.M, a.N, a.x, a.residual, a.weight, a.eps, a.residual_out, a.out, a.stream);
    }
    case RGLRU_CALL_ADD_RMSNORM_E4M3: {
        const auto &a = *static_cast<const rglru_add_rmsnorm_e4m3_args *>(args);
        return rglru_add_rmsnorm_e4m3(a.M, a.N, a.group, a.x, a.residual, a.weight, a.eps, a.residual_out, a.out,
                                      a.out_scale, a.stream);
    }
    case RGLRU_CALL_LINEAR_W4: {
        const auto &a = *static_cast<const rglru_linear_w4_args *>(args);
        return rglru_linear_w4(a.M, a.N, a.K, a.group, a.A, a.A_scale, a.a_group, a.W, a.W_scale, a.bias, a.out,
                               a.stream);
    }
    case RGLRU_CALL_PAGED_APPEND: {
        const auto &a = *static_cast<const rglru_paged_append_args *>(args);
        return rglru_paged_append(a.rows, a.S, a.H, a.Hkv, a.head_dim, a.page_size, a.num_pages, a.max_pages, a.max_new,
                                  a.max_total, a.qkv, a.cu_tokens, a.ctx_len, a.block_table, a.rope_base, a.q_out,
                                  a.k_cache, a.k_scale, a.v_cache, a.v_scale, a.workspace, a.workspace_bytes, a.stream);
    }
    case RGLRU_CALL_PAGED_ATTENTION: {
        const auto &a = *static_cast<const rglru_paged_attention_args *>(args);
        return rglru_paged_attention(a.rows, a.S, a.H, a.Hkv, a.head_dim, a.page_size, a.num_pages, a.max_pages,
                                     a.max_new, a.max_total, a.window, a.scale, a.q, a.cu_tokens, a.ctx_len,
                                     a.block_table, a.k_cache, a.k_scale, a.v_cache, a.v_scale, a.out, a.workspace,
                                     a.workspace_bytes, a.stream);
    }
    }
    return RGLRU_ERR_INVALID_ARG;
}
