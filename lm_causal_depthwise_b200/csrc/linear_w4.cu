// linear_w4.cu -- projections of a few rows with 4-bit weights and group scales.
//
//   out[m, n] = sum_g s[n, g] * sum_{k in group g} (q[n, k] - 8) * x[m, k] + bias[n]
//
// q in 0..15, two to a byte along K (the even k in the low half), s in bf16, x in bf16 or in
// e4m3 with a scale for each group of channels; the weights' integers and x are exact operands, the inner sums and
// the scaled total are fp32, and the output is rounded to bf16 once.  Bound by the weight
// bytes: N K / 2, and 2 N K / group for the scales.
#include "e4m3.cuh"
#include "internal.h"

namespace rglru {
namespace {

constexpr int kMaxM = 64;

struct W4Args {
    int M, N, K, group, a_group;
    const void *A;
    const float *A_scale;
    const uint8_t *W;
    const __nv_bfloat16 *W_scale;
    const float *bias;
    __nv_bfloat16 *out;
};

// One warp per output feature; a lane takes 8 consecutive k at a time, for every row.
__global__ void __launch_bounds__(256) rglru_linear_w4_kernel(const W4Args p)
{
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (n >= p.N) return;
    for (int m = 0; m < p.M; ++m) {
        float acc = 0.f;
        for (int k = lane * 8; k < p.K; k += 256) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(p.W + ((size_t)n * p.K + k) / 2);
            float part = 0.f;
            for (int e = 0; e < 8; ++e) {
                float x;
                if (p.A_scale == nullptr) {
                    x = __bfloat162float(static_cast<const __nv_bfloat16 *>(p.A)[(size_t)m * p.K + k + e]);
                } else {
                    float hi;
                    e4m3::to_f32x2(static_cast<const uint8_t *>(p.A)[(size_t)m * p.K + k + e], x, hi);
                    x *= p.A_scale[(size_t)m * (p.K / p.a_group) + (k + e) / p.a_group];
                }
                part = fmaf((float)((int)((w >> (4 * e)) & 15u) - 8), x, part);
            }
            acc = fmaf(part, __bfloat162float(p.W_scale[(size_t)n * (p.K / p.group) + k / p.group]), acc);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (lane == 0)
            p.out[(size_t)m * p.N + n] = __float2bfloat16_rn(acc + (p.bias != nullptr ? p.bias[n] : 0.f));
    }
}

}  // namespace
}  // namespace rglru

using namespace rglru;

extern "C" RGLRU_API rglru_status rglru_linear_w4(int M, int N, int K, int group, const void *A, const float *A_scale,
                                                  int a_group, const void *W, const void *W_scale, const float *bias,
                                                  void *out, cudaStream_t stream)
{
    if (M < 1 || N < 1 || K < 1) return RGLRU_ERR_INVALID_ARG;
    if (M > kMaxM || N > (1 << 20) || K > (1 << 20)) return RGLRU_ERR_UNSUPPORTED;
    if ((group != 32 && group != 64 && group != 128) || K % group != 0) return RGLRU_ERR_UNSUPPORTED;
    if (A_scale != nullptr &&
        ((a_group != 32 && a_group != 64 && a_group != 128 && a_group != 256) || K % a_group != 0))
        return RGLRU_ERR_UNSUPPORTED;
    if (!args::al16(A) || !args::al16(W) || !args::al16(W_scale) || !args::al16(out)) return RGLRU_ERR_INVALID_ARG;
    if ((A_scale != nullptr && !args::al16(A_scale)) || (bias != nullptr && !args::al16(bias)))
        return RGLRU_ERR_INVALID_ARG;
    const size_t mk = (size_t)M * K, nk = (size_t)N * K;
    if (!args::clear(args::span(out, 2 * (size_t)M * N),
                     {args::span(A, A_scale ? mk : 2 * mk), args::span(A_scale, A_scale ? mk / a_group * 4 : 0),
                      args::span(W, nk / 2), args::span(W_scale, nk / group * 2),
                      args::span(bias, bias ? 4 * (size_t)N : 0)}))
        return RGLRU_ERR_INVALID_ARG;
    const W4Args p = {M, N, K, group, A_scale ? a_group : 0, A, A_scale, static_cast<const uint8_t *>(W),
                      static_cast<const __nv_bfloat16 *>(W_scale), bias, static_cast<__nv_bfloat16 *>(out)};
    rglru_linear_w4_kernel<<<(N + 7) / 8, 256, 0, stream>>>(p);
    return cuda_status(cudaGetLastError());
}
