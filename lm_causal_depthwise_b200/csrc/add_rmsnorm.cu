// add_rmsnorm.cu -- the residual's addition and the RMSNorm that follows it, in one pass over the row.
//
//   h = bf16(x + residual)                      (the new residual stream)
//   y = h * rsqrt(mean_n(h^2) + eps) * weight   as bf16, or as e4m3 with one power-of-two
//                                               scale for each group of channels (e4m3.cuh)
//
// The decoder layer adds the temporal block's output to its input and normalises the sum (channel_pre_norm).  In one
// kernel the sum is read from registers instead of from memory: 8 bytes per element with a bf16 output (7 with an 8-bit
// one) against 10 for an addition and rglru_rmsnorm.  h is rounded to bf16 before the norm, so that the result is what
// the two calls give.  The sum of squares, the mean and the scaled row are fp32.  Memory bound: 32768 x 2560 takes
// 106 us, 6.3 TB/s; a few rows take the launch (4 x 2560: 9 us, 4 on the device).
#include "e4m3.cuh"
#include "internal.h"

namespace rglru {
namespace {

constexpr int kMaxN = 16384;
constexpr int kSms = 148;

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A CTA walks over rows, VPT vectors of 8 channels a thread: the weight stays in registers, and the next row's loads
// are issued before this row's sum is known.  group == 0: bf16 output.
template <int VPT, bool kE4m3, bool kRes>
__global__ void __launch_bounds__(512)
rglru_add_rmsnorm_kernel(int M, int N, int group, const uint4 *__restrict__ x, const uint4 *res,
                         const float4 *__restrict__ w, float eps, uint4 *res_out, void *__restrict__ out,
                         float *__restrict__ out_scale)
{
    __shared__ float part[2][16];
    const int tid = threadIdx.x, nvec = N / 8;
    float4 wv[VPT][2];
    uint4 v[VPT], r[VPT];
    auto load = [&](int row) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = k * blockDim.x + tid;
            v[k] = make_uint4(0, 0, 0, 0);
            if (kRes) r[k] = make_uint4(0, 0, 0, 0);
            if (i < nvec) {
                v[k] = __ldcs(x + (size_t)row * nvec + i);
                if (kRes) r[k] = __ldcs(res + (size_t)row * nvec + i);
            }
        }
    };
    load(blockIdx.x);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int i = k * blockDim.x + tid;
        wv[k][0] = i < nvec ? w[2 * i] : make_float4(0, 0, 0, 0);
        wv[k][1] = i < nvec ? w[2 * i + 1] : make_float4(0, 0, 0, 0);
    }
    int turn = 0;
    const int last = M - (int)gridDim.x;  // rows from here on are their CTA's last: the next one may lie past 2^31
    for (int row = blockIdx.x;; row += gridDim.x, turn ^= 1) {
        uint4 h[VPT];
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = k * blockDim.x + tid;
            h[k] = v[k];
            if (kRes) {
                h[k].x = bf_pack(bf_lo(v[k].x) + bf_lo(r[k].x), bf_hi(v[k].x) + bf_hi(r[k].x));
                h[k].y = bf_pack(bf_lo(v[k].y) + bf_lo(r[k].y), bf_hi(v[k].y) + bf_hi(r[k].y));
                h[k].z = bf_pack(bf_lo(v[k].z) + bf_lo(r[k].z), bf_hi(v[k].z) + bf_hi(r[k].z));
                h[k].w = bf_pack(bf_lo(v[k].w) + bf_lo(r[k].w), bf_hi(v[k].w) + bf_hi(r[k].w));
                if (i < nvec) res_out[(size_t)row * nvec + i] = h[k];
            }
            const uint32_t q[4] = {h[k].x, h[k].y, h[k].z, h[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ss = fmaf(bf_lo(q[e]), bf_lo(q[e]), ss);
                ss = fmaf(bf_hi(q[e]), bf_hi(q[e]), ss);
            }
        }
        if (row < last) load(row + gridDim.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        // two turns: a row's sums are read while the next row's are written
        if ((tid & 31) == 0) part[turn][tid >> 5] = ss;
        __syncthreads();
        ss = 0.f;
        for (int k = 0; k < (int)blockDim.x / 32; ++k) ss += part[turn][k];
        const float inv = rsqrtf(ss / (float)N + eps);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int i = k * blockDim.x + tid;
            const bool in = i < nvec;
            const float4 wa = wv[k][0], wb = wv[k][1];
            const float y[8] = {bf_lo(h[k].x) * inv * wa.x, bf_hi(h[k].x) * inv * wa.y, bf_lo(h[k].y) * inv * wa.z,
                                bf_hi(h[k].y) * inv * wa.w, bf_lo(h[k].z) * inv * wb.x, bf_hi(h[k].z) * inv * wb.y,
                                bf_lo(h[k].w) * inv * wb.z, bf_hi(h[k].w) * inv * wb.w};
            if (!kE4m3) {
                if (in)
                    static_cast<uint4 *>(out)[(size_t)row * nvec + i] =
                        make_uint4(bf_pack(y[0], y[1]), bf_pack(y[2], y[3]), bf_pack(y[4], y[5]), bf_pack(y[6], y[7]));
            } else {
                // a group is group / 8 (4 to 32, a power of two) adjacent lanes of one warp
                float amax = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));
                for (int o = group / 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const float s = e4m3::scale_of(amax), f = e4m3::inverse(s);
                if (in) {
                    static_cast<uint2 *>(out)[(size_t)row * nvec + i] =
                        make_uint2(e4m3::pack4(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                                   e4m3::pack4(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
                    if (i % (group / 8) == 0) out_scale[(size_t)row * (N / group) + i / (group / 8)] = s;
                }
            }
        }
        if (row >= last) break;
    }
}

template <int VPT, bool kE4m3>
rglru_status launch_vpt(int M, int N, int group, const void *x, const void *res, const float *w, float eps,
                        void *res_out, void *out, float *out_scale, cudaStream_t stream)
{
    const int threads = ((N / 8 + VPT - 1) / VPT + 31) / 32 * 32;
    // resident threads: 2048 an SM fill it, but the bf16 form with one vector a thread runs better with 1536 (below)
    const int most = kSms * ((VPT == 1 ? 1536 : 2048) / threads);
    const int grid = M < most ? M : most;
    const auto *xv = static_cast<const uint4 *>(x), *rv = static_cast<const uint4 *>(res);
    const auto *wv = reinterpret_cast<const float4 *>(w);
    auto *ro = static_cast<uint4 *>(res_out);
    if (res != nullptr)
        rglru_add_rmsnorm_kernel<VPT, kE4m3, true>
            <<<grid, threads, 0, stream>>>(M, N, group, xv, rv, wv, eps, ro, out, out_scale);
    else
        rglru_add_rmsnorm_kernel<VPT, kE4m3, false>
            <<<grid, threads, 0, stream>>>(M, N, group, xv, rv, wv, eps, ro, out, out_scale);
    return cuda_status(cudaGetLastError());
}

template <bool kE4m3>
rglru_status launch(int M, int N, int group, const void *x, const void *res, const float *w, float eps, void *res_out,
                    void *out, float *out_scale, cudaStream_t stream)
{
    // 32768 x 2560, bf16: one vector a thread and 1536 threads an SM 106 us (97% of the measured bandwidth with the
    // launch), 2048 threads 117, two vectors 113.  The e4m3 form has the maxima's shuffles to hide: two vectors and 2048
    // threads 111 us, one vector 123 to 131; 4099 x 4096 25 us against 31.
    if constexpr (!kE4m3)
        if (N <= 4096) return launch_vpt<1, kE4m3>(M, N, group, x, res, w, eps, res_out, out, out_scale, stream);
    if (N <= 2 * 4096) return launch_vpt<2, kE4m3>(M, N, group, x, res, w, eps, res_out, out, out_scale, stream);
    return launch_vpt<4, kE4m3>(M, N, group, x, res, w, eps, res_out, out, out_scale, stream);
}

rglru_status check(int M, int N, int group, const void *x, const void *res, const float *w, float eps,
                   const void *res_out, const void *out, const float *out_scale)
{
    if (M < 1 || N < 8 || !(eps > 0.f)) return RGLRU_ERR_INVALID_ARG;
    if (N % 8 != 0 || N > kMaxN) return RGLRU_ERR_UNSUPPORTED;
    if (group != 0 && ((group != 32 && group != 64 && group != 128 && group != 256) || N % group != 0))
        return RGLRU_ERR_UNSUPPORTED;
    if (!args::al16(x) || !args::al16(w) || !args::al16(out) || (group != 0 && !args::al16(out_scale)))
        return RGLRU_ERR_INVALID_ARG;
    if ((res == nullptr) != (res_out == nullptr)) return RGLRU_ERR_INVALID_ARG;
    if (res != nullptr && (!args::al16(res) || !args::al16(res_out))) return RGLRU_ERR_INVALID_ARG;
    const size_t n = (size_t)M * N;
    const args::Span sx = args::span(x, 2 * n), sr = args::span(res, res ? 2 * n : 0), sw = args::span(w, 4 * (size_t)N);
    const args::Span so = args::span(out, group ? n : 2 * n), sh = args::span(res_out, res ? 2 * n : 0);
    const args::Span ss = args::span(out_scale, group ? n / group * 4 : 0);
    if (!args::clear(so, {sx, sr, sw, sh, ss}) || !args::clear(ss, {sx, sr, sw, sh})) return RGLRU_ERR_INVALID_ARG;
    // each element of the new residual is written by the thread that read x and residual there
    if (args::meet(sh, sw) || (args::meet(sh, sx) && res_out != x) || (args::meet(sh, sr) && res_out != res))
        return RGLRU_ERR_INVALID_ARG;
    return RGLRU_OK;
}

}  // namespace
}  // namespace rglru

using namespace rglru;

extern "C" {

RGLRU_API rglru_status rglru_add_rmsnorm(int M, int N, const void *x, const void *residual, const float *weight,
                                         float eps, void *residual_out, void *out, cudaStream_t stream)
{
    const rglru_status c = check(M, N, 0, x, residual, weight, eps, residual_out, out, nullptr);
    if (c != RGLRU_OK) return c;
    return launch<false>(M, N, 0, x, residual, weight, eps, residual_out, out, nullptr, stream);
}

RGLRU_API rglru_status rglru_add_rmsnorm_e4m3(int M, int N, int group, const void *x, const void *residual,
                                              const float *weight, float eps, void *residual_out, void *out,
                                              float *out_scale, cudaStream_t stream)
{
    if (group == 0) return RGLRU_ERR_UNSUPPORTED;
    const rglru_status c = check(M, N, group, x, residual, weight, eps, residual_out, out, out_scale);
    if (c != RGLRU_OK) return c;
    return launch<true>(M, N, group, x, residual, weight, eps, residual_out, out, out_scale, stream);
}

}  // extern "C"
