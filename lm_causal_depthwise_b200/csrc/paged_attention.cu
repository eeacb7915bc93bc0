// paged_attention.cu -- causal sliding-window attention of the new tokens over a paged 8-bit cache.
//
//   out[t, h] = sum_p softmax_p(scale * q[t, h] . k[p]) v[p],   pos_t - window < p <= pos_t
//
// with k[p], v[p] = code * scale of p's page and head.  Positions outside a row's range
// are never read or never weighted; a row without any key gives zeros.
#include "paged.cuh"

namespace rglru {
namespace {

using paged::Batch;

struct AttendArgs {
    Batch b;
    int window;
    float scale;
    const __nv_bfloat16 *q;
    const uint8_t *k, *v;
    const float *ks, *vs;
    __nv_bfloat16 *out;
};

// One CTA per (token, head, sequence): warps take every eighth key, lanes D / 32 channels.
template <int D>
__global__ void __launch_bounds__(256) rglru_paged_attention_kernel(const AttendArgs p)
{
    constexpr int kPer = D / 32;
    __shared__ float sm[8], sl[8], so[8][D];
    const Batch &b = p.b;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y, i = blockIdx.z;
    const paged::Seq s = paged::load_seq(b, i);
    for (int t = blockIdx.x; t < s.n; t += gridDim.x) {
        const int pos = s.ctx + t, kv = h / (b.H / b.Hkv);
        const size_t row = ((size_t)(s.row0 + t) * b.H + h) * D + lane * kPer;
        float q[kPer], o[kPer] = {}, m = -INFINITY, l = 0.f;
        for (int e = 0; e < kPer; ++e) q[e] = __bfloat162float(p.q[row + e]) * p.scale;
        for (int key = max(0, pos - p.window + 1) + warp; key <= pos; key += 8) {
            const int page = paged::load_page(b, i, key / b.page);
            if (page < 0) continue;
            const size_t at = (size_t)page * b.Hkv + kv;
            const size_t off = (at * b.page + key % b.page) * D + lane * kPer;
            float d = 0.f, x0, x1;
            for (int e = 0; e < kPer; e += 2) {
                e4m3::to_f32x2(*reinterpret_cast<const uint16_t *>(p.k + off + e), x0, x1);
                d = fmaf(q[e], x0, fmaf(q[e + 1], x1, d));
            }
            for (int w = 16; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
            d *= p.ks[at];
            const float m2 = fmaxf(m, d), r = m == -INFINITY ? 0.f : __expf(m - m2), w = __expf(d - m2);
            l = l * r + w;
            for (int e = 0; e < kPer; e += 2) {
                e4m3::to_f32x2(*reinterpret_cast<const uint16_t *>(p.v + off + e), x0, x1);
                o[e] = o[e] * r + w * x0 * p.vs[at];
                o[e + 1] = o[e + 1] * r + w * x1 * p.vs[at];
            }
            m = m2;
        }
        __syncthreads();
        if (lane == 0) sm[warp] = m, sl[warp] = l;
        for (int e = 0; e < kPer; ++e) so[warp][lane * kPer + e] = o[e];
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += 256) {
            float mm = -INFINITY, ll = 0.f, oo = 0.f;
            for (int w = 0; w < 8; ++w) mm = fmaxf(mm, sm[w]);
            for (int w = 0; w < 8; ++w) {
                if (sl[w] == 0.f) continue;
                const float r = __expf(sm[w] - mm);
                ll += sl[w] * r;
                oo += so[w][c] * r;
            }
            p.out[((size_t)(s.row0 + t) * b.H + h) * D + c] = __float2bfloat16_rn(ll == 0.f ? 0.f : oo / ll);
        }
    }
}

}  // namespace
}  // namespace rglru

using namespace rglru;

extern "C" {

RGLRU_API size_t rglru_paged_attention_workspace_size(int H, int Hkv, int head_dim)
{
    if (H < 1 || Hkv < 1 || H > 256 || Hkv > 64 || H % Hkv != 0 || (head_dim != 128 && head_dim != 256)) return 0;
    return kWsHeaderBytes;
}

RGLRU_API rglru_status rglru_paged_attention(int rows, int S, int H, int Hkv, int head_dim, int page_size,
                                             int num_pages, int max_pages, int max_new, int max_total, int window,
                                             float scale, const void *q, const int32_t *cu_tokens,
                                             const int32_t *ctx_len, const int32_t *block_table, const void *k_cache,
                                             const float *k_scale, const void *v_cache, const float *v_scale, void *out,
                                             void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    const AttendArgs p = {{rows, S, H, Hkv, head_dim, page_size, num_pages, max_pages, max_new, max_total, cu_tokens,
                           ctx_len, block_table, static_cast<WsHeader *>(workspace)},
                          window, scale, static_cast<const __nv_bfloat16 *>(q), static_cast<const uint8_t *>(k_cache),
                          static_cast<const uint8_t *>(v_cache), k_scale, v_scale, static_cast<__nv_bfloat16 *>(out)};
    const size_t need = rglru_paged_attention_workspace_size(H, Hkv, head_dim);
    const rglru_status c = paged::check_batch(p.b, k_cache, k_scale, v_cache, v_scale, workspace_bytes, need);
    if (c != RGLRU_OK) return c;
    if (!args::al16(q) || !args::al16(out) || window < 1 || !(scale > 0.f) || scale > 1e30f) return RGLRU_ERR_INVALID_ARG;
    const size_t pool = (size_t)num_pages * Hkv, act = (size_t)rows * H * head_dim * 2;
    const args::Span in[] = {args::span(q, act),
                             args::span(cu_tokens, ((size_t)S + 1) * 4),
                             args::span(ctx_len, (size_t)S * 4),
                             args::span(block_table, (size_t)S * max_pages * 4),
                             args::span(k_cache, pool * page_size * head_dim),
                             args::span(k_scale, pool * 4),
                             args::span(v_cache, pool * page_size * head_dim),
                             args::span(v_scale, pool * 4)};
    const args::Span so = args::span(out, act), sw = args::span(workspace, need);
    for (const args::Span &s : in)
        if (args::meet(so, s) || args::meet(sw, s)) return RGLRU_ERR_INVALID_ARG;
    if (args::meet(so, sw)) return RGLRU_ERR_INVALID_ARG;
    const dim3 grid(max_new < 65536 ? max_new : 65536, H, S);
    if (head_dim == 256)
        rglru_paged_attention_kernel<256><<<grid, 256, 0, stream>>>(p);
    else
        rglru_paged_attention_kernel<128><<<grid, 256, 0, stream>>>(p);
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
