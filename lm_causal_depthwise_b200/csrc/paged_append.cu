// paged_append.cu -- the new tokens' keys and values into a paged 8-bit cache, rotated on the way.
//
// RoPE turns the pairs (x[i], x[i + D/2]) of the query heads and the keys by
// position * base^(-2i/D); q is written bf16, k and v as e4m3 codes.  A page's
// scale covers all its slots: the run of tokens that enters a page at its first slot sets it from
// its own largest magnitude; a run that enters later keeps the larger of the
// page's scale and its own, and when that raised the scale the older slots are moved to it (an exponent shift,
// rounded only where it underflows).
//
// Memory bound: 2 (H + 2 Hkv) D bytes read and 2 H D + 2 Hkv D written per token.  A CTA owns one
// page of one head, so that the page's maximum never leaves it: the run's values stay in registers
// between the maximum and the rounding.  The query heads need no maximum; other CTAs take 16 tokens and all
// their heads, which share one set of angles.
#include "paged.cuh"

namespace rglru {
namespace {

using paged::Batch;

constexpr int kThreads = 256;
constexpr int kQTokens = 16;  // tokens of a query CTA: their sines and cosines fill 16 KB of shared memory

struct AppendArgs {
    Batch b;
    const __nv_bfloat16 *qkv;
    __nv_bfloat16 *q_out;
    uint8_t *k, *v;
    float *ks, *vs;
    double log2_base;
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8])
{
    f[0] = bf_lo(v.x), f[1] = bf_hi(v.x), f[2] = bf_lo(v.y), f[3] = bf_hi(v.y);
    f[4] = bf_lo(v.z), f[5] = bf_hi(v.z), f[6] = bf_lo(v.w), f[7] = bf_hi(v.w);
}

// base^(-2i/D) / (2 pi) as turns per position, for every pair i
template <int D>
__device__ __forceinline__ void turns_table(double *t, double log2_base)
{
    for (int i = threadIdx.x; i < D / 2; i += kThreads)
        t[i] = exp2(-(double)i * (2.0 / D) * log2_base) * 0.15915494309189535;
    __syncthreads();
}
// the angle is reduced to a turn in fp64: positions past 2^20 keep it to 1e-7
__device__ __forceinline__ float2 angle(double turns_per_pos, int pos)
{
    double t = (double)pos * turns_per_pos;
    t -= rint(t);
    float s, c;
    sincospif((float)(2.0 * t), &s, &c);
    return make_float2(c, s);
}

// D channels a head, NP passes of kThreads / (D / 16) page rows; a thread holds the channels
// c .. c + 7 and c + D/2 .. c + D/2 + 7 of a row.
template <int D, int NP>
__global__ void __launch_bounds__(kThreads) rglru_paged_append_kernel(const AppendArgs p)
{
    constexpr int kCols = D / 16, kRows = kThreads / kCols, kHalf = D / 2;
    __shared__ double turns[kHalf];
    __shared__ float2 cs[kQTokens][kHalf];
    __shared__ float part[kThreads / 32];
    const Batch &b = p.b;
    const int tid = threadIdx.x, role = blockIdx.z;
    const paged::Seq s = paged::load_seq(b, blockIdx.y);
    if (s.n == 0) return;
    const int ps = b.page, width = (b.H + 2 * b.Hkv) * D;
    // this CTA's page of the run, and its slots [lo, hi) in it
    const int j = s.ctx / ps + blockIdx.x;
    const long long base = (long long)j * ps;
    const int lo = (int)max(0LL, s.ctx - base), hi = (int)min((long long)ps, (long long)s.ctx + s.n - base);
    if (hi <= lo) return;
    const long long tok0 = s.row0 + (base - s.ctx);  // row of slot 0 (slots before lo have none)

    if (role >= 2 * b.Hkv) {  // ------------------------------------------------ query heads of 16 tokens
        const int a = max(lo, (role - 2 * b.Hkv) * kQTokens), e = min(hi, (role - 2 * b.Hkv + 1) * kQTokens);
        if (e <= a) return;
        turns_table<D>(turns, p.log2_base);
        for (int i = tid; i < (e - a) * kHalf; i += kThreads)
            cs[i / kHalf][i % kHalf] = angle(turns[i % kHalf], (int)(base + a + i / kHalf));
        __syncthreads();
        for (int i = tid; i < (e - a) * b.H * kCols; i += kThreads) {
            const int t = i / (b.H * kCols), c = i % kCols * 8;
            const int head = i / kCols % b.H;
            const size_t row = (size_t)(tok0 + a + t);
            const __nv_bfloat16 *src = p.qkv + row * width + head * D + c;
            float x1[8], x2[8];
            unpack8(*reinterpret_cast<const uint4 *>(src), x1);
            unpack8(*reinterpret_cast<const uint4 *>(src + kHalf), x2);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float2 r = cs[t][c + q];
                const float y1 = x1[q] * r.x - x2[q] * r.y, y2 = x2[q] * r.x + x1[q] * r.y;
                x1[q] = y1, x2[q] = y2;
            }
            __nv_bfloat16 *dst = p.q_out + row * ((size_t)b.H * D) + head * D + c;
            *reinterpret_cast<uint4 *>(dst) =
                make_uint4(bf_pack(x1[0], x1[1]), bf_pack(x1[2], x1[3]), bf_pack(x1[4], x1[5]), bf_pack(x1[6], x1[7]));
            *reinterpret_cast<uint4 *>(dst + kHalf) =
                make_uint4(bf_pack(x2[0], x2[1]), bf_pack(x2[2], x2[3]), bf_pack(x2[4], x2[5]), bf_pack(x2[6], x2[7]));
        }
        return;
    }

    // --------------------------------------------------------------------------- one page of a key or value head
    const bool is_k = role < b.Hkv;
    const int head = is_k ? role : role - b.Hkv;
    const int page = paged::load_page(b, blockIdx.y, j);
    if (page < 0) return;
    uint8_t *codes = (is_k ? p.k : p.v) + ((size_t)page * b.Hkv + head) * ps * D;
    float *scale = (is_k ? p.ks : p.vs) + (size_t)page * b.Hkv + head;
    const int r0 = tid / kCols, c = tid % kCols * 8;
    if (is_k) turns_table<D>(turns, p.log2_base);
    float x[NP][16];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int slot = k * kRows + r0;
        float x1[8] = {}, x2[8] = {};
        if (slot >= lo && slot < hi) {
            const __nv_bfloat16 *src = p.qkv + (size_t)(tok0 + slot) * width + (b.H + role) * D + c;
            unpack8(*reinterpret_cast<const uint4 *>(src), x1);
            unpack8(*reinterpret_cast<const uint4 *>(src + kHalf), x2);
            if (is_k) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float2 r = angle(turns[c + q], (int)(base + slot));
                    const float y1 = x1[q] * r.x - x2[q] * r.y, y2 = x2[q] * r.x + x1[q] * r.y;
                    x1[q] = y1, x2[q] = y2;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            x[k][q] = x1[q], x[k][8 + q] = x2[q];
            amax = fmaxf(amax, fmaxf(fabsf(x1[q]), fabsf(x2[q])));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) part[tid >> 5] = amax;
    const float old = lo > 0 ? *scale : 0.f;
    __syncthreads();  // also: every thread has read the old scale
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) amax = fmaxf(amax, part[k]);
    const float s_new = fmaxf(old, e4m3::scale_of(amax));
    const float inv = 1.f / s_new;
    if (tid == 0) *scale = s_new;
    if (lo > 0 && s_new != old) {  // the older slots to the larger scale, 16 codes a thread
        const float f = old / s_new;
        for (int i = tid; i < lo * D / 16; i += kThreads) {
            uint4 v = reinterpret_cast<uint4 *>(codes)[i];
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float f0, f1, f2, f3;
                e4m3::to_f32x2(w[q] & 0xffffu, f0, f1);
                e4m3::to_f32x2(w[q] >> 16, f2, f3);
                w[q] = e4m3::pack4(f0 * f, f1 * f, f2 * f, f3 * f);
            }
            reinterpret_cast<uint4 *>(codes)[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int slot = k * kRows + r0;
        if (slot >= lo && slot < hi) {
            uint8_t *dst = codes + slot * D + c;
            float(&y)[16] = x[k];
            *reinterpret_cast<uint2 *>(dst) =
                make_uint2(e4m3::pack4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                           e4m3::pack4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
            *reinterpret_cast<uint2 *>(dst + kHalf) =
                make_uint2(e4m3::pack4(y[8] * inv, y[9] * inv, y[10] * inv, y[11] * inv),
                           e4m3::pack4(y[12] * inv, y[13] * inv, y[14] * inv, y[15] * inv));
        }
    }
}

}  // namespace

rglru_status paged::check_batch(const Batch &b, const void *k, const float *ks, const void *v, const float *vs,
                                size_t ws_bytes, size_t ws_need)
{
    if (b.rows < 1 || b.S < 1 || b.H < 1 || b.Hkv < 1 || b.num_pages < 1 || b.max_pages < 1 || b.max_new < 1 ||
        b.max_total < b.max_new)
        return RGLRU_ERR_INVALID_ARG;
    if (b.D != 128 && b.D != 256) return RGLRU_ERR_UNSUPPORTED;
    if (b.page != 16 && b.page != 32 && b.page != 64 && b.page != 128) return RGLRU_ERR_UNSUPPORTED;
    if (b.S > 65535 || b.H > 256 || b.Hkv > 64 || b.H % b.Hkv != 0 || b.rows > (1 << 24)) return RGLRU_ERR_UNSUPPORTED;
    if (b.max_total > (1 << 30) || b.num_pages > (1 << 28) || b.max_pages > (1 << 26)) return RGLRU_ERR_UNSUPPORTED;
    // every position below max_total has its entry in the table
    if ((int64_t)b.max_pages * b.page < b.max_total) return RGLRU_ERR_INVALID_ARG;
    for (const void *q : {static_cast<const void *>(b.cu), static_cast<const void *>(b.ctx),
                          static_cast<const void *>(b.table), k, static_cast<const void *>(ks), v,
                          static_cast<const void *>(vs)})
        if (!args::al16(q)) return RGLRU_ERR_INVALID_ARG;
    if (!args::al16(b.ws) || ws_bytes < ws_need) return RGLRU_ERR_WORKSPACE;
    return RGLRU_OK;
}

}  // namespace rglru

using namespace rglru;

extern "C" RGLRU_API rglru_status rglru_paged_append(
    int rows, int S, int H, int Hkv, int head_dim, int page_size, int num_pages, int max_pages, int max_new,
    int max_total, const void *qkv, const int32_t *cu_tokens, const int32_t *ctx_len, const int32_t *block_table,
    float rope_base, void *q_out, void *k_cache, float *k_scale, void *v_cache, float *v_scale, void *workspace,
    size_t workspace_bytes, cudaStream_t stream)
{
    AppendArgs p = {{rows, S, H, Hkv, head_dim, page_size, num_pages, max_pages, max_new, max_total, cu_tokens, ctx_len,
                     block_table, static_cast<WsHeader *>(workspace)},
                    static_cast<const __nv_bfloat16 *>(qkv), static_cast<__nv_bfloat16 *>(q_out),
                    static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), k_scale, v_scale, 0.0};
    const rglru_status c = paged::check_batch(p.b, k_cache, k_scale, v_cache, v_scale, workspace_bytes, kWsHeaderBytes);
    if (c != RGLRU_OK) return c;
    if (!args::al16(qkv) || !args::al16(q_out) || !(rope_base > 1.f) || rope_base > 1e30f) return RGLRU_ERR_INVALID_ARG;
    p.log2_base = log2((double)rope_base);
    const size_t pool = (size_t)num_pages * Hkv;
    const args::Span in[] = {args::span(qkv, (size_t)rows * (H + 2 * Hkv) * head_dim * 2),
                             args::span(cu_tokens, ((size_t)S + 1) * 4), args::span(ctx_len, (size_t)S * 4),
                             args::span(block_table, (size_t)S * max_pages * 4)};
    const args::Span out[] = {args::span(q_out, (size_t)rows * H * head_dim * 2),
                              args::span(k_cache, pool * page_size * head_dim), args::span(k_scale, pool * 4),
                              args::span(v_cache, pool * page_size * head_dim), args::span(v_scale, pool * 4),
                              args::span(workspace, kWsHeaderBytes)};
    for (size_t i = 0; i < 6; ++i) {
        if (!args::clear(out[i], {in[0], in[1], in[2], in[3]})) return RGLRU_ERR_INVALID_ARG;
        for (size_t k = i + 1; k < 6; ++k)
            if (args::meet(out[i], out[k])) return RGLRU_ERR_INVALID_ARG;
    }
    // pages that a run of max_new tokens can touch, whatever slot it enters at
    const int runs = (max_new + page_size - 2) / page_size + 1;
    const dim3 grid(runs, S, 2 * Hkv + (page_size + kQTokens - 1) / kQTokens);
    const int np = page_size * (head_dim / 16) / kThreads;
#define RGLRU_APPEND(D_, NP_) rglru_paged_append_kernel<D_, NP_><<<grid, kThreads, 0, stream>>>(p)
    if (head_dim == 256) {
        if (np <= 1) RGLRU_APPEND(256, 1);
        else if (np == 2) RGLRU_APPEND(256, 2);
        else if (np == 4) RGLRU_APPEND(256, 4);
        else RGLRU_APPEND(256, 8);
    } else {
        if (np <= 1) RGLRU_APPEND(128, 1);
        else if (np == 2) RGLRU_APPEND(128, 2);
        else RGLRU_APPEND(128, 4);
    }
#undef RGLRU_APPEND
    return cuda_status(cudaGetLastError());
}
