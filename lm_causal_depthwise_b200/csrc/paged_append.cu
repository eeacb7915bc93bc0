// paged_append.cu -- the new tokens' keys and values into a paged 8-bit cache, rotated on the way.
//
// RoPE turns the pairs (x[i], x[i + D/2]) of the query heads and the keys by position * base^(-2i/D); q is written
// bf16, k and v as e4m3 codes.  A page's scale covers all its slots: the run of tokens that enters a page at its first
// slot sets it from its own largest magnitude; a run that enters later keeps the larger of the page's scale and its
// own, and when that raised the scale the older slots are moved to it (an exponent shift, rounded only where it
// underflows).
//
// Memory bound: 2 (H + 2 Hkv) D bytes read and 2 H D + 2 Hkv D written per token.  A CTA owns one page of one key or
// value head, so that the page's maximum never leaves it: the run's values stay in registers between the maximum and
// the rounding (computed a second time instead, they spilled: 35.9 us against 18.5 for 37 runs of up to 300 tokens).
// The query heads need no maximum: other CTAs take a token and 16 channels a thread, and up to five heads with the
// same sines and cosines, all of their loads in flight at once.
//
// Angles: position times frequency is a fixed-point product modulo one turn.  The frequency is held as turns per
// position in units of 2^-64, so the product's low 64 bits are the fraction of a turn, whose upper 32 bits (2^-32 of a
// turn) are kept: no position loses bits, and no double is needed.  Sine and cosine are the hardware's (absolute error
// 2^-21 on [-pi, pi]), far below the roundings to bf16 (2^-9) and e4m3 (2^-4) that follow.
//
// Measured: 8 prompts of up to 4096 tokens, 10 heads of 256: 35.1 us with the launch, 4.8 TB/s; 37 runs of up to 300
// tokens, 16 heads of 128 on 4, pages of 16: 18.5 us.
#include "paged.cuh"

namespace rglru {
namespace {

using paged::Batch;

struct AppendArgs {
    Batch b;
    const __nv_bfloat16 *qkv;
    __nv_bfloat16 *q_out;
    uint8_t *k, *v;
    float *ks, *vs;
    uint64_t turns[128];  // base^(-2i/D) / (2 pi), in units of 2^-64
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
__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(bf_pack(f[0], f[1]), bf_pack(f[2], f[3]), bf_pack(f[4], f[5]), bf_pack(f[6], f[7]));
}

// (cos, sin) of position pos at a frequency in turns of 2^-64
__device__ __forceinline__ float2 angle(uint64_t turns, int pos)
{
    const uint32_t frac = (uint32_t)pos * (uint32_t)(turns >> 32) + __umulhi((uint32_t)pos, (uint32_t)turns);
    const float a = (float)(int)frac * 1.4629180792671596e-9f;  // 2 pi / 2^32
    return make_float2(__cosf(a), __sinf(a));
}
__device__ __forceinline__ void rotate(float (&x1)[8], float (&x2)[8], const float2 (&r)[8])
{
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const float y1 = x1[q] * r[q].x - x2[q] * r[q].y, y2 = x2[q] * r[q].x + x1[q] * r[q].y;
        x1[q] = y1, x2[q] = y2;
    }
}

constexpr int kQHeads = 5;  // query heads of a CTA, at most

// 512 threads are held to 64 registers, so that two such CTAs fit an SM (twice the loads in flight of two CTAs of 256
// threads with four passes, which took 36.9 us for the prompts above).
// D channels a head, NP passes of T / (D / 16) rows of the run; a thread holds the channels
// c .. c + 7 and c + D/2 .. c + D/2 + 7 of a row.
template <int D, int NP, int T>
__global__ void __launch_bounds__(T, T == 512 ? 2 : 0) rglru_paged_append_kernel(const __grid_constant__ AppendArgs p)
{
    constexpr int kCols = D / 16, kRows = T / kCols, kHalf = D / 2;
    __shared__ float part[T / 32];
    // read by lanes at different places, which the parameters' constant bank would serve one by one (43 us, here 37)
    __shared__ uint64_t turns[kHalf];
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
    const int r0 = tid / kCols, c = tid % kCols * 8;
    if (role < b.Hkv || role >= 2 * b.Hkv) {
        for (int i = tid; i < kHalf; i += T) turns[i] = p.turns[i];
        __syncthreads();
    }

    if (role >= 2 * b.Hkv) {  // ------------------------------------------------ query heads of kRows tokens
        const int splits = (b.H + kQHeads - 1) / kQHeads, part = (role - 2 * b.Hkv) % splits;
        const int h0 = b.H * part / splits, h1 = b.H * (part + 1) / splits;
        const int slot = lo + (role - 2 * b.Hkv) / splits * kRows + r0;
        if (slot >= hi) return;
        const size_t row = (size_t)(tok0 + slot);
        const __nv_bfloat16 *src = p.qkv + row * width + h0 * D + c;
        __nv_bfloat16 *dst = p.q_out + (row * b.H + h0) * D + c;
        uint4 v[kQHeads][2];
#pragma unroll
        for (int u = 0; u < kQHeads; ++u)
            if (h0 + u < h1) {
                v[u][0] = __ldcs(reinterpret_cast<const uint4 *>(src + u * D));
                v[u][1] = __ldcs(reinterpret_cast<const uint4 *>(src + u * D + kHalf));
            }
        float2 r[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] = angle(turns[c + q], (int)(base + slot));
#pragma unroll
        for (int u = 0; u < kQHeads; ++u)
            if (h0 + u < h1) {
                float x1[8], x2[8];
                unpack8(v[u][0], x1);
                unpack8(v[u][1], x2);
                rotate(x1, x2, r);
                *reinterpret_cast<uint4 *>(dst + u * D) = pack8(x1);
                *reinterpret_cast<uint4 *>(dst + u * D + kHalf) = pack8(x2);
            }
        return;
    }

    // --------------------------------------------------------------------------- one page of a key or value head
    const bool is_k = role < b.Hkv;
    const int head = is_k ? role : role - b.Hkv;
    uint4 raw[NP][2];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int slot = lo + k * kRows + r0;
        raw[k][0] = raw[k][1] = make_uint4(0, 0, 0, 0);
        if (slot < hi) {
            const __nv_bfloat16 *src = p.qkv + (size_t)(tok0 + slot) * width + (b.H + role) * D + c;
            raw[k][0] = __ldcs(reinterpret_cast<const uint4 *>(src));
            raw[k][1] = __ldcs(reinterpret_cast<const uint4 *>(src + kHalf));
        }
    }
    const int page = paged::load_page(b, blockIdx.y, j);
    if (page < 0) return;
    uint8_t *codes = (is_k ? p.k : p.v) + ((size_t)page * b.Hkv + head) * ps * D;
    float *scale = (is_k ? p.ks : p.vs) + (size_t)page * b.Hkv + head;
    const float old = lo > 0 ? *scale : 0.f;
    float x[NP][2][8];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        unpack8(raw[k][0], x[k][0]);
        unpack8(raw[k][1], x[k][1]);
        if (is_k) {
            float2 r[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) r[q] = angle(turns[c + q], (int)(base + lo + k * kRows + r0));
            rotate(x[k][0], x[k][1], r);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) amax = fmaxf(amax, fmaxf(fabsf(x[k][0][q]), fabsf(x[k][1][q])));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) part[tid >> 5] = amax;
    __syncthreads();  // also: every thread has read the old scale
#pragma unroll
    for (int k = 0; k < T / 32; ++k) amax = fmaxf(amax, part[k]);
    const float s_new = fmaxf(old, e4m3::scale_of(amax));
    const float inv = 1.f / s_new;
    if (tid == 0) *scale = s_new;
    if (lo > 0 && s_new != old) {  // the older slots to the larger scale, 16 codes a thread
        const float f = old / s_new;
        constexpr int kBatch = 4;  // loads in flight
        const int all = lo * D / 16;
        for (int i0 = tid; i0 < all; i0 += kBatch * T) {
            uint4 v[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (i0 + u * T < all) v[u] = reinterpret_cast<const uint4 *>(codes)[i0 + u * T];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float f0, f1, f2, f3;
                    e4m3::to_f32x2(w[q] & 0xffffu, f0, f1);
                    e4m3::to_f32x2(w[q] >> 16, f2, f3);
                    w[q] = e4m3::pack4(f0 * f, f1 * f, f2 * f, f3 * f);
                }
                if (i0 + u * T < all) reinterpret_cast<uint4 *>(codes)[i0 + u * T] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int slot = lo + k * kRows + r0;
        if (slot < hi) {
            uint8_t *dst = codes + slot * D + c;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float(&y)[8] = x[k][h];
                *reinterpret_cast<uint2 *>(dst + h * kHalf) =
                    make_uint2(e4m3::pack4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                               e4m3::pack4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
            }
        }
    }
}

template <int D, int NP, int T>
rglru_status launch(const AppendArgs &p, int rows, cudaStream_t stream)
{
    const int per = T / (D / 16), splits = (p.b.H + kQHeads - 1) / kQHeads;
    // pages that a run of max_new tokens can touch, whatever slot it enters at
    const int runs = (p.b.max_new + p.b.page - 2) / p.b.page + 1;
    const dim3 grid(runs, p.b.S, 2 * p.b.Hkv + (rows + per - 1) / per * splits);
    rglru_paged_append_kernel<D, NP, T><<<grid, T, 0, stream>>>(p);
    return cuda_status(cudaGetLastError());
}
// The smallest CTA that holds a page's share of the longest run: single tokens take 64 threads (with 256, and room for a
// whole page of 64 slots in 120 registers, two CTAs fit an SM and 256 sequences took 18 us with the launch, with 64 threads 14).
template <int D>
rglru_status launch(const AppendArgs &p, cudaStream_t stream)
{
    const int rows = p.b.max_new < p.b.page ? p.b.max_new : p.b.page, items = rows * (D / 16);
    if (items <= 64) return launch<D, 1, 64>(p, rows, stream);
    if (items <= 128) return launch<D, 2, 64>(p, rows, stream);
    if (items <= 256) return launch<D, 2, 128>(p, rows, stream);
    if (items <= 512) return launch<D, 2, 256>(p, rows, stream);
    if constexpr (D == 256)  // a page of 128 slots: twice 1024
        if (items > 1024) return launch<D, 8, 256>(p, rows, stream);
    return launch<D, 2, 512>(p, rows, stream);
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
                    static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), k_scale, v_scale, {}};
    const rglru_status c = paged::check_batch(p.b, k_cache, k_scale, v_cache, v_scale, workspace_bytes, kWsHeaderBytes);
    if (c != RGLRU_OK) return c;
    if (!args::al16(qkv) || !args::al16(q_out) || !(rope_base > 1.f) || rope_base > 1e30f) return RGLRU_ERR_INVALID_ARG;
    // a geometric series: at most 128 roundings of 2^-53, which is 2^-22 of a turn at position 2^24
    const double ratio = exp2(-2.0 / head_dim * log2((double)rope_base));
    double turn = 0.15915494309189535 * 18446744073709551616.0;
    for (int i = 0; i < head_dim / 2; ++i, turn *= ratio) p.turns[i] = (uint64_t)turn;
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
    return head_dim == 256 ? launch<256>(p, stream) : launch<128>(p, stream);
}
