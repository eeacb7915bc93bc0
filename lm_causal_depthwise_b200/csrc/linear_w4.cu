// linear_w4.cu -- projections of a few rows with 4-bit weights and group scales.
//
//   out[m, n] = sum_g s[n, g] * sum_{k in group g} (q[n, k] - 8) * x[m, k] + bias[n]
//
// q in 0..15, two to a byte along K (the even k in the low half), s in bf16, x in bf16 or in
// e4m3 with a scale for each group of channels.  Bound by the weight bytes, N K / 2 and 2 N K / group for the scales, while
// there are few rows.
//
// Both kernels use the mma m16n8k16 with the weights as the 16-row operand and the
// rows of x as its 8 columns.  q - 8 is exact in bf16: the nibble is set into the mantissa of 128 (0x4300 | q is
// 128 + q) and 136 is subtracted, two values an instruction, and the scale multiplies the fp32 sum of a group, so
// no weight is ever rounded.  A word of eight nibbles k0 .. k7 gives the pairs (k0, k4), (k1, k5),
// (k2, k6), (k3, k7) by shift and mask alone; x is paired the same way, since the order of a sum's terms is free.
// Of a block of 128 k (four sub-blocks of 32) thread j of a quad takes word j of each sub-block: an mma never mixes two
// groups of 32 or more.
#include "e4m3.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace rglru {
namespace {

constexpr int kMaxM = 64;
constexpr int kBlockK = 128;

struct W4Args {
    int M, N, K, group_shift, a_shift;  // log2 of the groups
    const void *A;
    const float *A_scale;
    const uint8_t *W;
    const uint16_t *W_scale;  // bf16 bits
    const float *bias;
    __nv_bfloat16 *out;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from zero: the first product of a group
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float bf16_bits(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// eight nibbles to four bf16 pairs q - 8: (k0, k4), (k1, k5), (k2, k6), (k3, k7)
__device__ __forceinline__ void unpack(uint32_t w, uint32_t (&r)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t t = ((w >> (4 * e)) & 0x000f000fu) | 0x43004300u;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r[e]) : "r"(t), "r"(0x43084308u));
    }
}
// eight consecutive bf16 to the same pairs
__device__ __forceinline__ void pair_up(uint4 x, uint32_t (&r)[4])
{
    r[0] = __byte_perm(x.x, x.z, 0x5410), r[1] = __byte_perm(x.x, x.z, 0x7632);
    r[2] = __byte_perm(x.y, x.w, 0x5410), r[3] = __byte_perm(x.y, x.w, 0x7632);
}
// eight consecutive e4m3 codes times s; a power of two s leaves them exact
__device__ __forceinline__ void pair_up_e4m3(uint2 x, float s, uint32_t (&r)[4])
{
    float f[8];
    e4m3::to_f32x2(x.x & 0xffffu, f[0], f[1]);
    e4m3::to_f32x2(x.x >> 16, f[2], f[3]);
    e4m3::to_f32x2(x.y & 0xffffu, f[4], f[5]);
    e4m3::to_f32x2(x.y >> 16, f[6], f[7]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[e]) : "f"(f[e + 4] * s), "f"(f[e] * s));
}

// ------------------------------------------------------------------------------------------------ up to 16 rows
// A CTA takes 16 R outputs, its 8 warps every eighth block of 128 k; the warps' sums meet in shared memory.  A
// warp's weights come by cp.async into its own ring (1 KB a block and row tile; 16-byte chunk i of row r sits at
// i ^ (r / 2 % 4), so that the 4-byte reads of a sub-block touch every bank once), its x and scales straight into
// registers one block ahead.
constexpr int kWarps = 8, kRing = 4;
template <int NT, int R>
struct Few {
    static constexpr int kRingBytes = kWarps * kRing * R * 1024, kSums = kWarps * 16 * R * (8 * NT + 1) * 4;
    static constexpr int kSmem = (kRingBytes > kSums ? kRingBytes : kSums) + 128;
};

template <int NT, int R, bool kE4m3>
__global__ void __launch_bounds__(kWarps * 32) rglru_linear_w4_kernel(const W4Args p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, j = lane & 3;
    const int n0 = blockIdx.x * 16 * R;
    const int blocks = (p.K + kBlockK - 1) / kBlockK;
    const int mine = blocks > warp ? (blocks - warp + kWarps - 1) / kWarps : 0;
    const int groups = p.K >> p.group_shift;
    uint8_t *ring = smem + warp * kRing * R * 1024;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);

    auto load_w = [&](int b) {  // block b of this warp's
        const int k0 = (warp + b * kWarps) * kBlockK;
#pragma unroll
        for (int q = 0; q < 2 * R; ++q) {
            const int r = q * 8 + quad;  // row of the tile, chunk j
            const bool in = n0 + r < p.N && k0 + 32 * j < p.K;
            cp16(base + (b % kRing) * R * 1024 + r * 64 + ((j ^ ((r >> 1) & 3)) << 4),
                 p.W + (in ? ((size_t)(n0 + r) * p.K + k0 + 32 * j) / 2 : 0), in);
        }
    };
    uint4 xb[NT][4];      // bf16: 8 values a sub-block; e4m3: 8 codes in .x, .y and the scale in .z
    uint16_t sb[R][2][4];
    auto load_x = [&](int b) {
        const int k0 = (warp + b * kWarps) * kBlockK;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int m = t * 8 + quad;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = k0 + 32 * i + 8 * j;
                xb[t][i] = make_uint4(0, 0, 0, 0);
                if (m < p.M && k < p.K) {
                    if (kE4m3) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(p.A) + (size_t)m * p.K + k);
                        xb[t][i].x = v.x, xb[t][i].y = v.y;
                        xb[t][i].z = __float_as_uint(p.A_scale[(size_t)m * (p.K >> p.a_shift) + (k >> p.a_shift)]);
                    } else {
                        xb[t][i] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.A) + (size_t)m * p.K + k);
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int n = n0 + 16 * r + 8 * h + quad;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k = k0 + 32 * i;
                    // a sub-block that ends its group needs the group's scale
                    const bool ends = ((k + 32) & ((1 << p.group_shift) - 1)) == 0;
                    sb[r][h][i] = n < p.N && k < p.K && ends ? p.W_scale[(size_t)n * groups + (k >> p.group_shift)] : (uint16_t)0;
                }
            }
    };

#pragma unroll
    for (int b = 0; b < kRing - 1; ++b) {
        if (b < mine) load_w(b);
        cp_commit();
    }
    if (mine > 0) load_x(0);
    float acc[R][NT][4] = {}, part[R][NT][4] = {};
    for (int b = 0; b < mine; ++b) {
        uint4 x[NT][4];
        float s[R][2][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[t][i] = xb[t][i];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[r][h][i] = bf16_bits(sb[r][h][i]);
        if (b + 1 < mine) load_x(b + 1);
        __syncwarp();  // the slot that is filled now was read a block ago
        if (b + kRing - 1 < mine) load_w(b + kRing - 1);
        cp_commit();
        cp_wait<kRing - 1>();
        __syncwarp();
        const uint8_t *w = ring + (b % kRing) * R * 1024;
        const int k0 = (warp + b * kWarps) * kBlockK;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (k0 + 32 * i >= p.K) break;
            const bool begins = ((k0 + 32 * i) & ((1 << p.group_shift) - 1)) == 0;
            uint32_t xp[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (kE4m3)
                    pair_up_e4m3(make_uint2(x[t][i].x, x[t][i].y), __uint_as_float(x[t][i].z), xp[t]);
                else
                    pair_up(x[t][i], xp[t]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int sw = ((i ^ (quad >> 1)) << 4) + 4 * j;  // rows quad and quad + 8 share the swizzle
                uint32_t lo[4], hi[4];
                unpack(*reinterpret_cast<const uint32_t *>(w + (16 * r + quad) * 64 + sw), lo);
                unpack(*reinterpret_cast<const uint32_t *>(w + (16 * r + quad + 8) * 64 + sw), hi);
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (begins)
                        mma_bf16_first(part[r][t], a0, xp[t][0], xp[t][1]);
                    else
                        mma_bf16(part[r][t], a0, xp[t][0], xp[t][1]);
                    mma_bf16(part[r][t], a1, xp[t][2], xp[t][3]);
                }
            }
            if (((k0 + 32 * i + 32) & ((1 << p.group_shift) - 1)) == 0) {  // the group ends here
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[r][t][e] = fmaf(part[r][t][e], s[r][e >> 1][i], acc[r][t][e]);
            }
        }
    }
    cp_wait<0>();
    __syncthreads();
    auto sum_at = [&](int w, int r, int m) -> float & {  // over the rings
        return reinterpret_cast<float *>(smem)[(w * 16 * R + r) * (8 * NT + 1) + m];
    };
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum_at(warp, 16 * r + 8 * (e >> 1) + quad, 8 * t + 2 * j + (e & 1)) = acc[r][t][e];
    __syncthreads();
    for (int i = tid; i < 16 * R * p.M; i += kWarps * 32) {
        const int r = i % (16 * R), m = i / (16 * R), n = n0 + r;
        if (n >= p.N) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += sum_at(w, r, m);
        p.out[(size_t)m * p.N + n] = __float2bfloat16_rn(v + (p.bias != nullptr ? p.bias[n] : 0.f));
    }
}

// ------------------------------------------------------------------------------------------------ 17 to 64 rows
// A CTA takes 128 outputs (8 warps of 16) over its share of K's blocks, x is shared by its warps: its block comes by
// cp.async, is paired (and taken out of e4m3) once per CTA a block ahead, and then read as whole operands.  CTAs of a
// cluster share the outputs and split K; their sums meet through distributed shared memory.
constexpr int kWideThreads = 256, kWideN = 128, kWideRing = 4;

template <int NT>
struct Wide {
    static constexpr int kW = kWideN * 64;            // weights of a block
    static constexpr int kX = 8 * NT * kBlockK * 2;   // x of a block: as it comes (bf16; e4m3 half of it), and paired
    static constexpr int kStage = kW + kX;
    static constexpr int kSums = kWideN * (8 * NT + 1) * 4;
    static constexpr int kLoop = kWideRing * kStage + 2 * kX + 2 * 4 * kWideN * 4;
    static constexpr int kSmem = (kLoop > kSums ? kLoop : kSums) + 128;
};

// the same shared-memory place in CTA `rank` of the cluster
__device__ __forceinline__ const float *peer(const float *x, int rank)
{
    uint64_t a;
    asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(x), "r"(rank));
    return reinterpret_cast<const float *>(a);
}

template <int NT>
__global__ void __launch_bounds__(kWideThreads, 2) rglru_linear_w4_wide_kernel(const W4Args p, int cluster)
{
    using C = Wide<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    uint8_t *paired = smem + kWideRing * C::kStage;
    float *scales = reinterpret_cast<float *>(paired + 2 * C::kX);  // [2][4 sub-blocks][128 rows]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, j = lane & 3;
    const int srow = tid & (kWideN - 1), shalf = tid / kWideN;  // whose scales this thread loads: row, sub-block pair
    const int rank = (int)(blockIdx.x % cluster), n0 = (int)(blockIdx.x / cluster) * kWideN;
    const int blocks = (p.K + kBlockK - 1) / kBlockK;
    const int b0 = (int)((long long)blocks * rank / cluster), count = (int)((long long)blocks * (rank + 1) / cluster) - b0;
    const int groups = p.K >> p.group_shift, gmask = (1 << p.group_shift) - 1;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    const bool e4 = p.A_scale != nullptr;

    auto load = [&](int b) {
        const int k0 = (b0 + b) * kBlockK;
        const uint32_t st = base + (b % kWideRing) * C::kStage;
#pragma unroll
        for (int q = 0; q < kWideN * 4 / kWideThreads; ++q) {
            const int r = q * (kWideThreads / 4) + (tid >> 2), i = tid & 3;
            const bool in = n0 + r < p.N && k0 + 32 * i < p.K;
            cp16(st + r * 64 + ((i ^ ((r >> 1) & 3)) << 4), p.W + (in ? ((size_t)(n0 + r) * p.K + k0 + 32 * i) / 2 : 0), in);
        }
        const int per = e4 ? 8 : 16, bytes = e4 ? 1 : 2;  // 16-byte chunks of a row of x
        for (int c = tid; c < 8 * NT * per; c += kWideThreads) {
            const int m = c / per, k = k0 + c % per * (16 / bytes);
            const bool in = m < p.M && k < p.K;
            cp16(st + C::kW + c * 16, static_cast<const uint8_t *>(p.A) + (in ? ((size_t)m * p.K + k) * bytes : 0), in);
        }
    };
    // x of block b, from its stage to operands: [sub-block][row][j] of 16 bytes, the 4 threads of a quad side by side
    auto convert = [&](int b) {
        const uint8_t *src = smem + (b % kWideRing) * C::kStage + C::kW;
        uint4 *dst = reinterpret_cast<uint4 *>(paired + (b & 1) * C::kX);
#pragma unroll
        for (int q = 0; q < (8 * NT * 16 + kWideThreads - 1) / kWideThreads; ++q) {
            const int c = q * kWideThreads + tid, m = c >> 4, o = c & 15;  // octet o of row m: sub-block o / 4, thread o % 4
            if (c >= 8 * NT * 16) break;
            uint32_t r[4];
            if (e4) {
                const int k = (b0 + b) * kBlockK + 8 * o;
                const float s = m < p.M && k < p.K ? p.A_scale[(size_t)m * (p.K >> p.a_shift) + (k >> p.a_shift)] : 0.f;
                pair_up_e4m3(*reinterpret_cast<const uint2 *>(src + c * 8), s, r);
            } else {
                pair_up(*reinterpret_cast<const uint4 *>(src + c * 16), r);
            }
            dst[(o >> 2) * 32 * NT + m * 4 + (o & 3)] = make_uint4(r[0], r[1], r[2], r[3]);
        }
    };
    // the scales of a block, at the sub-blocks that end a group
    uint16_t sc[2];
    auto load_scales = [&](int b) {
        const uint16_t *src = p.W_scale + (size_t)(n0 + srow) * groups;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = (b0 + b) * kBlockK + 64 * shalf + 32 * i;
            sc[i] = n0 + srow < p.N && k < p.K && ((k + 32) & gmask) == 0 ? src[k >> p.group_shift] : (uint16_t)0;
        }
    };
    auto store_scales = [&](int b) {
#pragma unroll
        for (int i = 0; i < 2; ++i) scales[((b & 1) * 4 + 2 * shalf + i) * kWideN + srow] = bf16_bits(sc[i]);
    };

#pragma unroll
    for (int b = 0; b < kWideRing - 1; ++b) {
        if (b < count) load(b);
        cp_commit();
    }
    float acc[NT][4] = {}, part[NT][4] = {};
    if (count > 0) {
        load_scales(0);
        cp_wait<kWideRing - 2>();
        __syncthreads();
        convert(0);
        store_scales(0);
        if (count > 1) load_scales(1);
    }
    for (int b = 0; b < count; ++b) {
        cp_wait<kWideRing - 3>();
        __syncthreads();  // block b is paired, block b + 1 has landed, block b - 1 is done with
        if (b + kWideRing - 1 < count) load(b + kWideRing - 1);
        cp_commit();
        if (b + 1 < count) {
            convert(b + 1);
            store_scales(b + 1);
            if (b + 2 < count) load_scales(b + 2);
        }
        const uint8_t *w = smem + (b % kWideRing) * C::kStage;
        const uint4 *xs = reinterpret_cast<const uint4 *>(paired + (b & 1) * C::kX);
        const float *s = scales + (b & 1) * 4 * kWideN + warp * 16 + quad;
        const int k0 = (b0 + b) * kBlockK;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (k0 + 32 * i >= p.K) break;
            const bool begins = ((k0 + 32 * i) & gmask) == 0;
            const int sw = ((i ^ (quad >> 1)) << 4) + 4 * j;
            uint32_t lo[4], hi[4];
            unpack(*reinterpret_cast<const uint32_t *>(w + (warp * 16 + quad) * 64 + sw), lo);
            unpack(*reinterpret_cast<const uint32_t *>(w + (warp * 16 + quad + 8) * 64 + sw), hi);
            const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
            if (begins) {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint4 x = xs[i * 32 * NT + t * 32 + lane];
                    mma_bf16_first(part[t], a0, x.x, x.y);
                    mma_bf16(part[t], a1, x.z, x.w);
                }
            } else {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const uint4 x = xs[i * 32 * NT + t * 32 + lane];
                    mma_bf16(part[t], a0, x.x, x.y);
                    mma_bf16(part[t], a1, x.z, x.w);
                }
            }
            if (((k0 + 32 * i + 32) & gmask) == 0) {
                const float s0 = s[i * kWideN], s1 = s[i * kWideN + 8];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(part[t][e], e < 2 ? s0 : s1, acc[t][e]);
            }
        }
    }
    cp_wait<0>();
    __syncthreads();
    float *sums = reinterpret_cast<float *>(smem);  // [128 outputs][8 NT + 1], over the ring
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sums[(warp * 16 + 8 * (e >> 1) + quad) * (8 * NT + 1) + 8 * t + 2 * j + (e & 1)] = acc[t][e];
    sm100::cluster_sync();
    // this CTA's outputs of the cluster's, summed in rank order
    const int r0 = kWideN * rank / cluster, share = kWideN * (rank + 1) / cluster - r0;
    for (int i = tid; i < share * p.M; i += kWideThreads) {
        const int r = r0 + i % share, m = i / share, n = n0 + r;
        if (n >= p.N) continue;
        float v = 0.f;
#pragma unroll 4
        for (int c = 0; c < cluster; ++c) v += *peer(sums + r * (8 * NT + 1) + m, c);
        p.out[(size_t)m * p.N + n] = __float2bfloat16_rn(v + (p.bias != nullptr ? p.bias[n] : 0.f));
    }
    sm100::cluster_sync();  // no CTA leaves while another reads its sums
}

constexpr int kSms = 148;

template <int NT, int R, bool kE4m3>
rglru_status launch_few(const W4Args &p, cudaStream_t stream)
{
    using C = Few<NT, R>;
    static PerDeviceFlag flag;
    const rglru_status st =
        set_smem_limit_once(reinterpret_cast<const void *>(rglru_linear_w4_kernel<NT, R, kE4m3>), C::kSmem, flag);
    if (st != RGLRU_OK) return st;
    rglru_linear_w4_kernel<NT, R, kE4m3><<<(unsigned)((p.N + 16 * R - 1) / (16 * R)), kWarps * 32, C::kSmem, stream>>>(p);
    return cuda_status(cudaGetLastError());
}
template <int NT>
rglru_status launch_few(const W4Args &p, cudaStream_t stream)
{
    // two row tiles a CTA read x half as often, once that leaves a CTA for every SM
    if (p.N > 32 * kSms)
        return p.A_scale != nullptr ? launch_few<NT, 2, true>(p, stream) : launch_few<NT, 2, false>(p, stream);
    return p.A_scale != nullptr ? launch_few<NT, 1, true>(p, stream) : launch_few<NT, 1, false>(p, stream);
}

template <int NT>
rglru_status launch_wide(const W4Args &p, cudaStream_t stream)
{
    using C = Wide<NT>;
    static PerDeviceFlag flag;
    const rglru_status st =
        set_smem_limit_once(reinterpret_cast<const void *>(rglru_linear_w4_wide_kernel<NT>), C::kSmem, flag);
    if (st != RGLRU_OK) return st;
    // K is split so that the busiest SM has the least to do: its CTAs times a CTA's blocks and about two blocks' time
    // to begin and end one
    const int tiles = (p.N + kWideN - 1) / kWideN, blocks = (p.K + kBlockK - 1) / kBlockK;
    int cluster = 1;
    long long best = -1;
    for (int c = 1; c <= 8; ++c) {
        const long long cost = (((long long)tiles * c + kSms - 1) / kSms) * ((blocks + c - 1) / c + 2);
        if (best < 0 || cost < best) best = cost, cluster = c;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * cluster)), cfg.blockDim = dim3(kWideThreads), cfg.stream = stream;
    cfg.dynamicSmemBytes = C::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, rglru_linear_w4_wide_kernel<NT>, p, cluster));
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
    auto log2i = [](int v) { int s = 0; while ((1 << s) < v) ++s; return s; };
    const W4Args p = {M, N, K, log2i(group), A_scale ? log2i(a_group) : 0, A, A_scale, static_cast<const uint8_t *>(W),
                      static_cast<const uint16_t *>(W_scale), bias, static_cast<__nv_bfloat16 *>(out)};
    switch ((M + 7) / 8) {
    case 1: return launch_few<1>(p, stream);
    case 2: return launch_few<2>(p, stream);
    case 3: return launch_wide<3>(p, stream);
    case 4: return launch_wide<4>(p, stream);
    case 5: return launch_wide<5>(p, stream);
    case 6: return launch_wide<6>(p, stream);
    case 7: return launch_wide<7>(p, stream);
    default: return launch_wide<8>(p, stream);
    }
}
