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

// Scales of a row at the sub-blocks of a block that end a group, as bf16 pairs (sub-blocks 0, 1 and 2, 3): one load where
// the row's groups are a multiple of a block's (its address is aligned then), none for sub-blocks inside a group.
template <bool kVec>
__device__ __forceinline__ uint2 load_scales(const uint16_t *row, int k0, int K, int shift)
{
    if (row == nullptr) return make_uint2(0, 0);
    const uint16_t *src = row + (k0 >> shift);
    if (kVec) {
        if (shift == 7) return make_uint2(0, (uint32_t)src[0] << 16);
        if (shift == 5) return *reinterpret_cast<const uint2 *>(src);
        const uint32_t v = *reinterpret_cast<const uint32_t *>(src);
        return make_uint2(v << 16, v & 0xffff0000u);
    }
    uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = k0 + 32 * i;
        if (k < K && ((k + 32) & ((1 << shift) - 1)) == 0) v[i] = row[k >> shift];
    }
    return make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
}
__device__ __forceinline__ float scale_at(uint2 v, int i)
{
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
}

// kVec: K is a multiple of 128 (then so are the scales' rows of a block's groups, and no block is cut)
template <int NT, int R, bool kE4m3, bool kVec>
__global__ void __launch_bounds__(kWarps * 32) rglru_linear_w4_kernel(const W4Args p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, j = lane & 3;
    const int n0 = blockIdx.x * 16 * R;
    const int blocks = (p.K + kBlockK - 1) / kBlockK;
    const int mine = blocks > warp ? (blocks - warp + kWarps - 1) / kWarps : 0;
    const int groups = p.K >> p.group_shift, gmask = (1 << p.group_shift) - 1;
    uint8_t *ring = smem + warp * kRing * R * 1024;

    // this lane's places: chunk j of its 2 R rows of W, its rows of x, its rows of scales; a warp's next block is kWarps on
    const uint8_t *wp[2 * R];
    const uint16_t *sp[2 * R];
    uint32_t wdst[2 * R];
#pragma unroll
    for (int q = 0; q < 2 * R; ++q) {
        const int r = q * 8 + quad, n = n0 + r;
        wp[q] = n < p.N ? p.W + ((size_t)n * p.K + warp * kBlockK) / 2 + 16 * j : nullptr;
        sp[q] = n < p.N ? p.W_scale + (size_t)n * groups : nullptr;
        wdst[q] = (uint32_t)__cvta_generic_to_shared(ring) + r * 64 + ((j ^ ((r >> 1) & 3)) << 4);
    }
    constexpr int kBytes = kE4m3 ? 1 : 2;
    const uint8_t *xp[NT];
    const float *asp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int m = t * 8 + quad;
        xp[t] = m < p.M ? static_cast<const uint8_t *>(p.A) + ((size_t)m * p.K + warp * kBlockK + 8 * j) * kBytes : nullptr;
        asp[t] = kE4m3 && m < p.M ? p.A_scale + (size_t)m * (p.K >> p.a_shift) : nullptr;
    }
    auto load_w = [&](int b, int slot) {  // block b of this warp's
        const bool in = kVec || (warp + b * kWarps) * kBlockK + 32 * j < p.K;
#pragma unroll
        for (int q = 0; q < 2 * R; ++q) {
            const bool take = in && wp[q] != nullptr;
            cp16(wdst[q] + slot * R * 1024, take ? wp[q] + (size_t)b * (kWarps * kBlockK / 2) : p.W, take);
        }
    };
    uint4 xb[NT][4];  // bf16: 8 values a sub-block; e4m3: 8 codes in .x, .y and the scale in .z
    uint2 sb[2 * R];
    auto load_x = [&](int b) {
        const int k0 = (warp + b * kWarps) * kBlockK;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint8_t *src = xp[t] + (size_t)b * (kWarps * kBlockK * kBytes);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xb[t][i] = make_uint4(0, 0, 0, 0);
                if (xp[t] != nullptr && (kVec || k0 + 32 * i < p.K)) {
                    if (kE4m3) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(src + 32 * i);
                        xb[t][i] = make_uint4(v.x, v.y, __float_as_uint(asp[t][(k0 + 32 * i) >> p.a_shift]), 0);
                    } else {
                        xb[t][i] = *reinterpret_cast<const uint4 *>(src + 64 * i);
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 2 * R; ++q) sb[q] = load_scales<kVec>(sp[q], k0, p.K, p.group_shift);
    };

#pragma unroll
    for (int b = 0; b < kRing - 1; ++b) {
        if (b < mine) load_w(b, b);
        cp_commit();
    }
    if (mine > 0) load_x(0);
    float acc[R][NT][4] = {}, part[R][NT][4] = {};
    for (int b = 0; b < mine; ++b) {
        uint4 x[NT][4];
        uint2 s[2 * R];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[t][i] = xb[t][i];
#pragma unroll
        for (int q = 0; q < 2 * R; ++q) s[q] = sb[q];
        if (b + 1 < mine) load_x(b + 1);
        __syncwarp();  // the slot that is filled now was read a block ago
        if (b + kRing - 1 < mine) load_w(b + kRing - 1, (b + kRing - 1) % kRing);
        cp_commit();
        cp_wait<kRing - 1>();
        __syncwarp();
        const uint8_t *w = ring + (b % kRing) * R * 1024 + quad * 64 + 4 * j;
        const int k0 = (warp + b * kWarps) * kBlockK;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!kVec && k0 + 32 * i >= p.K) break;
            const bool begins = ((32 * i + (kVec ? 0 : k0)) & gmask) == 0, ends = ((32 * i + 32 + (kVec ? 0 : k0)) & gmask) == 0;
            uint32_t xq[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (kE4m3)
                    pair_up_e4m3(make_uint2(x[t][i].x, x[t][i].y), __uint_as_float(x[t][i].z), xq[t]);
                else
                    pair_up(x[t][i], xq[t]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int sw = (i ^ (quad >> 1)) << 4;  // rows quad and quad + 8 share the swizzle
                uint32_t lo[4], hi[4];
                unpack(*reinterpret_cast<const uint32_t *>(w + r * 1024 + sw), lo);
                unpack(*reinterpret_cast<const uint32_t *>(w + r * 1024 + 512 + sw), hi);
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
                if (begins) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_bf16_first(part[r][t], a0, xq[t][0], xq[t][1]);
                } else {
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_bf16(part[r][t], a0, xq[t][0], xq[t][1]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_bf16(part[r][t], a1, xq[t][2], xq[t][3]);
                if (ends) {
                    const float s0 = scale_at(s[2 * r], i), s1 = scale_at(s[2 * r + 1], i);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[r][t][e] = fmaf(part[r][t][e], e < 2 ? s0 : s1, acc[r][t][e]);
                }
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
// K is split over the CTAs of a cluster, so that a CTA holds its share of x in shared memory as finished operands (paired, and
// taken out of e4m3, once) while it walks over the outputs: a round is 128 of them, 16 a warp, and no warp waits for another
// within it.  A warp's weights come by cp.async into its own ring, across rounds, its scales into registers one block ahead.  At a
// round's end the cluster's sums meet through distributed shared memory, in rank order.
// With x re-read for every 128 outputs instead (a barrier and a conversion each block) 37 rows of
// 12289 x 4096 took 68 us.
constexpr int kWideThreads = 256, kWideN = 128, kWideRing = 4;

template <int NT>
struct Wide {
    static constexpr int kX = 8 * NT * kBlockK * 2;  // operands of a block
    static constexpr int kRingBytes = kWarps * kWideRing * 1024;
    // sums of two rounds: [2][128 outputs][M, made odd]
    static constexpr int sums(int M) { return 2 * kWideN * (M | 1) * 4; }
    static constexpr int smem(int blocks, int M) { return blocks * kX + kRingBytes + sums(M) + 128; }
    static constexpr int max_blocks(int M) { return (226 * 1024 - kRingBytes - sums(M) - 128) / kX; }
};

// the same shared-memory place in CTA `rank` of the cluster
__device__ __forceinline__ const float *peer(const float *x, int rank)
{
    uint64_t a;
    asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(x), "r"(rank));
    return reinterpret_cast<const float *>(a);
}

// kShift: log2 of the group where K is a multiple of 128, or 0: any group, any K.  held: blocks of x in shared memory at a
// time.
template <int NT, int kShift>
__global__ void __launch_bounds__(kWideThreads, 2) rglru_linear_w4_wide_kernel(const W4Args p, int cluster, int held)
{
    using C = Wide<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    uint4 *xs = reinterpret_cast<uint4 *>(smem);  // [block][sub-block][row of x][thread of a quad]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, j = lane & 3;
    uint8_t *ring = smem + held * C::kX + warp * kWideRing * 1024;
    float *sums = reinterpret_cast<float *>(smem + held * C::kX + C::kRingBytes);  // [2][128 outputs][sum_row]
    const int rank = (int)(blockIdx.x % cluster), first = (int)(blockIdx.x / cluster), step = (int)(gridDim.x / cluster);
    const int tiles = (p.N + kWideN - 1) / kWideN, blocks = (p.K + kBlockK - 1) / kBlockK;
    const int b0 = (int)((long long)blocks * rank / cluster), count = (int)((long long)blocks * (rank + 1) / cluster) - b0;
    constexpr bool kVec = kShift != 0;
    const int shift = kVec ? kShift : p.group_shift, groups = p.K >> shift, gmask = (1 << shift) - 1, sum_row = p.M | 1;
    const int rounds = (tiles - first + step - 1) / step;  // at least one: the grid has no more clusters than tiles
    const uint32_t wdst = (uint32_t)__cvta_generic_to_shared(ring) + quad * 64 + ((j ^ (quad >> 1)) << 4);

    auto load_x = [&](int b, int n) {  // blocks b .. b + n - 1 of this rank's into xs
        constexpr int kBatch = 4;  // loads in flight a thread
        const int all = n * 8 * NT * 16;
        for (int c0 = tid; c0 < all; c0 += kBatch * kWideThreads) {
            uint4 v[kBatch];
            float sc[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int c = c0 + u * kWideThreads, o = c & 15, m = (c >> 4) % (8 * NT);  // octet o of row m
                const int k = (b0 + b + c / (8 * NT * 16)) * kBlockK + 8 * o;
                v[u] = make_uint4(0, 0, 0, 0);
                sc[u] = 0.f;
                if (c < all && m < p.M && k < p.K) {
                    if (p.A_scale != nullptr) {
                        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(p.A) + (size_t)m * p.K + k);
                        v[u].x = w.x, v[u].y = w.y;
                        sc[u] = p.A_scale[(size_t)m * (p.K >> p.a_shift) + (k >> p.a_shift)];
                    } else {
                        v[u] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.A) + (size_t)m * p.K + k);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int c = c0 + u * kWideThreads, o = c & 15, m = (c >> 4) % (8 * NT), x = c / (8 * NT * 16);
                uint32_t r[4];
                if (p.A_scale != nullptr)
                    pair_up_e4m3(make_uint2(v[u].x, v[u].y), sc[u], r);
                else
                    pair_up(v[u], r);
                if (c < all) xs[(x * 4 + (o >> 2)) * 32 * NT + m * 4 + (o & 3)] = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
    };

    // A warp's line of blocks, over all rounds; the weights are kRing - 1 blocks ahead, the scales one.  Rows quad and
    // quad + 8 of the warp's 16: chunk j of their weights, their scales.
    struct Ahead {
        int round, b;
        const uint8_t *w[2];
        const uint16_t *s[2];
    };
    auto place = [&](Ahead &a) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = (first + a.round * step) * kWideN + warp * 16 + 8 * h + quad;
            a.w[h] = n < p.N ? p.W + ((size_t)n * p.K + b0 * kBlockK) / 2 + 16 * j : nullptr;
            a.s[h] = n < p.N ? p.W_scale + (size_t)n * groups : nullptr;
        }
    };
    Ahead aw = {0, 0, {}, {}}, as = {0, 0, {}, {}};
    place(aw), place(as);
    int ld_slot = 0, slot = 0;
    uint2 sb[2] = {};
    auto load_w = [&]() {
        if (aw.round < rounds) {
            const bool in = kVec || (b0 + aw.b) * kBlockK + 32 * j < p.K;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool take = in && aw.w[h] != nullptr;
                cp16(wdst + ld_slot * 1024 + 512 * h, take ? aw.w[h] + aw.b * (kBlockK / 2) : p.W, take);
            }
            if (++ld_slot == kWideRing) ld_slot = 0;
            if (++aw.b == count) aw.b = 0, ++aw.round, place(aw);
        }
        cp_commit();
    };
    auto load_s = [&]() {
        if (as.round < rounds) {
#pragma unroll
            for (int h = 0; h < 2; ++h) sb[h] = load_scales<kVec>(as.s[h], (b0 + as.b) * kBlockK, p.K, shift);
            if (++as.b == count) as.b = 0, ++as.round, place(as);
        }
    };
    if (count > 0) {
#pragma unroll
        for (int b = 0; b < kWideRing - 1; ++b) load_w();
        load_s();
    }
    // this CTA's outputs of the cluster's, of one round
    auto join = [&](int round) {
        const int n0 = (first + round * step) * kWideN, r0 = kWideN * rank / cluster;
        const int share = kWideN * (rank + 1) / cluster - r0;
        const float *from = sums + (round & 1) * kWideN * sum_row;
        for (int i = tid; i < share * p.M; i += kWideThreads) {
            const int r = r0 + i % share, m = i / share, n = n0 + r;
            if (n >= p.N) continue;
            float v = 0.f;
#pragma unroll 4
            for (int c = 0; c < cluster; ++c) v += *peer(from + r * sum_row + m, c);
            p.out[(size_t)m * p.N + n] = __float2bfloat16_rn(v + (p.bias != nullptr ? p.bias[n] : 0.f));
        }
        __syncwarp();
    };
    const bool once = count <= held;
    if (once) {
        load_x(0, count);
        __syncthreads();
    }
    for (int round = 0; round < rounds; ++round) {
        float acc[NT][4] = {}, part[NT][4] = {};
        for (int b = 0; b < count; ++b) {
            if (!once && b % held == 0) {
                __syncthreads();
                load_x(b, min(held, count - b));
                __syncthreads();
            }
            const uint2 s[2] = {sb[0], sb[1]};
            load_s();
            __syncwarp();  // the slot that is filled now was read a block ago
            load_w();
            cp_wait<kWideRing - 1>();
            __syncwarp();
            const uint8_t *w = ring + slot * 1024 + quad * 64 + 4 * j;
            if (++slot == kWideRing) slot = 0;
            const uint4 *xb = xs + (once ? b : b % held) * 4 * 32 * NT + lane;
            const int k0 = (b0 + b) * kBlockK;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!kVec && k0 + 32 * i >= p.K) break;
                const int sw = (i ^ (quad >> 1)) << 4;
                uint32_t lo[4], hi[4];
                unpack(*reinterpret_cast<const uint32_t *>(w + sw), lo);
                unpack(*reinterpret_cast<const uint32_t *>(w + 512 + sw), hi);
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
                uint4 x[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) x[t] = xb[(i * NT + t) * 32];
                if (((32 * i + (kVec ? 0 : k0)) & gmask) == 0) {  // a group begins
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_bf16_first(part[t], a0, x[t].x, x[t].y);
                } else {
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_bf16(part[t], a0, x[t].x, x[t].y);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_bf16(part[t], a1, x[t].z, x[t].w);
                if (((32 * i + 32 + (kVec ? 0 : k0)) & gmask) == 0) {
                    const float s0 = scale_at(s[0], i), s1 = scale_at(s[1], i);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(part[t][e], e < 2 ? s0 : s1, acc[t][e]);
                }
            }
        }
        // the last round's sums meet now that a round's work has passed since they were written
        if (round > 0) {
            sm100::cluster_wait();
            join(round - 1);
        }
        float *mine = sums + (round & 1) * kWideN * sum_row;  // all have read what was here: that was before they arrived
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (8 * t + 2 * j + (e & 1) < p.M)
                    mine[(warp * 16 + 8 * (e >> 1) + quad) * sum_row + 8 * t + 2 * j + (e & 1)] = acc[t][e];
        __syncwarp();
        sm100::cluster_arrive();
    }
    sm100::cluster_wait();
    join(rounds - 1);
    cp_wait<0>();
    __syncwarp();
    sm100::cluster_sync();  // no CTA leaves while another reads its sums
}

constexpr int kSms = 148;

template <int NT, int R, bool kE4m3, bool kVec>
rglru_status launch_few(const W4Args &p, cudaStream_t stream)
{
    using C = Few<NT, R>;
    static PerDeviceFlag flag;
    const rglru_status st =
        set_smem_limit_once(reinterpret_cast<const void *>(rglru_linear_w4_kernel<NT, R, kE4m3, kVec>), C::kSmem, flag);
    if (st != RGLRU_OK) return st;
    rglru_linear_w4_kernel<NT, R, kE4m3, kVec>
        <<<(unsigned)((p.N + 16 * R - 1) / (16 * R)), kWarps * 32, C::kSmem, stream>>>(p);
    return cuda_status(cudaGetLastError());
}
template <int NT, int R>
rglru_status launch_few(const W4Args &p, cudaStream_t stream)
{
    const bool vec = p.K % kBlockK == 0;
    if (p.A_scale != nullptr) return vec ? launch_few<NT, R, true, true>(p, stream) : launch_few<NT, R, true, false>(p, stream);
    return vec ? launch_few<NT, R, false, true>(p, stream) : launch_few<NT, R, false, false>(p, stream);
}
template <int NT>
rglru_status launch_few(const W4Args &p, cudaStream_t stream)
{
    // two row tiles a CTA read x half as often, once that leaves a CTA for every SM
    return p.N > 32 * kSms ? launch_few<NT, 2>(p, stream) : launch_few<NT, 1>(p, stream);
}

template <int NT, int kShift>
rglru_status launch_wide(const W4Args &p, cudaStream_t stream)
{
    using C = Wide<NT>;
    // The split of K: rounds of the busiest SM times a round's blocks (and about two blocks' time to end it), over
    // cluster sizes; two CTAs on an SM share its issue slots, but hide each other's latency (three quarters of the time).
    // Clusters of several CTAs find room on 132 of the 148 SMs (33 clusters of 4 were resident, the rest of a GPC
    // does not hold one): one cluster more would run after all others.
    const int tiles = (p.N + kWideN - 1) / kWideN, blocks = (p.K + kBlockK - 1) / kBlockK, most = C::max_blocks(p.M);
    int cluster = 1, clusters = 1, held = 1;
    long long best = -1;
    for (int c = 1; c <= 8; c *= 2) {
        const int share = (blocks + c - 1) / c, h = share < most ? share : most;
        const int per_sm = C::smem(h, p.M) <= 113 * 1024 ? 2 : 1;
        int n = (c == 1 ? kSms : 132) * per_sm / c;
        if (n > tiles) n = tiles;
        const int busy = n * c > kSms ? 6 : 4;  // CTAs that share an SM
        const long long cost = ((long long)(tiles + n - 1) / n) * (share + 2 + (share > h ? share : 0)) * busy;
        if (best < 0 || cost < best) best = cost, cluster = c, clusters = n, held = h;
    }
    static PerDeviceFlag flag;
    const rglru_status st = set_smem_limit_once(reinterpret_cast<const void *>(rglru_linear_w4_wide_kernel<NT, kShift>),
                                                227 * 1024, flag);
    if (st != RGLRU_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * cluster)), cfg.blockDim = dim3(kWideThreads), cfg.stream = stream;
    cfg.dynamicSmemBytes = C::smem(held, p.M);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, rglru_linear_w4_wide_kernel<NT, kShift>, p, cluster, held));
}
template <int NT>
rglru_status launch_wide(const W4Args &p, cudaStream_t stream)
{
    if (p.K % kBlockK != 0) return launch_wide<NT, 0>(p, stream);
    return p.group_shift == 5   ? launch_wide<NT, 5>(p, stream)
           : p.group_shift == 6 ? launch_wide<NT, 6>(p, stream)
                                : launch_wide<NT, 7>(p, stream);
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
    case 3:
    case 4: return launch_wide<4>(p, stream);
    case 5: return launch_wide<5>(p, stream);
    case 6: return launch_wide<6>(p, stream);
    default: return launch_wide<8>(p, stream);
    }
}
