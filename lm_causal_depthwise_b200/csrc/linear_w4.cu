// linear_w4.cu -- projections of a few rows with 4-bit weights and group scales.
//
//   out[m, n] = sum_g s[n, g] * sum_{k in group g} (q[n, k] - 8) * x[m, k] + bias[n]
//
// q in 0..15, two to a byte along K (the even k in the low half), s in bf16, x in bf16 or in e4m3 with a scale for each
// group of channels.  Bound by the weight bytes, N K / 2 and 2 N K / group for the scales, while there are few rows.
//
// Both kernels have the weights as the operand of many rows and the rows of x as its columns.  q - 8 is exact in bf16:
// the nibble is set into the mantissa of 128 (0x4300 | q is 128 + q) and 136 is subtracted, two values an instruction,
// and the scale multiplies the fp32 sum of a group, so no weight is ever rounded.  A word of eight nibbles k0 .. k7
// gives the pairs (k0, k4), (k1, k5), (k2, k6), (k3, k7) by shift and mask alone; x is paired the same way, since the
// order of a sum's terms is free.
//
// Measured with the launch: 1 row of 2560 x 2560 8 us, 8 rows (e4m3) of 7680 x 2560 10 us, 37 rows of 12289 x 4096 in
// groups of 32 38 us.
#include "e4m3.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace rglru {
namespace {

constexpr int kMaxM = 64;
constexpr int kBlockK = 128;

struct W4Args {
    int M, N, K, group_shift, a_shift;  // log2 of the groups
    int withhold;  // test hook: 1 + the CTA that keeps an arrival back, 0 = none
    const void *A;
    const float *A_scale;
    const uint8_t *W;
    const uint16_t *W_scale;  // bf16 bits
    const float *bias;
    __nv_bfloat16 *out;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// 16 bytes of weights, read once; the lines around them into L2 (a block takes 64 bytes of a row, the next one those behind)
__device__ __forceinline__ uint4 ld_ahead(const uint4 *src)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src));
    return v;
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
// mma m16n8k16, 16 outputs and 8 rows of x.  A CTA takes 16 R outputs, its 8 warps every eighth block of 128 k; the
// warps' sums meet in shared memory.  Of a block (four sub-blocks of 32 k) thread j of a quad takes word j of each
// sub-block: an mma never mixes two groups of 32 or more.  A warp's weights come by cp.async into its own ring (1 KB a
// block and row tile; 16-byte chunk i of row r sits at i ^ (r / 2 % 4), so that the 4-byte reads of a sub-block touch
// every bank once), its x and scales straight into registers, kAhead blocks ahead.
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
    // blocks of x and scales in registers: most warps' whole share where the grid is one CTA an SM, fewer where two are to fit
    constexpr int kAhead = R == 1 ? (NT == 1 ? 3 : 2) : 1;
    uint4 xr[kAhead][NT][4];  // bf16: 8 values a sub-block; e4m3: 8 codes in .x, .y and the scale in .z
    uint2 sr[kAhead][2 * R];
    auto load_x = [&](int b, uint4 (&xb)[NT][4], uint2 (&sb)[2 * R]) {
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
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (u < mine) load_x(u, xr[u], sr[u]);
    float acc[R][NT][4] = {}, part[R][NT][4] = {};
    auto block = [&](int b, uint4 (&x)[NT][4], uint2 (&s)[2 * R]) {
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
        if (b + kAhead < mine) load_x(b + kAhead, x, s);
    };
    for (int b = 0; b < mine; b += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (b + u < mine) block(b + u, xr[u], sr[u]);
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

// ------------------------------------------------------------------------------------------------ more rows or outputs
// The weights of 128 outputs and 128 k become a bf16 operand in TMEM, once for all rows of x, and the products run on
// tcgen05 (M = 128 outputs, N = rows of x): with mma.sync each warp unpacked, paired and scaled for itself, 613
// instructions for 16 outputs and 128 k, and 37 rows of 12289 x 4096 took 53 us.  Unpacked into shared memory the
// stores and the products' reads of the weights held each other up (a block's products 0.9 us, 0.45 without the
// stores; 46 us).  In TMEM it takes 38 us, 26 of them without the adding of the groups' sums (0.9 us a block in groups
// of 32: four times 48 columns through registers), which is what bounds it.
//   warps 0-3    thread = output = TMEM lane: adds a group's sum, times its scale, to fp32 accumulators
//   warp 4       issues the products: a group at a time into its own TMEM columns
//   warps 5-12   unpack: a thread has 64 k of one output, read 32 bytes at a time several blocks ahead
// K is split over the CTAs of a cluster; a CTA keeps its share of x in shared memory as operand boxes (64 k, 128-byte
// swizzle; taken out of e4m3 there) while it walks over the outputs, 128 a round.  The cluster's sums meet through
// distributed shared memory, in rank order.
constexpr int kTcN = 128, kTcThreads = 13 * 32, kTcUnpack = 8 * 32, kTcStages = 2, kTcAhead = 4;
constexpr uint32_t kTcColA = 512 - kTcStages * 64;  // unpacked blocks; the groups' sums before them
constexpr uint64_t kTimeoutNs = 2000000000ull;

template <int NP>  // rows of x, in sixteens
struct Tc {
    static constexpr int kBox = NP * 128;                  // x: 64 k
    static constexpr int kX = 2 * kBox;                    // x of a block
    static constexpr int sums(int M) { return kTcN * M * 4; }
    static constexpr int max_blocks(int M) { return (226 * 1024 - sums(M) - 1024) / kX; }
};

// the same shared-memory place in CTA `rank` of the cluster
__device__ __forceinline__ const float *peer(const float *x, int rank)
{
    uint64_t a;
    asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(x), "r"(rank));
    return reinterpret_cast<const float *>(a);
}
// A wait that gives up after 2 s returns false.  Who gave up waits no more and passes the barriers of the CTA and the
// cluster with the others, but arrives on no mbarrier and starts nothing: every arrival stands for a wait that was won, so
// those behind run out of their waits too, up to the threads of the outputs, which become NaN.
__device__ __noinline__ bool w4_wait_slow(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = sm100::globaltimer();
    while (sm100::globaltimer() - t0 < kTimeoutNs)
        if (sm100::mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    return false;
}
__device__ __forceinline__ bool w4_wait(uint64_t *bar, uint32_t parity)
{
    return sm100::mbar_try_wait(bar, parity) || w4_wait_slow(bar, parity);
}

// held: blocks of x in shared memory at a time
template <int NP, bool kVec>
__global__ void __launch_bounds__(kTcThreads, 1) rglru_linear_w4_tc_kernel(const W4Args p, int cluster, int held)
{
    using namespace sm100;
    using C = Tc<NP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *xs = smem;
    float *sums = reinterpret_cast<float *>(xs + held * C::kX);  // [M][128 outputs]
    __shared__ uint64_t a_full[kTcStages], a_free[kTcStages], d_full[2], d_free[2], drain;
    __shared__ uint32_t tmem_holder;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)(blockIdx.x % cluster), first = (int)(blockIdx.x / cluster), step = (int)(gridDim.x / cluster);
    const int tiles = (p.N + kTcN - 1) / kTcN, blocks = (p.K + kBlockK - 1) / kBlockK;
    const int b0 = (int)((long long)blocks * rank / cluster), count = (int)((long long)blocks * (rank + 1) / cluster) - b0;
    const int shift = p.group_shift, groups = p.K >> shift, per = kBlockK >> shift;
    const int rounds = (tiles - first + step - 1) / step;  // at least one: the grid has no more clusters than tiles

    if (warp == 4) {
        tmem_alloc(&tmem_holder, 512);
        if (lane == 0) {
            for (int i = 0; i < kTcStages; ++i) mbar_init(a_full + i, kTcUnpack), mbar_init(a_free + i, 1);
            for (int i = 0; i < 2; ++i) mbar_init(d_full + i, 1), mbar_init(d_free + i, 128);
            mbar_init(&drain, 1);
            mbar_fence_init();
        }
    }
    auto load_x = [&](int b, int n) {  // blocks b .. b + n - 1 of this rank's into xs, octets paired as the weights are
        constexpr int kBatch = 4;      // loads in flight a thread
        const int all = n * NP * 16;
        for (int c0 = tid; c0 < all; c0 += kBatch * kTcThreads) {
            uint4 v[kBatch];
            float sc[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int c = c0 + u * kTcThreads, o = c & 15, m = (c >> 4) % NP;  // octet o of row m
                const int k = (b0 + b + c / (NP * 16)) * kBlockK + 8 * o;
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
                const int c = c0 + u * kTcThreads, o = c & 15, m = (c >> 4) % NP, x = c / (NP * 16);
                uint32_t r[4];
                if (p.A_scale != nullptr)
                    pair_up_e4m3(make_uint2(v[u].x, v[u].y), sc[u], r);
                else
                    pair_up(v[u], r);
                if (c < all)
                    *reinterpret_cast<uint4 *>(xs + x * C::kX + (o >> 3) * C::kBox + m * 128 + (((o & 7) ^ (m & 7)) << 4)) =
                        make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
        fence_proxy_async_smem();
    };
    const bool once = count <= held;
    if (once) load_x(0, count);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_holder;
    // blocks whose groups' sums fit at a time (one only for 64 rows in groups of 32)
    const int sets = 2 * per * NP <= (int)kTcColA ? 2 : 1;
    bool alive = true;

    // an unpacking thread's place in its line of blocks: 64 k (a box) of one output a block, kTcAhead blocks in registers
    const int urow = (warp & 3) * 32 + lane, ubox = (warp - 5) >> 2;  // a warp reaches the TMEM lanes of its quarter
    // one set of registers for what a thread keeps: those words, or (warps 0-3) the sums of its output
    uint32_t keep[NP > 8 * kTcAhead ? NP : 8 * kTcAhead];
    int ld_round = 0, ld_b = 0;
    auto load_w = [&](uint32_t *keep) {
        uint4 w[2] = {};
        auto put = [&]() {
#pragma unroll
            for (int h = 0; h < 2; ++h) keep[4 * h] = w[h].x, keep[4 * h + 1] = w[h].y, keep[4 * h + 2] = w[h].z, keep[4 * h + 3] = w[h].w;
        };
        if (ld_round >= rounds || count == 0) return put();
        const int n = (first + ld_round * step) * kTcN + urow, k = (b0 + ld_b) * kBlockK + 64 * ubox;
        if (n < p.N) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.W + ((size_t)n * p.K + k) / 2);
            if (kVec || k < p.K) w[0] = ld_ahead(src);
            if (kVec || k + 32 < p.K) w[1] = ld_ahead(src + 1);
        }
        put();
        if (++ld_b == count) ld_b = 0, ++ld_round;
    };
    // the scales of a thread's output, two blocks ahead over all rounds
    int sc_round = 0, sc_b = 0;
    uint2 sc[2];
    auto load_sc = [&]() {
        if (sc_round >= rounds || count == 0) return make_uint2(0, 0);
        const int n = (first + sc_round * step) * kTcN + tid;
        const uint2 v = load_scales<kVec>(n < p.N ? p.W_scale + (size_t)n * groups : nullptr, (b0 + sc_b) * kBlockK, p.K, shift);
        if (++sc_b == count) sc_b = 0, ++sc_round;
        return v;
    };
    if (warp < 4) sc[0] = load_sc(), sc[1] = load_sc();
    if (warp >= 5) {
#pragma unroll
        for (int u = 0; u < kTcAhead; ++u) load_w(keep + 8 * u);
    }
    int at = 0;  // whose turn it is of those in registers
    int slot = 0, turn = 0;  // this role's place in the ring of unpacked blocks
    int set = 0, set_turn = 0;  // and in the sets of sums
    auto next_set = [&]() {
        if (++set == sets) set = 0, ++set_turn;
    };
    auto next_slot = [&]() {
        if (++slot == kTcStages) slot = 0, ++turn;
    };
    for (int round = 0; round < rounds; ++round) {
        const int n0 = (first + round * step) * kTcN;
        if (warp < 4) {
#pragma unroll
            for (int m = 0; m < NP; ++m) keep[m] = 0;
        }
        for (int pass = 0; pass < count; pass += held) {
            const int end = min(count, pass + held);
            if (!once) {
                __syncthreads();  // the products of the last pass have been read: their operands are done with
                load_x(pass, end - pass);
                __syncthreads();
            }
            if (warp >= 5) {
                // ------------------------------------------------------------ weights to operands
                for (int b = pass; b < end; ++b) {
                    // a warp's verdict: its store to TMEM is one instruction, and the last block there may be in use
                    if (turn > 0 && alive) alive = w4_wait(a_free + slot, (uint32_t)(turn - 1) & 1u);
                    alive = __all_sync(0xffffffffu, alive);
                    auto write = [&](uint32_t *words) {  // a register queue needs its place known when compiled
                        uint32_t r[32];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            uint32_t q[4];
                            unpack(words[c], q);
                            r[4 * c] = q[0], r[4 * c + 1] = q[1], r[4 * c + 2] = q[2], r[4 * c + 3] = q[3];
                        }
                        load_w(words);
                        __syncwarp();
                        if (alive) tmem_st32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + kTcColA + (uint32_t)(slot * 64 + ubox * 32), r);
                    };
                    tc_fence_after();
                    switch (at) {
                    case 0: write(keep); break;
                    case 1: write(keep + 8); break;
                    case 2: write(keep + 16); break;
                    default: write(keep + 24); break;
                    }
                    at = (at + 1) % kTcAhead;
                    tmem_wait_st();
                    tc_fence_before();
                    if (alive && !(tid == 5 * 32 && round == 0 && b == 0 && p.withhold == (int)blockIdx.x + 1)) mbar_arrive(a_full + slot);
                    next_slot();
                }
            } else if (warp == 4) {
                // ------------------------------------------------------------ products
                const uint32_t idesc = umma_idesc_bf16(kTcN, NP);
                const int steps_log = shift - 4;  // of 16 k in a group
                for (int b = pass; b < end; ++b) {
                    if (alive) alive = w4_wait(a_full + slot, (uint32_t)turn & 1u);
                    if (set_turn > 0 && alive) alive = w4_wait(d_free + set, (uint32_t)(set_turn - 1) & 1u);
                    alive = __all_sync(0xffffffffu, alive);
                    if (!alive) break;
                    tc_fence_after();
                    const uint64_t xd = umma_desc_sw128(smem_u32(xs + (b - (once ? 0 : pass)) * C::kX));
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_ts_warp(tmem + (uint32_t)((set * per + (kk >> steps_log)) * NP), tmem + kTcColA + (uint32_t)(slot * 64 + kk * 8),
                                     xd + (uint64_t)(((kk >> 2) * C::kBox + (kk & 3) * 32) >> 4), idesc, (kk & ((1 << steps_log) - 1)) != 0);
                    umma_commit_warp(d_full + set);
                    umma_commit_warp(a_free + slot);
                    __syncwarp();
                    next_slot();
                    next_set();
                }
            } else {
                // ------------------------------------------------------------ groups to outputs, thread = output
                const uint32_t lanes = (uint32_t)(warp * 32) << 16;
                for (int b = pass; b < end; ++b) {
                    if (alive) alive = w4_wait(d_full + set, (uint32_t)set_turn & 1u);
                    __syncwarp();
                    tc_fence_after();
                    const uint2 now = sc[0];
                    sc[0] = sc[1];
                    sc[1] = load_sc();
                    // 16 columns at a time, the next ones on their way while these are added
                    const int live = kVec ? per : min(per, (p.K - (b0 + b) * kBlockK) >> shift);
                    const uint32_t from = tmem + lanes + (uint32_t)(set * per * NP);
                    uint32_t d[2][16];
                    tmem_ld16(from, d[0]);
#pragma unroll 1
                    for (int g0 = 0; g0 < live; g0 += 2) {
#pragma unroll
                        for (int gg = 0; gg < 2; ++gg) {  // two groups: an even count of loads, so that the buffers' turns are fixed
                            const int g = g0 + gg;
                            if (g >= live) break;
                            const f2_t w = f2_splat(scale_at(now, ((g + 1) << (shift - 5)) - 1));
#pragma unroll
                            for (int c = 0; c < NP / 16; ++c) {
                                const int x = gg * (NP / 16) + c;
                                uint32_t(&cur)[16] = d[x & 1], (&next)[16] = d[(x & 1) ^ 1];
                                tmem_wait_ld();
                                if (c + 1 < NP / 16 || g + 1 < live) tmem_ld16(from + (uint32_t)(g * NP + 16 * (c + 1)), next);
#pragma unroll
                                for (int e = 0; e < 16; e += 2) {
                                    const f2_t v = f2_fma(f2_make(__uint_as_float(cur[e]), __uint_as_float(cur[e + 1])), w,
                                                          f2_make(__uint_as_float(keep[16 * c + e]), __uint_as_float(keep[16 * c + e + 1])));
                                    keep[16 * c + e] = __float_as_uint(f2_lo(v)), keep[16 * c + e + 1] = __float_as_uint(f2_hi(v));
                                }
                            }
                        }
                    }
                    tmem_wait_ld();
                    tc_fence_before();
                    if (alive) mbar_arrive(d_free + set);
                    next_set();
                }
            }
        }
        // The cluster's sums of this round: written, then read by warps 0-3.  The other warps pass both barriers of a
        // round at the end of their next one, and are unpacking it meanwhile.
        __syncwarp();
        if (warp >= 4) {
            if (round > 0) cluster_wait(), cluster_arrive(), cluster_wait();
            cluster_arrive();
            continue;
        }
        if (round > 0) cluster_wait();  // every CTA has read the last round's
#pragma unroll
        for (int m = 0; m < NP; ++m)
            if (m < p.M) sums[m * kTcN + tid] = __uint_as_float(alive ? keep[m] : 0x7fc00000u);
        __syncwarp();
        cluster_sync();
        // this CTA's outputs, four neighbours a thread: a distributed load covers whole lines (with the rows of x innermost,
        // every lane's load was a request of its own and the join took 8 us)
        const int share = kTcN / cluster, r0 = share * rank, quads = share / 4, quads_log = 31 - __clz(quads);
        for (int c = tid; c < quads * p.M; c += 128) {
            const int r = r0 + 4 * (c & (quads - 1)), m = c >> quads_log, n = n0 + r;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.bias != nullptr) {
                if (n < p.N) v.x = p.bias[n];
                if (n + 1 < p.N) v.y = p.bias[n + 1];
                if (n + 2 < p.N) v.z = p.bias[n + 2];
                if (n + 3 < p.N) v.w = p.bias[n + 3];
            }
#pragma unroll 4
            for (int k = 0; k < cluster; ++k) {
                const float4 u = *reinterpret_cast<const float4 *>(peer(sums + m * kTcN + r, k));
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
            __nv_bfloat16 *dst = p.out + (size_t)m * p.N + n;
            if (n < p.N) dst[0] = __float2bfloat16_rn(v.x);
            if (n + 1 < p.N) dst[1] = __float2bfloat16_rn(v.y);
            if (n + 2 < p.N) dst[2] = __float2bfloat16_rn(v.z);
            if (n + 3 < p.N) dst[3] = __float2bfloat16_rn(v.w);
        }
        __syncwarp();
        cluster_arrive();
    }
    __syncwarp();
    if (warp >= 4) cluster_wait(), cluster_arrive();
    cluster_wait();  // no CTA leaves while another reads its sums
    if (warp == 4) {  // nor while a product is in flight
        umma_commit_warp(&drain);
        w4_wait(&drain, 0);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tmem, 512);
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

template <int NP, bool kVec>
rglru_status launch_tc(const W4Args &p, cudaStream_t stream)
{
    using C = Tc<NP>;
    // The split of K: rounds of the busiest CTA times a round's blocks (and about three blocks' time to end it), over
    // cluster sizes.  Clusters of several CTAs find room on 132 of the 148 SMs (33 clusters of 4 were resident, the rest
    // of a GPC does not hold one): one cluster more would run after all others.
    const int tiles = (p.N + kTcN - 1) / kTcN, blocks = (p.K + kBlockK - 1) / kBlockK;
    int cluster = 1, clusters = 1, held = 1;
    long long best = -1;
    for (int c = 1; c <= 8; c *= 2) {
        const int share = (blocks + c - 1) / c, most = C::max_blocks(p.M), h = share < most ? share : most;
        int n = (c == 1 ? kSms : 132) / c;
        if (n > tiles) n = tiles;
        const long long cost = ((long long)(tiles + n - 1) / n) * (share + 3 + (share > h ? 2 * share : 0));
        if (best < 0 || cost < best) best = cost, cluster = c, clusters = n, held = h;
    }
    // At least half of the SM's shared memory: two CTAs on an SM would take turns with TMEM, and of two clusters (or one and
    // another kernel whose CTAs wait for each other; those take 170 KB or more) each could hold what the other's peers
    // wait for.  Not all of it: the rest is L1, and 37 rows of 12289 x 4096 took 44 us instead of 38.
    constexpr int kSmem = 226 * 1024, kLeast = 115 * 1024;
    static_assert(2 * (kLeast + 1024) > 228 * 1024, "one CTA an SM");
    static PerDeviceFlag flag;
    const rglru_status st =
        set_smem_limit_once(reinterpret_cast<const void *>(rglru_linear_w4_tc_kernel<NP, kVec>), kSmem, flag);
    if (st != RGLRU_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * cluster)), cfg.blockDim = dim3(kTcThreads), cfg.stream = stream;
    const int need = held * C::kX + C::sums(p.M) + 1024;
    cfg.dynamicSmemBytes = need < kLeast ? kLeast : need;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, rglru_linear_w4_tc_kernel<NP, kVec>, p, cluster, held));
}
template <int NP>
rglru_status launch_tc(const W4Args &p, cudaStream_t stream)
{
    return p.K % kBlockK == 0 ? launch_tc<NP, true>(p, stream) : launch_tc<NP, false>(p, stream);
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
    const W4Args p = {M, N, K, log2i(group), A_scale ? log2i(a_group) : 0, debug_withheld, A, A_scale, static_cast<const uint8_t *>(W),
                      static_cast<const uint16_t *>(W_scale), bias, static_cast<__nv_bfloat16 *>(out)};
    // Up to 16 rows the first kernel is the faster one at every size measured, by 2 to 4 us where x is e4m3 and there are two
    // row tiles of it, by 4 to 15 otherwise.  First and second kernel, us behind a flush of L2, groups of 128, x in bf16 (e4m3):
    //   rows    2560 x 2560             7680 x 2560             12288 x 4096
    //      1     6 and 11 ( 7 and 12)   10 and 18 (10 and 19)   19 and 32 (20 and 33)
    //      8     7 and 12 ( 7 and 12)   10 and 18 (11 and 19)   19 and 33 (21 and 34)
    //     16     8 and 12 ( 9 and 13)   12 and 19 (16 and 20)   22 and 34 (32 and 34)
    if (M <= 16) return M <= 8 ? launch_few<1>(p, stream) : launch_few<2>(p, stream);
    switch ((M + 15) / 16) {
    case 2: return launch_tc<32>(p, stream);
    case 3: return launch_tc<48>(p, stream);
    default: return launch_tc<64>(p, stream);
    }
}
