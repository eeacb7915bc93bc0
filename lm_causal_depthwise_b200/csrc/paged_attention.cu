// paged_attention.cu -- causal sliding-window attention of the new tokens over a paged 8-bit cache.
//
//   out[t, h] = sum_p softmax_p(scale * q[t, h] . k[p]) v[p],   pos_t - window < p <= pos_t
//
// with k[p], v[p] = code * scale of p's page and head.  Positions outside a row's range
// are never read or never weighted; a row without any key gives zeros.
#include "paged.cuh"
#include "sm100.cuh"

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

// ------------------------------------------------------------------------------------------------ schedule
// A unit is 16 rows (row = token * G + head in the group, G = H / Hkv) of one sequence and key/value head;
// its work is the 64-key tiles of the sequence's attended range.  All units' tiles form one line, cut into
// gridDim.x equal pieces: long and short sequences balance, and one long sequence spreads over every SM.
constexpr int kRowTile = 16, kKeyTile = 64, kThreads = 128, kMinTiles = 2;
constexpr int kSms = 148, kMaxCtas = 3 * kSms;
constexpr size_t align_up_d(size_t v, size_t a) { return (v + a - 1) / a * a; }

template <int D>
struct Cfg {
    static constexpr int kStages = D == 256 ? 3 : 4;
    static constexpr int kCtasPerSm = D == 256 ? 2 : 3;
    static constexpr int kStageBytes = 2 * kKeyTile * D;
    static constexpr int kSmem = kStages * kStageBytes;
};

struct Plan {  // the unit that begins in a CTA's piece and does not end there
    int parts, seq, unit, rows;
};
// Workspace: header, plans, then per CTA two partial results (slot 2 c: a unit begun in an earlier CTA; 2 c + 1: one begun
// here) of 16 rows: m, mv, l, pad (float4) and O [16][D].
constexpr size_t kPlanBytes = (size_t)kMaxCtas * sizeof(Plan);
__host__ __device__ constexpr size_t part_floats(int D) { return (size_t)kRowTile * (4 + D); }
inline size_t attention_bytes(int D)
{
    return kWsHeaderBytes + align_up_d(kPlanBytes, 256) + (size_t)kMaxCtas * 2 * part_floats(D) * 4;
}

struct Geometry {
    int row0, n, ctx, tile0, tiles, units;  // tiles per unit
};
__device__ __forceinline__ Geometry geometry(const AttendArgs &p, int i)
{
    const paged::Seq s = paged::load_seq(p.b, i);
    Geometry g = {s.row0, s.n, s.ctx, 0, 0, 0};
    if (s.n > 0) {
        g.tile0 = max(0, s.ctx - p.window + 1) / kKeyTile;
        g.tiles = (s.ctx + s.n - 1) / kKeyTile - g.tile0 + 1;
        const int G = p.b.H / p.b.Hkv;
        g.units = p.b.Hkv * (int)(((long long)s.n * G + kRowTile - 1) / kRowTile);
    }
    return g;
}

// A place on the line of tiles.
struct Cursor {
    int seq, unit, tile;
    Geometry g;
};
__device__ __forceinline__ void advance(const AttendArgs &p, Cursor &c)
{
    if (++c.tile < c.g.tiles) return;
    c.tile = 0;
    if (++c.unit < c.g.units) return;
    c.unit = 0;
    while (++c.seq < p.b.S) {
        c.g = geometry(p, c.seq);
        if (c.g.units > 0) return;
    }
}

struct Unit {
    int head, row, rows;    // key/value head, first row (token * G + head in group), rows
    int pos0, pos1;         // positions of the first and last row
    int lo, hi;             // keys any row attends
};
__device__ __forceinline__ Unit unit_of(const AttendArgs &p, const Cursor &c)
{
    const int G = p.b.H / p.b.Hkv, per_head = c.g.units / p.b.Hkv;
    Unit u;
    u.head = c.unit / per_head;
    u.row = c.unit % per_head * kRowTile;
    u.rows = min(kRowTile, c.g.n * G - u.row);
    u.pos0 = c.g.ctx + u.row / G;
    u.pos1 = c.g.ctx + (u.row + u.rows - 1) / G;
    u.lo = max(0, u.pos0 - p.window + 1);
    u.hi = u.pos1 + 1;
    return u;
}

// ------------------------------------------------------------------------------------------------ pieces
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }

// bytes of w that are NaN codes become 0xff, the others 0
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w)
{
    const uint32_t t = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    return (t >> 7) * 0xffu;
}

// The exact line [begin, end) of CTA c out of n over `total` tiles.
__device__ __forceinline__ long long piece_begin(long long total, int c, int n) { return total * c / n; }
__device__ __forceinline__ int piece_of(long long total, long long t, int n) { return (int)(((t + 1) * n - 1) / total); }

// ------------------------------------------------------------------------------------------------ the kernel
// Four warps.  A 64-key tile of k and v (codes) arrives by cp.async in a ring.  S = Q K^T: warp w has the 16 keys of group w
// (one page, so one scale) and all 16 rows; the row maxima meet in shared memory, P goes
// there as f16 in the layout of an mma operand, and O += P V: warp w has channels w D/4 .. of all keys, so that O is never summed
// across warps.  Codes turn into f16 operands exactly, in registers.  k's scale multiplies the scores; v's enters the
// exponent: P holds 2^(s - m + log2 vs - mv) with mv the running maximum of s - m + log2 vs, beside the softmax's own
// maximum m and sum l = sum 2^(s - m), so that P keeps f16's bits whatever the pages' scales (mv is relative to m: a
// large score would swallow log2 vs).
template <int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kCtasPerSm) rglru_paged_attention_kernel(const AttendArgs p)
{
    using C = Cfg<D>;
    constexpr int kStages = C::kStages, kChunks = D / 16, kKb = D / 64, kNt = D / 32, kSlice = D / 4;
    constexpr int kRowsPerPass = kThreads / kChunks, kPasses = kKeyTile / kRowsPerPass;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ float4 wmax[kRowTile], wlv;
    __shared__ uint4 pbuf[4][32];
    __shared__ float lsum[4][kRowTile];
    __shared__ long long scan[5];
    __shared__ int where[4];
    const Batch &b = p.b;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, j = lane & 3;
    const int G = b.H / b.Hkv, page_shift = 31 - __clz(b.page);

    // ---------------------------------------------------------------- this CTA's piece of the line
    const int per = (b.S + kThreads - 1) / kThreads, s0 = min(b.S, tid * per), s1 = min(b.S, s0 + per);
    long long mine = 0;
    for (int i = s0; i < s1; ++i) {
        const Geometry g = geometry(p, i);
        mine += (long long)g.tiles * g.units;
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    before += inc - mine;
    const int n_ctas = (int)min((long long)gridDim.x, (total + kMinTiles - 1) / kMinTiles), cta = blockIdx.x;
    Plan *plans = reinterpret_cast<Plan *>(reinterpret_cast<char *>(b.ws) + kWsHeaderBytes);
    if (cta >= n_ctas) {
        if (tid == 0) plans[cta] = {0, 0, 0, 0};
        return;
    }
    const long long begin = piece_begin(total, cta, n_ctas), end = piece_begin(total, cta + 1, n_ctas);
    if (begin >= before && begin < before + mine) {
        long long at = before;
        for (int i = s0; i < s1; ++i) {
            const Geometry g = geometry(p, i);
            const long long c = (long long)g.tiles * g.units;
            if (begin < at + c) {
                where[0] = i;
                where[1] = (int)((begin - at) / g.tiles);
                where[2] = (int)((begin - at) % g.tiles);
                break;
            }
            at += c;
        }
    }
    __syncthreads();
    Cursor pc;  // the producer's place: the next tile to load
    pc.seq = where[0], pc.unit = where[1], pc.tile = where[2];
    pc.g = geometry(p, pc.seq);
    Cursor cc = pc;  // the consumer's
    const int count = (int)(end - begin);
    float *parts = reinterpret_cast<float *>(reinterpret_cast<char *>(b.ws) + kWsHeaderBytes + align_up_d(kPlanBytes, 256));
    Plan plan = {0, 0, 0, 0};

    // ---------------------------------------------------------------- loads
    const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);
    const int ld_row = tid / kChunks, ld_chunk = tid % kChunks;
    int pages[4];                                  // of the next tile to load; -1: nothing to read there
    Unit pu = unit_of(p, pc);
    auto look_up = [&]() {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int p0 = (pc.g.tile0 + pc.tile) * kKeyTile + 16 * q;
            pages[q] = p0 + 16 > pu.lo && p0 < pu.hi ? b.table[(size_t)pc.seq * b.max_pages + (p0 >> page_shift)] : -2;
        }
    };
    float ksr[kStages], lvr[kStages];              // scales of this warp's 16 keys, one entry a tile in flight
    auto issue = [&](int stage) {
        const uint32_t dk = ring_addr + stage * C::kStageBytes, dv = dk + kKeyTile * D;
        const int key0 = (pc.g.tile0 + pc.tile) * kKeyTile;
        float ks = 0.f, vs = 0.f;
        bool mine_ok = false;
        size_t at[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (pages[q] != -2 && (pages[q] < 0 || pages[q] >= b.num_pages)) {
                paged::record_invalid(b.ws);
                pages[q] = -2;
            }
            at[q] = (size_t)(pages[q] < 0 ? 0 : pages[q]) * b.Hkv + pu.head;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q == warp && pages[q] >= 0) ks = p.ks[at[q]], vs = p.vs[at[q]], mine_ok = true;
#pragma unroll
        for (int r = 0; r < kPasses; ++r) {
            const int row = r * kRowsPerPass + ld_row, q = r * kRowsPerPass / 16;   // 16 keys: one page
            const int key = key0 + row;
            const bool in = pages[q] >= 0 && key >= pu.lo && key < pu.hi;
            const size_t off = in ? ((at[q] << page_shift) + (key & (b.page - 1))) * D + ld_chunk * 16 : 0;
            cp16(dk + row * D + ((ld_chunk ^ ((row & 1) << 2)) << 4), p.k + off, in);
            cp16(dv + row * D + ((ld_chunk ^ (((row >> 1) & 3) << 1)) << 4), p.v + off, in);
        }
        ksr[kStages - 1] = ks, lvr[kStages - 1] = mine_ok ? log2f(vs) : -INFINITY;
        advance(p, pc);
    };
    int loaded = 0;
    look_up();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
#pragma unroll
        for (int q = 0; q + 1 < kStages; ++q) ksr[q] = ksr[q + 1], lvr[q] = lvr[q + 1];
        if (loaded < count) {
            issue(s);
            if (++loaded < count) {
                pu = unit_of(p, pc);
                look_up();
            }
        }
        cp_commit();
    }

    // ---------------------------------------------------------------- tiles
    uint32_t qf[kKb][4][4];
    float acc[kNt][4], m[2], mv[2], l[2], qs[2];
    int pos[2];
    Unit cu = {};
    bool start = true;
    int unit_first = 0;  // whether the piece holds the unit's first tile
    for (int it = 0; it < count; ++it) {
        cp_wait<kStages - 2>();
        __syncthreads();
#pragma unroll
        for (int q = 0; q + 1 < kStages; ++q) ksr[q] = ksr[q + 1], lvr[q] = lvr[q + 1];
        if (loaded < count) {
            issue((it + kStages - 1) % kStages);
            if (++loaded < count) {
                pu = unit_of(p, pc);
                look_up();
            }
        }
        cp_commit();

        if (start) {  // a new unit: its queries as operands, its sums empty
            start = false;
            unit_first = cc.tile == 0;
            cu = unit_of(p, cc);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = quad + 8 * h;
                const bool live = r < cu.rows;
                const int row = cu.row + (live ? r : 0);
                pos[h] = cc.g.ctx + row / G;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    p.q + ((size_t)(cc.g.row0 + row / G) * b.H + cu.head * G + row % G) * D + 16 * j);
                uint4 v[kKb][2];
                uint32_t top = 0;
#pragma unroll
                for (int kb = 0; kb < kKb; ++kb) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        v[kb][e] = live ? src[kb * 8 + e] : make_uint4(0, 0, 0, 0);
                        const uint32_t w[4] = {v[kb][e].x, v[kb][e].y, v[kb][e].z, v[kb][e].w};
#pragma unroll
                        for (int x = 0; x < 4; ++x) top = max(top, max((w[x] << 16) & 0x7f800000u, w[x] & 0x7f800000u));
                    }
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // the row's largest exponent to 2^13: every bf16 down to 2^-27 of it is a normal f16
                int e = min(100, max(-100, (int)(top >> 23) - 127 - 13));
                if (top == 0) e = 0;
                const float f = __uint_as_float((uint32_t)(127 - e) << 23);
                qs[h] = p.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int kb = 0; kb < kKb; ++kb) {
                    const uint32_t w[8] = {v[kb][0].x, v[kb][0].y, v[kb][0].z, v[kb][0].w,
                                           v[kb][1].x, v[kb][1].y, v[kb][1].z, v[kb][1].w};
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        qf[kb][s][h] = pack_f16(bf_lo(w[2 * s]) * f, bf_hi(w[2 * s]) * f);
                        qf[kb][s][2 + h] = pack_f16(bf_lo(w[2 * s + 1]) * f, bf_hi(w[2 * s + 1]) * f);
                    }
                }
                m[h] = mv[h] = -INFINITY;
                l[h] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < kNt; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
        }
        const uint8_t *sk = ring + (it % kStages) * C::kStageBytes, *sv = sk + kKeyTile * D;
        const int key0 = (cc.g.tile0 + cc.tile) * kKeyTile;

        // S of this warp's 16 keys
        float s[2][4] = {};
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const int row = warp * 16 + nt * 8 + quad;
                const uint4 c = *reinterpret_cast<const uint4 *>(sk + row * D + (((kb * 4 + j) ^ ((row & 1) << 2)) << 4));
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    mma_f16(s[nt], qf[kb][x], e4m3::to_f16x2(w[x] & 0xffffu), e4m3::to_f16x2(w[x] >> 16));
            }
        }
        const float ks = ksr[0], lv = lvr[0];
        const bool ok = lv != -INFINITY || ks != 0.f;
        // whether some key of the tile is outside some row's range (rows of one token: outside keys were never loaded, but
        // they must not be weighted either)
        const bool edge = key0 < cu.pos1 - p.window + 1 || key0 + kKeyTile - 1 > cu.pos0 || !ok;
        float tmax[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nt][e] *= qs[e >> 1] * ks;
                if (edge) {
                    const int key = key0 + warp * 16 + nt * 8 + 2 * j + (e & 1);
                    if (!ok || key > pos[e >> 1] || key <= pos[e >> 1] - p.window) s[nt][e] = -INFINITY;
                }
                tmax[e >> 1] = fmaxf(tmax[e >> 1], s[nt][e]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            tmax[h] = fmaxf(tmax[h], __shfl_xor_sync(0xffffffffu, tmax[h], 1));
            tmax[h] = fmaxf(tmax[h], __shfl_xor_sync(0xffffffffu, tmax[h], 2));
            if (j == 0) {
                reinterpret_cast<float *>(&wmax[quad + 8 * h])[warp] = tmax[h];
            }
        }
        if (lane == 0) reinterpret_cast<float *>(&wlv)[warp] = ok ? lv : 0.f;
        __syncthreads();
        float f[2];
        bool moved = false;
        uint32_t pk[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 a = wmax[quad + 8 * h], v = wlv;
            const float m1 = fmaxf(m[h], fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w))), mz = finite_or_0(m1);
            const float step = m[h] - mz;
            const float v1 = fmaxf(fmaxf(mv[h] + step, fmaxf(v.x + (a.x - mz), v.y + (a.y - mz))),
                                   fmaxf(v.z + (a.z - mz), v.w + (a.w - mz)));
            const float vz = finite_or_0(v1);
            l[h] *= sm100::ex2_approx(step);
            f[h] = sm100::ex2_approx(mv[h] + step - vz);
            moved |= f[h] != 1.f;
            m[h] = m1, mv[h] = v1;
            const float d = ok ? lv - vz : 0.f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const float s0v = s[nt][2 * h] - mz, s1v = s[nt][2 * h + 1] - mz;
                l[h] += sm100::ex2_approx(s0v) + sm100::ex2_approx(s1v);
                pk[2 * nt + h] = pack_f16(sm100::ex2_approx(s0v + d), sm100::ex2_approx(s1v + d));
            }
        }
        pbuf[warp][lane] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int t = 0; t < kNt; ++t) acc[t][0] *= f[0], acc[t][1] *= f[0], acc[t][2] *= f[1], acc[t][3] *= f[1];
        }
        __syncthreads();

        // O += P V for this warp's channels: thread's 8 (D = 256; 4) channels of the keys 2j, 2j + 1, 2j + 8, 2j + 9
        const bool mixed = edge && cu.pos0 != cu.pos1;  // rows that do not see the same keys
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const uint4 pa = pbuf[kk][lane];
            const uint32_t a[4] = {pa.x, pa.y, pa.z, pa.w};
            uint32_t v[4][kNt / 4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = kk * 16 + 2 * j + (q & 1) + (q >> 1) * 8;
                const int byte = warp * kSlice + quad * kNt;
                const uint8_t *src = sv + row * D + (((byte >> 4) ^ (((row >> 1) & 3) << 1)) << 4) + (byte & 15);
                if (kNt == 8) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(src);
                    v[q][0] = w.x, v[q][kNt / 4 - 1] = w.y;
                } else {
                    v[q][0] = *reinterpret_cast<const uint32_t *>(src);
                }
            }
            uint32_t bad[4][kNt / 4];
            bool any = false;
            if (mixed) {  // a NaN may only reach the rows that see its key: it is taken out of the product
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int x = 0; x < kNt / 4; ++x) {
                        bad[q][x] = nan_bytes(v[q][x]);
                        v[q][x] &= ~bad[q][x];
                        any |= bad[q][x] != 0;
                    }
                any = __any_sync(0xffffffffu, any);
            }
#pragma unroll
            for (int x = 0; x < kNt / 4; ++x) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t b0 = __byte_perm(v[0][x], v[1][x], y ? 0x7362 : 0x5140);
                    const uint32_t b1 = __byte_perm(v[2][x], v[3][x], y ? 0x7362 : 0x5140);
                    mma_f16(acc[4 * x + 2 * y], a, e4m3::to_f16x2(b0 & 0xffffu), e4m3::to_f16x2(b1 & 0xffffu));
                    mma_f16(acc[4 * x + 2 * y + 1], a, e4m3::to_f16x2(b0 >> 16), e4m3::to_f16x2(b1 >> 16));
                }
            }
            if (mixed && any) {
                // rows that see a NaN: the product of "sees" and "is NaN" is positive there
                uint32_t see[4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const int key = key0 + kk * 16 + nt * 8 + 2 * j;
                        const bool s0v = key <= pos[h] && key > pos[h] - p.window;
                        const bool s1v = key + 1 <= pos[h] && key + 1 > pos[h] - p.window;
                        see[2 * nt + h] = (s0v ? 0x3c00u : 0u) | (s1v ? 0x3c000000u : 0u);
                    }
#pragma unroll
                for (int x = 0; x < kNt / 4; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        float n[4] = {};
                        const uint32_t sel = 8 * y;
                        const uint32_t b0 = ((bad[0][x] >> sel) & 1 ? 0x3c00u : 0u) | ((bad[1][x] >> sel) & 1 ? 0x3c000000u : 0u);
                        const uint32_t b1 = ((bad[2][x] >> sel) & 1 ? 0x3c00u : 0u) | ((bad[3][x] >> sel) & 1 ? 0x3c000000u : 0u);
                        mma_f16(n, see, b0, b1);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n[e] > 0.f) acc[4 * x + y][e] = __uint_as_float(0x7fc00000u);
                    }
            }
        }

        // ---------------------------------------------------------------- the unit's end, or the piece's
        const bool last = cc.tile + 1 == cc.g.tiles;
        if (last || it + 1 == count) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                if (j == 0) lsum[warp][quad + 8 * h] = l[h];
            }
            __syncthreads();
            const bool whole = unit_first && last;
            float *slot = parts + ((size_t)cta * 2 + (unit_first ? 1 : 0)) * part_floats(D);
            if (!whole && unit_first) {
                // the piece ends inside the unit, which began here: the later CTAs with a part of it
                const long long unit_end = end + (cc.g.tiles - 1 - cc.tile);
                plan = {piece_of(total, unit_end - 1, n_ctas) - cta + 1, cc.seq, cc.unit, cu.rows};
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = quad + 8 * h;
                const float lt = (lsum[0][r] + lsum[1][r]) + (lsum[2][r] + lsum[3][r]);
                if (r >= cu.rows) continue;
                const int c0 = warp * kSlice + 2 * kNt * j;  // 2 kNt contiguous channels
                if (whole) {
                    const float o = lt == 0.f ? 0.f : sm100::ex2_approx(finite_or_0(mv[h])) / lt;
                    uint32_t w[kNt];
#pragma unroll
                    for (int t = 0; t < kNt; ++t) {
                        const int e = 2 * t / kNt, x = 2 * t % kNt;  // channel 2 t of the thread's 2 kNt
                        w[t] = pack_bf16(acc[x][2 * h + e] * o, acc[x + 1][2 * h + e] * o);
                    }
                    const int row = cu.row + r;
                    uint4 *dst = reinterpret_cast<uint4 *>(
                        p.out + ((size_t)(cc.g.row0 + row / G) * b.H + cu.head * G + row % G) * D + c0);
#pragma unroll
                    for (int t = 0; t < kNt / 4; ++t) dst[t] = make_uint4(w[4 * t], w[4 * t + 1], w[4 * t + 2], w[4 * t + 3]);
                } else {
                    if (warp == 0 && j == 0) *reinterpret_cast<float4 *>(slot + 4 * r) = make_float4(m[h], mv[h], lt, 0.f);
                    float4 *dst = reinterpret_cast<float4 *>(slot + 4 * kRowTile + r * D + c0);
#pragma unroll
                    for (int t = 0; t < kNt / 2; ++t) {
                        const int e = 4 * t / kNt, x = 4 * t % kNt;
                        dst[t] = make_float4(acc[x][2 * h + e], acc[x + 1][2 * h + e], acc[x + 2][2 * h + e], acc[x + 3][2 * h + e]);
                    }
                }
            }
            start = true;
        }
        if (it + 1 < count) advance(p, cc);
    }
    if (tid == 0) plans[cta] = plan;
}

// Joins the parts of the units that were cut: an item is one row and 64 channels of such a unit; warps take
// every eighth part, in an order that does not depend on which CTA was done first.
template <int D>
__global__ void __launch_bounds__(256) rglru_paged_combine_kernel(const AttendArgs p, int n)
{
    constexpr int kSlices = D / 64;
    __shared__ int first[kMaxCtas + 1];
    __shared__ int sums[8];
    __shared__ float2 o[8][32];
    __shared__ float red[8][3];
    const Batch &b = p.b;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = b.H / b.Hkv;
    const Plan *plans = reinterpret_cast<const Plan *>(reinterpret_cast<const char *>(b.ws) + kWsHeaderBytes);
    const float *parts =
        reinterpret_cast<const float *>(reinterpret_cast<const char *>(b.ws) + kWsHeaderBytes + align_up_d(kPlanBytes, 256));
    int have[2], sum = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int c = 2 * tid + k;
        have[k] = c < n && plans[c].parts > 1 ? plans[c].rows * kSlices : 0;
        sum += have[k];
    }
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += v;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int at = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w < warp) at += sums[w];
        total += sums[w];
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (2 * tid + k <= n) first[2 * tid + k] = at;
        at += have[k];
    }
    __syncthreads();
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        int lo = 0, hi = n;  // the last c with first[c] <= item
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (first[mid] <= item) lo = mid; else hi = mid;
        }
        const int c = lo, r = (item - first[c]) / kSlices, ch = (item - first[c]) % kSlices * 64;
        const Plan pl = plans[c];
        auto part = [&](int k) { return parts + ((size_t)(c + k) * 2 + (k == 0)) * part_floats(D); };
        // m over the parts, then mv relative to it
        float m = -INFINITY, mv = -INFINITY;
        for (int k = tid; k < pl.parts; k += 256) m = fmaxf(m, part(k)[4 * r]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if (lane == 0) red[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w][0]);
        const float mz = finite_or_0(m);
        for (int k = tid; k < pl.parts; k += 256) mv = fmaxf(mv, part(k)[4 * r + 1] + (part(k)[4 * r] - mz));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, d));
        if (lane == 0) red[warp][1] = mv;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) mv = fmaxf(mv, red[w][1]);
        const float vz = finite_or_0(mv);
        float l = 0.f;
        float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int k = warp; k < pl.parts; k += 8) {
            const float4 st = *reinterpret_cast<const float4 *>(part(k) + 4 * r);
            const float2 v = *reinterpret_cast<const float2 *>(part(k) + 4 * kRowTile + r * D + ch + 2 * lane);
            const float f = sm100::ex2_approx(st.y + (st.x - mz) - vz);
            l += st.z * sm100::ex2_approx(st.x - mz);
            sum2.x += v.x * f, sum2.y += v.y * f;
        }
        o[warp][lane] = sum2;
        if (lane == 0) red[warp][2] = l;
        __syncthreads();
        if (warp == 0) {
            float lt = 0.f;
            float2 t = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 8; ++w) lt += red[w][2], t.x += o[w][lane].x, t.y += o[w][lane].y;
            const float f = lt == 0.f ? 0.f : sm100::ex2_approx(vz) / lt;
            const Geometry g = geometry(p, pl.seq);
            const int per_head = g.units / b.Hkv, row = pl.unit % per_head * kRowTile + r, head = pl.unit / per_head;
            *reinterpret_cast<uint32_t *>(p.out + ((size_t)(g.row0 + row / G) * b.H + head * G + row % G) * D + ch + 2 * lane) =
                pack_bf16(t.x * f, t.y * f);
        }
        __syncthreads();
    }
}

template <int D>
rglru_status launch(const AttendArgs &p, cudaStream_t stream)
{
    using C = Cfg<D>;
    static PerDeviceFlag flag;
    const rglru_status st =
        set_smem_limit_once(reinterpret_cast<const void *>(rglru_paged_attention_kernel<D>), C::kSmem, flag);
    if (st != RGLRU_OK) return st;
    const int grid = kSms * C::kCtasPerSm;
    rglru_paged_attention_kernel<D><<<grid, kThreads, C::kSmem, stream>>>(p);
    rglru_paged_combine_kernel<D><<<kSms * 2, 256, 0, stream>>>(p, grid);
    return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace rglru

using namespace rglru;

extern "C" {

RGLRU_API size_t rglru_paged_attention_workspace_size(int H, int Hkv, int head_dim)
{
    if (H < 1 || Hkv < 1 || H > 256 || Hkv > 64 || H % Hkv != 0 || (head_dim != 128 && head_dim != 256)) return 0;
    return attention_bytes(head_dim);
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
    return head_dim == 256 ? launch<256>(p, stream) : launch<128>(p, stream);
}

}  // extern "C"
