// paged_attention.cu -- causal sliding-window attention of the new tokens over a paged 8-bit cache.
//
//   out[t, h] = sum_p softmax_p(scale * q[t, h] . k[p]) v[p],   pos_t - window < p <= pos_t
//
// with k[p], v[p] = code * scale of p's page and head.  Positions outside a row's range are never read or never
// weighted; a row without any key gives zeros.  One pass over the keys with the softmax's running maximum and sum.
// Short runs take 16 rows at a time (mma.sync, bound by the cache's bytes), chunks 128 (tcgen05).
#include "paged.cuh"
#include "sm100.cuh"

#include <climits>

namespace rglru {
namespace {

using paged::Batch;

struct AttendArgs {
    Batch b;
    int window;
    float scale;
    float top, raise;  // 128 rows at a time: log2 of the largest P at its reference, and how far P may pass it
    int withhold;  // test hook: 1 + the CTA that keeps back the arrival on its first tile of v, 0 = none
    const __nv_bfloat16 *q;
    const uint8_t *k, *v;
    const float *ks, *vs;
    __nv_bfloat16 *out;
};

// ------------------------------------------------------------------------------------------------ schedule
// A unit is 16 rows (row = token * G + head in the group, G = H / Hkv) of one sequence and key/value head;
// its work is the 64-key tiles of the sequence's attended range.  All units' tiles form one line, cut into
// gridDim.x equal pieces: long and short sequences balance, and one long sequence spreads over every SM.
constexpr int kRowTile = 16, kKeyTile = 64, kMinTiles = 2, kManyTiles = 10;
constexpr int kConsumers = 128, kThreads = kConsumers + 32;
constexpr int kSms = 148, kMaxCtas = 3 * kSms;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr float kTop = 15.f;  // log2 of the largest P (f16 ends at 2^16)
constexpr size_t align_up_d(size_t v, size_t a) { return (v + a - 1) / a * a; }

struct Meta {                // of one tile in the ring, written by the producer
    float ks[4], lv[4];      // per 16 keys: k's scale, log2 of v's
    int ok;                  // bit q: the 16 keys of group q can be attended by some row
    int key0;                // position of the tile's first key
    int flags;               // 1: first tile of its unit, 2: last tile of its unit
    int row0, ctx;           // the sequence: first row, tokens before the call
    int head, row, rows, left;  // the unit; tiles of it after this one
};

template <int D>
struct Cfg {
    // three CTAs with few slots rather than two with more: a tile's chain is latency (256 sequences over 2048 keys, D 256,
    // behind a flush of L2: 70.0 us against 72.4; two CTAs with three slots 71.6; the same over 2000 keys of four heads of
    // 128, 200 sequences: 86 against 100)
    static constexpr int kCtasPerSm = 3;
    static constexpr int kHalf = kKeyTile * 128;      // 64 keys x 128 channels (one swizzled box column)
    static constexpr int kSlotBytes = kKeyTile * D;   // k or v of a tile
    static constexpr int kSlots = D == 256 ? 3 : 7;
    static constexpr int kQBytes = kRowTile * D * 2;  // a unit's rows as they come, and as f16 operands
    static constexpr int kSmem = kSlots * kSlotBytes + 2 * kQBytes + 1024;
};
constexpr int kMeta = 8;  // k of tile t + kSlots - 1 takes the slot of v of tile t or a later one

struct Plan {  // the unit that begins in a CTA's piece and does not end there: its parts, rows and first row's place
    short parts, rows;
    int row0, row, head;  // the sequence's first row; the unit's first (token * G + head in group), its key/value head
};
// Workspace: header, plans, then partial results, R rows each: m, mv, l, lost (float4) and O [R][D].  The 16-row
// kernel has two a CTA (slot 2 c: a unit begun in an earlier CTA; 2 c + 1: one begun here), the 128-row kernel one.
constexpr int kWideRows = 128;
constexpr size_t kPlanBytes = (size_t)kMaxCtas * sizeof(Plan);
__host__ __device__ constexpr size_t part_floats(int rows, int D) { return (size_t)rows * (4 + D); }
inline size_t attention_bytes(int D)
{
    const size_t few = (size_t)kMaxCtas * 2 * part_floats(kRowTile, D), wide = kSms * part_floats(kWideRows, D);
    return kWsHeaderBytes + align_up_d(kPlanBytes, 256) + (few > wide ? few : wide) * 4;
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

// ------------------------------------------------------------------------------------------------ pieces
// A wait gives up after 2 s, or once another of its CTA has (`lost`, in shared memory); the first to give up records it.
// Who gave up waits no more and passes the CTA's barriers with the others, but arrives on no mbarrier (the 128-row
// kernel's softmax threads excepted) and starts no copy or product: an arrival stands for a wait that was won, so the
// others run out of theirs as well, and none takes a slot that is half full for a full one.  The rows held up are not
// written, and the CTA's parts say that they are not there.
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, WsHeader *ws, volatile int *lost, int where)
{
    const uint64_t t0 = sm100::globaltimer();
    do {
        if (sm100::mbar_try_wait_sleep(bar, parity, 20000u)) return true;
        if (*lost) return false;
    } while (sm100::globaltimer() - t0 < kTimeoutNs);
    *lost = 1;
    __threadfence_block();
    atomicCAS(&ws->status, 0, (int)RGLRU_ERR_TIMEOUT);
    atomicCAS(&ws->detail, 0, (int)(blockIdx.x << 8) | (where + 1));
    return false;
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, WsHeader *ws, volatile int *lost, int where)
{
    return sm100::mbar_try_wait(bar, parity) || wait_slow(bar, parity, ws, lost, where);
}
// For what is in flight when a CTA ends, whether or not a wait was lost (2 s also where the test hook keeps the arrival back
// that would end the wait: the copy has landed by then).
__device__ __noinline__ void drain_wait(uint64_t *bar, uint32_t parity)
{
    const uint64_t t0 = sm100::globaltimer();
    while (!sm100::mbar_try_wait_sleep(bar, parity, 20000u) && sm100::globaltimer() - t0 < kTimeoutNs) {
    }
}
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// barrier `id` of `count` threads; whether any of them has x
__device__ __forceinline__ bool bar_any(int id, int count, bool x)
{
    int any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                 : "=r"(any)
                 : "r"((int)x), "r"(id), "r"(count)
                 : "memory");
    return any != 0;
}
__device__ __forceinline__ void mbar_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(sm100::smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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
// One producer warp and four consumer warps.  The producer walks the piece's tiles, looks pages and scales up for eight
// tiles at a time, and fetches the codes by TMA (128-byte swizzle) into a ring of slots, in the order of their use: k of
// tile 0, then k of tile t + 1 and v of tile t.  S = Q K^T: consumer warp w has the 16 keys of group w (one page, so one
// scale) and all 16 rows; the row maxima meet in shared memory, P goes there as f16 in the layout of an mma operand, and
// O += P V: warp w has channels w D/4 .. of all keys, so that O is never summed across warps.  S of tile t + 1 is
// computed next to the softmax of tile t: one tile's chain (two barriers, 16 dependent mma, exponentials) is latency,
// and the next one's products fill it.
// Codes turn into f16 operands exactly, in registers (the e4m3 form of this mma is slower: it runs as conversions and
// f16 products, 5.0 cycles against 2.2).  k's scale multiplies the scores; v's enters the exponent: P holds
// 2^(s - m + log2 vs - mv) with mv the running maximum of s - m + log2 vs less 15, beside the softmax's own maximum m and
// sum l = sum 2^(s - m), so that P keeps f16's bits whatever the pages' scales (mv is relative to m: a large score would
// swallow log2 vs).  The 15 put the largest P at f16's upper end: a key keeps its bits down to 2^-29 of the largest and is
// off by at most 2^-40 of it below.
// Measured, 10 heads of 256 to one key head: 256 sequences over 2048 keys 65 us with the launch and the join (4.1 TB/s
// of codes; a CTA's tile takes 1.7 us and more also out of L2, which is the consumers' chain); one sequence over 131072
// keys 29 us, of which 6 to the first tile's end and 7 the join.
//
// Columns of an 8-key mma tile: column n is key n for even n, n ^ 4 for odd n.  With the swizzle (16-byte chunk c of
// row r sits at c ^ (r & 7)) both the 16-byte reads of k (two rows a phase) and the 8-byte reads of v (four
// rows a phase) then touch every bank once.
template <int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::kCtasPerSm)
rglru_paged_attention_kernel(const AttendArgs p, const __grid_constant__ CUtensorMap tm_k,
                             const __grid_constant__ CUtensorMap tm_v)
{
    using C = Cfg<D>;
    constexpr int kSlots = C::kSlots, kKb = D / 64, kNt = D / 32, kSlice = D / 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qbuf = ring + kSlots * C::kSlotBytes;                   // the next unit's rows, bf16
    uint4 *qfrag = reinterpret_cast<uint4 *>(qbuf + C::kQBytes);     // this unit's as mma operands: [D / 16][32 lanes]
    __shared__ Meta meta[kMeta];
    __shared__ uint64_t full[kSlots], empty[kSlots], q_full, q_empty;
    __shared__ float4 wmax[kRowTile], wlv;
    __shared__ float qscale[kRowTile];
    __shared__ uint4 pbuf[4][32];
    __shared__ float lsum[4][kRowTile];
    __shared__ long long scan[kThreads / 32];
    __shared__ int where[3], lost;
    __shared__ Geometry where_g;
    const Batch &b = p.b;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = b.H / b.Hkv;
    sm100::griddep_launch_dependents();  // the joining kernel waits for this grid's end by itself

    // ---------------------------------------------------------------- this CTA's piece of the line
    if (tid < kSlots) {
        sm100::mbar_init(full + tid, 1);
        sm100::mbar_init(empty + tid, kConsumers / 32);
        if (tid == 0) sm100::mbar_init(&q_full, 1), sm100::mbar_init(&q_empty, kConsumers / 32), lost = 0;
        sm100::mbar_fence_init();
    }
    const int per = (b.S + kThreads - 1) / kThreads, s0 = min(b.S, tid * per), s1 = min(b.S, s0 + per);
    long long mine = 0;
    Geometry g01[2] = {};  // of this thread's first two sequences: batches of up to 2 * kThreads are read once
    for (int i = s0; i < s1; ++i) {
        const Geometry g = geometry(p, i);
        if (i == s0) g01[0] = g;
        if (i == s0 + 1) g01[1] = g;
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
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    before += inc - mine;
    const int n_ctas = (int)min((long long)gridDim.x, (total + kMinTiles - 1) / kMinTiles), cta = blockIdx.x;
    Plan *plans = reinterpret_cast<Plan *>(reinterpret_cast<char *>(b.ws) + kWsHeaderBytes);
    if (cta >= n_ctas) {
        if (tid == 0) plans[cta] = {0, 0, 0, 0, 0};
        return;
    }
    const long long begin = piece_begin(total, cta, n_ctas), end = piece_begin(total, cta + 1, n_ctas);
    const int count = (int)(end - begin);
    if (begin >= before && begin < before + mine) {
        long long at = before;
        for (int i = s0; i < s1; ++i) {
            const Geometry g = i == s0 ? g01[0] : i == s0 + 1 ? g01[1] : geometry(p, i);
            const long long c = (long long)g.tiles * g.units;
            if (begin < at + c) {
                where_g = g;
                where[0] = i;
                where[1] = (int)((begin - at) / g.tiles);
                where[2] = (int)((begin - at) % g.tiles);
                break;
            }
            at += c;
        }
    }
    __syncthreads();

    if (warp == kConsumers / 32) {
        // ---------------------------------------------------------------- producer
        const int page_shift = 31 - __clz(b.page), box = min(b.page, kKeyTile);
        int seq = where[0], unit = where[1], tile = where[2], it = 0, units = 0, slot = 0, uses = 0;
        Geometry g = where_g;
        // a slot to fill: `boxes` of this lane's c1 (lanes 0 .. 3 with `leads`), k or v; false when the wait for it was lost
        auto fill = [&](const CUtensorMap *tm, bool leads, int c1) {
            if (uses > 0 && !__all_sync(0xffffffffu, wait(empty + slot, (uint32_t)(uses - 1) & 1u, b.ws, &lost, 0))) return false;
            const uint32_t n = (uint32_t)__popc(__ballot_sync(0xffffffffu, leads));
            if (lane == 0) mbar_expect(full + slot, n * (uint32_t)box * D);
            __syncwarp();
            if (leads) {
                uint8_t *dst = ring + slot * C::kSlotBytes + 16 * lane * 128;
#pragma unroll
                for (int x = 0; x < D / 128; ++x) sm100::tma_load_2d(dst + x * C::kHalf, tm, full + slot, x * 128, c1);
            }
            return true;
        };
        auto filled = [&](bool first_v = false) {
            __syncwarp();
            if (lane == 0 && !(first_v && p.withhold == cta + 1)) sm100::mbar_arrive(full + slot);
            if (++slot == kSlots) slot = 0, ++uses;
        };
        bool v_leads = false;  // of the tile whose v comes next
        int v_c1 = 0;
        auto walk = [&]() {
            for (; it < count;) {
                const int per_head = g.units / b.Hkv, head = unit / per_head, row = unit % per_head * kRowTile;
                const int rows = min(kRowTile, g.n * G - row);
                const int lo = max(0, g.ctx + row / G - p.window + 1), hi = g.ctx + (row + rows - 1) / G + 1;
                const int tiles = min(g.tiles - tile, count - it);  // of this unit, in this piece
                // its query rows, once the consumers have turned the last unit's into operands
                if (units > 0 && !__all_sync(0xffffffffu, wait(&q_empty, (uint32_t)(units - 1) & 1u, b.ws, &lost, 3))) return;
                if (lane == 0) sm100::mbar_arrive_expect_tx(&q_full, (uint32_t)rows * D * 2);
                __syncwarp();
                if (lane < rows) {
                    const int r = row + lane;
                    sm100::bulk_load(qbuf + lane * D * 2, p.q + ((size_t)(g.row0 + r / G) * b.H + head * G + r % G) * D, D * 2,
                                     &q_full);
                }
                ++units;
                for (int t0 = 0; t0 < tiles; t0 += 8) {
                    // lane: group lane % 4 of tile t0 + lane / 4
                    const int q = lane & 3, key0 = (g.tile0 + tile + t0 + (lane >> 2)) * kKeyTile, key = key0 + 16 * q;
                    int page = -1;
                    float ks = 0.f, vs = 0.f;
                    const int bk = key & ~(box - 1);  // the box's first key
                    const bool wanted = t0 + (lane >> 2) < tiles && bk + box > lo && bk < hi;
                    if (wanted) {
                        page = b.table[(size_t)seq * b.max_pages + (key >> page_shift)];
                        if (page < 0 || page >= b.num_pages) {
                            paged::record_invalid(b.ws);
                            page = -1;
                        }
                    }
                    const size_t at = (size_t)max(page, 0) * b.Hkv + head;
                    if (page >= 0) ks = p.ks[at], vs = p.vs[at];
                    const bool ok = page >= 0 && key + 16 > lo && key < hi;
                    const int leads = page >= 0 && key == bk;
                    const uint32_t oks = __ballot_sync(0xffffffffu, ok);
                    const int c1 = (int)((at << page_shift) + (key & (b.page - 1)));
                    for (int t = 0; t < min(8, tiles - t0); ++t, ++it) {
                        const bool k_leads = __shfl_sync(0xffffffffu, leads, 4 * t + q) != 0 && lane < 4;
                        const int k_c1 = __shfl_sync(0xffffffffu, c1, 4 * t + q);
                        if (!fill(&tm_k, k_leads, k_c1)) return;
                        if ((lane >> 2) == t) {
                            Meta &mt = meta[it % kMeta];
                            mt.ks[q] = ks;
                            mt.lv[q] = ok ? log2f(vs) : 0.f;
                            if (q == 0) {
                                mt.ok = (int)((oks >> (4 * t)) & 0xfu);
                                mt.key0 = key0;
                                const int left = g.tiles - 1 - (tile + t0 + t);
                                mt.flags = (tile + t0 + t == 0 ? 1 : 0) | (left == 0 ? 2 : 0) | (t0 + t == 0 ? 4 : 0);
                                mt.row0 = g.row0, mt.ctx = g.ctx, mt.head = head;
                                mt.row = row, mt.rows = rows, mt.left = left;
                            }
                        }
                        filled();
                        if (it > 0) {
                            if (!fill(&tm_v, v_leads, v_c1)) return;
                            filled(it == 1);
                        }
                        v_leads = k_leads, v_c1 = k_c1;
                    }
                }
                tile = 0;
                ++unit;
                if (unit == g.units && it < count) {
                    unit = 0;
                    do g = geometry(p, ++seq); while (g.units == 0);
                }
            }
            if (fill(&tm_v, v_leads, v_c1)) filled(count == 1);
        };
        walk();
        // no copy is in flight when the CTA ends
        for (int k = 0; k < kSlots; ++k) {  // the slots' last uses, oldest first
            if (uses > 0 || k < slot) {
                const int x = uses > 0 ? (slot + k) % kSlots : k;
                drain_wait(full + x, (uint32_t)(x < slot ? uses : uses - 1) & 1u);
            }
        }
        if (units > 0) drain_wait(&q_full, (uint32_t)(units - 1) & 1u);
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int quad = lane >> 2, j = lane & 3;
    float *parts = reinterpret_cast<float *>(reinterpret_cast<char *>(b.ws) + kWsHeaderBytes + align_up_d(kPlanBytes, 256));
    Plan plan = {0, 0, 0, 0, 0};
    const int kq = quad & 1 ? quad ^ 4 : quad;                 // this thread's key in an 8-key tile (row of k)
    const int je = 2 * j, jo = (2 * j + 1) ^ 4;                // keys of the score columns 2j, 2j + 1 (rows of v)
    const int k_off = (warp * 16 + kq) * 128 + ((j ^ kq) << 4);
    // this warp's channels of v: first byte of the thread's kNt, in its 128-byte row
    const int v_byte = (warp * kSlice + quad * kNt) & 127;
    const int v_half = (warp * kSlice) / 128 * C::kHalf;
    const int v_off[2] = {v_half + je * 128 + (((v_byte >> 4) ^ (je & 7)) << 4) + (v_byte & 15),
                          v_half + jo * 128 + (((v_byte >> 4) ^ (jo & 7)) << 4) + (v_byte & 15)};
    float acc[kNt][4], m[2], mv[2], l[2], qs[2], s[2][4];
    int pos[2];
    int pos_first = 0, pos_last = 0, unit_first = 0, slot = 0;
    uint32_t phase = 0;
    bool alive = true;  // this thread has won all its waits
    auto take = [&]() {  // the next slot of the ring, full
        if (alive) alive = wait(full + slot, phase, b.ws, &lost, 2);
        return ring + slot * C::kSlotBytes;
    };
    auto release = [&]() {
        __syncwarp();
        if (lane == 0 && alive) sm100::mbar_arrive(empty + slot);
        if (++slot == kSlots) slot = 0, phase ^= 1u;
    };
    // A unit's rows as f16 operands, each row times a power of two that brings its largest exponent to 2^13: every bf16
    // down to 2^-27 of it is a normal f16.  Warp w converts the 64 channels of step w.
    auto load_queries = [&](int rows, uint32_t turn) {
        if (alive) alive = wait(&q_full, turn & 1u, b.ws, &lost, 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = quad + 8 * h;
            const bool live = r < rows;
            const uint4 *src = reinterpret_cast<const uint4 *>(qbuf + r * D * 2 + 32 * j);
            uint32_t top = 0;
#pragma unroll
            for (int kb = 0; kb < 2 * kKb; ++kb) {
                const uint4 v = live ? src[(kb >> 1) * 8 + (kb & 1)] : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) top = max(top, max((w[x] << 16) & 0x7f800000u, w[x] & 0x7f800000u));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            int e = max(-126, (int)(top >> 23) - 127 - 13);
            if (top == 0) e = 0;
            const float f = __uint_as_float((uint32_t)(127 - e) << 23);
            if (warp == 0 && j == 0)  // a row with an infinity or NaN is NaN
                qscale[r] = top == 0x7f800000u ? __uint_as_float(0x7fc00000u)
                                               : p.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
            if (warp < kKb) {
                const uint4 v0 = live ? src[warp * 8] : make_uint4(0, 0, 0, 0), v1 = live ? src[warp * 8 + 1] : make_uint4(0, 0, 0, 0);
                const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t *dst = reinterpret_cast<uint32_t *>(qfrag + (warp * 4 + x) * 32 + lane);
                    dst[h] = pack_f16(bf_lo(w[2 * x]) * f, bf_hi(w[2 * x]) * f);
                    dst[2 + h] = pack_f16(bf_lo(w[2 * x + 1]) * f, bf_hi(w[2 * x + 1]) * f);
                }
            }
        }
        __syncwarp();
        if (lane == 0 && alive) sm100::mbar_arrive(&q_empty);
        consumer_sync();
    };
    // raw scores of this warp's 16 keys of the next tile
    auto scores = [&](float (&s)[2][4]) {
        const uint8_t *st = take();
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb) {
            uint32_t w[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const uint4 c = *reinterpret_cast<const uint4 *>(st + (kb >> 1) * C::kHalf + nt * 1024 +
                                                                 (kb & 1 ? k_off ^ 64 : k_off));
                w[nt][0] = c.x, w[nt][1] = c.y, w[nt][2] = c.z, w[nt][3] = c.w;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint4 qa = qfrag[(kb * 4 + x) * 32 + lane];
                const uint32_t a[4] = {qa.x, qa.y, qa.z, qa.w};
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    uint32_t b0, b1;
                    e4m3::to_f16x2x2(w[nt][x], b0, b1);
                    mma_f16(s[nt], a, b0, b1);
                }
            }
        }
        release();
    };
    uint32_t units = 0;
    if (alive) alive = wait(full, 0, b.ws, &lost, 2);  // tile 0's k, and with it its meta
    load_queries(meta[0].rows, units++);
    scores(s);
    // Whether some consumer has lost a wait, settled at a barrier: the branches below that hold barriers go by a tile's
    // meta, which only a won wait has brought.
    bool held_up = bar_any(1, kConsumers, !alive);
    for (int it = 0; it < count && !held_up; ++it) {
        const Meta &mt = meta[it % kMeta];
        if (mt.flags & 4) {  // the unit's first tile in this piece: its sums are empty
            unit_first = mt.flags & 1;
            pos_first = mt.ctx + mt.row / G;
            pos_last = mt.ctx + (mt.row + mt.rows - 1) / G;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = quad + 8 * h;
                pos[h] = mt.ctx + (mt.row + min(r, mt.rows - 1)) / G;
                qs[h] = qscale[r];
                m[h] = mv[h] = -INFINITY;
                l[h] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < kNt; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
        }
        const int key0 = mt.key0, okm = mt.ok;
        const float ks = mt.ks[warp], lv = mt.lv[warp];
        // whether some key of the tile is outside some row's range, or was not loaded
        const bool edge = okm != 15 || key0 < pos_last - p.window + 1 || key0 + kKeyTile - 1 > pos_first;
        float tmax[2] = {-INFINITY, -INFINITY};
        const float qk[2] = {qs[0] * ks, qs[1] * ks};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] *= qk[e >> 1];
        if (edge) {
            const bool ok = (okm >> warp) & 1;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + warp * 16 + nt * 8 + (e & 1 ? jo : je);
                    if (!ok || key > pos[e >> 1] || key <= pos[e >> 1] - p.window) s[nt][e] = -INFINITY;
                }
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) tmax[e >> 1] = fmaxf(tmax[e >> 1], s[nt][e]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            tmax[h] = fmaxf(tmax[h], __shfl_xor_sync(0xffffffffu, tmax[h], 1));
            tmax[h] = fmaxf(tmax[h], __shfl_xor_sync(0xffffffffu, tmax[h], 2));
            if (j == 0) reinterpret_cast<float *>(&wmax[quad + 8 * h])[warp] = tmax[h];
        }
        if (lane == 0) reinterpret_cast<float *>(&wlv)[warp] = lv - kTop;
        consumer_sync();
        float sn[2][4] = {};
        if (it + 1 < count) {
            if (mt.left == 0) {  // another unit follows: every warp is done with the old operands
                if (alive) alive = wait(full + slot, phase, b.ws, &lost, 2);
                load_queries(meta[(it + 1) % kMeta].rows, units++);
            }
            scores(sn);
        }
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
            const float d = lv - vz;
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
        held_up = bar_any(1, kConsumers, !alive);  // P is there, and with it the next tile's meta
        if (held_up) break;
        const uint8_t *st = take();

        // O += P V for this warp's channels: 16 keys a step, the thread's kNt channels of four of them
        auto load_v = [&](int kk, uint32_t (&v)[4][kNt / 4]) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint8_t *src = st + v_off[q & 1] + kk * 2048 + (q >> 1) * 1024;
                if (kNt == 8) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(src);
                    v[q][0] = w.x, v[q][kNt / 4 - 1] = w.y;
                } else {
                    v[q][0] = *reinterpret_cast<const uint32_t *>(src);
                }
            }
        };
        auto times_v = [&](int kk, const uint32_t (&v)[4][kNt / 4]) {
            const uint4 pa = pbuf[kk][lane];
            const uint32_t a[4] = {pa.x, pa.y, pa.z, pa.w};
#pragma unroll
            for (int x = 0; x < kNt / 4; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t c0[2], c1[2];
                    e4m3::to_f16x2x2(__byte_perm(v[0][x], v[1][x], y ? 0x7362 : 0x5140), c0[0], c0[1]);
                    e4m3::to_f16x2x2(__byte_perm(v[2][x], v[3][x], y ? 0x7362 : 0x5140), c1[0], c1[1]);
                    mma_f16(acc[4 * x + 2 * y], a, c0[0], c1[0]);
                    mma_f16(acc[4 * x + 2 * y + 1], a, c0[1], c1[1]);
                }
        };
        if (!edge) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t v[4][kNt / 4];
                load_v(kk, v);
                times_v(kk, v);
            }
        } else {
            // slots that no row attends may hold anything, and rows may see different keys: a NaN may only reach the
            // rows that see its key, so it is taken out of the product
#pragma unroll 1
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t v[4][kNt / 4], bad[4][kNt / 4], any = 0;
                load_v(kk, v);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int x = 0; x < kNt / 4; ++x) {
                        bad[q][x] = nan_bytes(v[q][x]);
                        v[q][x] &= ~bad[q][x];
                        any |= bad[q][x];
                    }
                times_v(kk, v);
                if (!__any_sync(0xffffffffu, any != 0)) continue;
                // rows that see a NaN: the product of "sees" and "is NaN" is positive there
                uint32_t see[4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        uint32_t w = 0;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = key0 + kk * 16 + nt * 8 + (e ? jo : je);
                            if (((okm >> kk) & 1) && key <= pos[h] && key > pos[h] - p.window) w |= 0x3c00u << (16 * e);
                        }
                        see[2 * nt + h] = w;
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
        const bool last = (mt.flags & 2) != 0;
        if (last || it + 1 == count) {
            const int urow = mt.row, urows = mt.rows, row0 = mt.row0, head = mt.head;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                if (j == 0) lsum[warp][quad + 8 * h] = l[h];
            }
            held_up = bar_any(1, kConsumers, !alive);
            const bool whole = unit_first && last;
            float *slot = parts + ((size_t)cta * 2 + (unit_first ? 1 : 0)) * part_floats(kRowTile, D);
            if (!whole && unit_first)  // the unit began here and goes on: the later CTAs with a part of it
                plan = {(short)(piece_of(total, end + mt.left - 1, n_ctas) - cta + 1), (short)urows, row0, urow, head};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = quad + 8 * h;
                const float lt = (lsum[0][r] + lsum[1][r]) + (lsum[2][r] + lsum[3][r]);
                if (r >= urows || held_up) continue;
                const int c0 = warp * kSlice + 2 * kNt * j;  // 2 kNt contiguous channels
                if (whole) {
                    const float o = lt == 0.f ? 0.f : 1.f / lt, o2 = sm100::ex2_approx(finite_or_0(mv[h]));
                    uint32_t w[kNt];
#pragma unroll
                    for (int t = 0; t < kNt; ++t) {
                        const int e = 2 * t / kNt, x = 2 * t % kNt;  // channel 2 t of the thread's 2 kNt
                        w[t] = pack_bf16(acc[x][2 * h + e] * o * o2, acc[x + 1][2 * h + e] * o * o2);
                    }
                    const int row = urow + r;
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + ((size_t)(row0 + row / G) * b.H + head * G + row % G) * D + c0);
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
        }
        release();  // v's slot, and with it the tile's meta
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = sn[nt][e];
    }
    if (held_up) {
        plan = {0, 0, 0, 0, 0};
        for (int r = tid; r < 2 * kRowTile; r += kConsumers)
            *reinterpret_cast<float4 *>(parts + ((size_t)cta * 2 + r / kRowTile) * part_floats(kRowTile, D) + 4 * (r % kRowTile)) =
                make_float4(0.f, 0.f, 0.f, 1.f);
    }
    if (tid == 0) plans[cta] = plan;
}

// Joins the parts of the units that were cut, in their order along the line, whichever CTA was done first.  Units of few
// parts: a warp takes a row.  Units of many parts (a long sequence over many SMs): a CTA takes 64 channels of a row, its
// half warps every 64th part.  Each CTA lists the items from the plans (one scan) and takes every gridDim.x-th.  Latency
// bound: 6 to 8 us, of which a launch alone is 3.
constexpr int kFewParts = 24, kJoinThreads = 1024;

// R: rows of a part
template <int D, int R>
__global__ void __launch_bounds__(kJoinThreads) rglru_paged_combine_kernel(const AttendArgs p, int n)
{
    constexpr int kSlices = D / 64, kVec = D / 128, kWarps = kJoinThreads / 32;
    constexpr int kBatch = (kMaxCtas + 2 * kWarps - 1) / (2 * kWarps);  // parts a half warp takes of a long unit
    __shared__ int first[2][kMaxCtas + 1];  // running item counts: rows of short units, slices of long ones
    __shared__ int sums[2][kWarps];
    __shared__ Plan list[kMaxCtas];
    __shared__ float4 o[kWarps][16];
    __shared__ float red[kWarps][3];
    const Batch &b = p.b;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = b.H / b.Hkv;
    const Plan *plans = reinterpret_cast<const Plan *>(reinterpret_cast<const char *>(b.ws) + kWsHeaderBytes);
    const float *parts =
        reinterpret_cast<const float *>(reinterpret_cast<const char *>(b.ws) + kWsHeaderBytes + align_up_d(kPlanBytes, 256));
    sm100::griddep_wait();
    int have[2], inc[2];
    {
        Plan pl = {0, 0, 0, 0, 0};
        if (tid < n) list[tid] = pl = plans[tid];
        have[0] = pl.parts > 1 && pl.parts <= kFewParts ? pl.rows : 0;
        have[1] = pl.parts > kFewParts ? pl.rows * kSlices : 0;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        inc[x] = have[x];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc[x], d);
            if (lane >= d) inc[x] += v;
        }
        if (lane == 31) sums[x][warp] = inc[x];
    }
    __syncthreads();
    int total[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        int at = lane < kWarps ? sums[x][lane] : 0;
        int before = lane < warp ? at : 0;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            at += __shfl_xor_sync(0xffffffffu, at, d);
            before += __shfl_xor_sync(0xffffffffu, before, d);
        }
        total[x] = at;
        if (tid <= n) first[x][tid] = before + inc[x] - have[x];
    }
    __syncthreads();
    auto find = [&](int x, int item) {  // the last c with first[x][c] <= item
        int lo = 0, hi = n;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (first[x][mid] <= item) lo = mid; else hi = mid;
        }
        return lo;
    };
    auto part = [&](int c, int k) {
        return parts + (R == kRowTile ? (size_t)(c + k) * 2 + (k == 0) : (size_t)(c + k)) * part_floats(R, D);
    };
    auto out_row = [&](const Plan &pl, int r) {
        const int row = pl.row + r;
        return p.out + ((size_t)(pl.row0 + row / G) * b.H + pl.head * G + row % G) * D;
    };

    for (int item = warp * gridDim.x + blockIdx.x; item < total[0]; item += gridDim.x * kWarps) {
        const int c = find(0, item), r = item - first[0][c];
        const Plan pl = list[c];
        const bool has = lane < pl.parts;  // at most 24: a lane holds one part's sums
        const float4 st = has ? *reinterpret_cast<const float4 *>(part(c, lane) + 4 * r) : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
        float4 v0[2][kVec];  // the first two parts, under the sums
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int x = 0; x < kVec; ++x)
                v0[k][x] = (reinterpret_cast<const float4 *>(part(c, k) + 4 * R + r * D) + lane)[32 * x];
        if (__any_sync(0xffffffffu, st.w != 0.f)) continue;  // a part was lost
        float m = st.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float mz = finite_or_0(m), rel = st.y + (st.x - mz);
        float mv = rel;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, d));
        const float vz = finite_or_0(mv);
        float l = has ? st.z * sm100::ex2_approx(st.x - mz) : 0.f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        const float f = has ? sm100::ex2_approx(rel - vz) : 0.f;
        float4 t[kVec];
#pragma unroll
        for (int x = 0; x < kVec; ++x) {
            const float f0 = __shfl_sync(0xffffffffu, f, 0), f1 = __shfl_sync(0xffffffffu, f, 1);
            t[x].x = v0[0][x].x * f0 + v0[1][x].x * f1, t[x].y = v0[0][x].y * f0 + v0[1][x].y * f1;
            t[x].z = v0[0][x].z * f0 + v0[1][x].z * f1, t[x].w = v0[0][x].w * f0 + v0[1][x].w * f1;
        }
#pragma unroll 4
        for (int k = 2; k < pl.parts; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, k);
            const float4 *src = reinterpret_cast<const float4 *>(part(c, k) + 4 * R + r * D) + lane;
#pragma unroll
            for (int x = 0; x < kVec; ++x) {
                const float4 v = src[32 * x];
                t[x].x += v.x * fk, t[x].y += v.y * fk, t[x].z += v.z * fk, t[x].w += v.w * fk;
            }
        }
        const float g = l == 0.f ? 0.f : 1.f / l, g2 = sm100::ex2_approx(vz);
        uint2 *dst = reinterpret_cast<uint2 *>(out_row(pl, r)) + lane;
#pragma unroll
        for (int x = 0; x < kVec; ++x)
            dst[32 * x] = make_uint2(pack_bf16(t[x].x * g * g2, t[x].y * g * g2), pack_bf16(t[x].z * g * g2, t[x].w * g * g2));
    }

    for (int item = blockIdx.x; item < total[1]; item += gridDim.x) {
        const int c = find(1, item), r = (item - first[1][c]) / kSlices, ch = (item - first[1][c]) % kSlices * 64;
        const Plan pl = list[c];
        // a half warp: every 64th part, four channels a lane; all loads before the sums
        float4 v[kBatch], st[kBatch];
        float m = -INFINITY, mv = -INFINITY, l = 0.f;
        bool gone = false;  // a part was lost
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const int k = 2 * kWarps * x + 2 * warp + (lane >> 4);
            const bool in = k < pl.parts;
            st[x] = in ? *reinterpret_cast<const float4 *>(part(c, k) + 4 * r) : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
            v[x] = in ? *reinterpret_cast<const float4 *>(part(c, k) + 4 * R + r * D + ch + 4 * (lane & 15))
                      : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // m over the parts, then mv relative to it
#pragma unroll
        for (int x = 0; x < kBatch; ++x) m = fmaxf(m, st[x].x), gone |= st[x].w != 0.f;
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (lane == 0) red[warp][0] = m;
        __syncthreads();
        m = lane < kWarps ? red[lane][0] : -INFINITY;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float mz = finite_or_0(m);
#pragma unroll
        for (int x = 0; x < kBatch; ++x) mv = fmaxf(mv, st[x].y + (st[x].x - mz));
        mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, 16));
        if (lane == 0) red[warp][1] = mv;
        __syncthreads();
        mv = lane < kWarps ? red[lane][1] : -INFINITY;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, d));
        const float vz = finite_or_0(mv);
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const float f = sm100::ex2_approx(st[x].y + (st[x].x - mz) - vz);
            l += st[x].z * sm100::ex2_approx(st[x].x - mz);
            t.x += v[x].x * f, t.y += v[x].y * f, t.z += v[x].z * f, t.w += v[x].w * f;
        }
        t.x += __shfl_xor_sync(0xffffffffu, t.x, 16), t.y += __shfl_xor_sync(0xffffffffu, t.y, 16);
        t.z += __shfl_xor_sync(0xffffffffu, t.z, 16), t.w += __shfl_xor_sync(0xffffffffu, t.w, 16);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (lane < 16) o[warp][lane] = t;
        if (lane == 0) red[warp][2] = l;
        gone = __syncthreads_or(gone);
        if (tid < 16 && !gone) {
            float lt = 0.f;
            t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 x = o[w][tid];
                lt += red[w][2], t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
            }
            const float f = lt == 0.f ? 0.f : 1.f / lt, f2 = sm100::ex2_approx(vz);
            reinterpret_cast<uint2 *>(out_row(pl, r) + ch)[tid] =
                make_uint2(pack_bf16(t.x * f * f2, t.y * f * f2), pack_bf16(t.z * f * f2, t.w * f * f2));
        }
        __syncthreads();
    }
}

// The pool as a matrix of codes [pages * Hkv * page_size, D]; a box is 128 channels of up to 64 slots of a page.
bool encode_pool(CUtensorMap *m, const uint8_t *base, const Batch &b)
{
    const auto encode = encode_fn();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)b.D, (cuuint64_t)b.num_pages * b.Hkv * b.page}, strides[1] = {(cuuint64_t)b.D};
    const cuuint32_t box[2] = {128, (cuuint32_t)(b.page < kKeyTile ? b.page : kKeyTile)}, estride[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(base), dims, strides, box, estride,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------------------------------------------------ 128 rows at a time
// Chunks of tokens: products on tcgen05 with M = 128 rows (row = token * G + head in the group), 64 keys a tile.
//   warps 0-3 and 8-11  softmax, thread = row = TMEM lane and half of the tile's keys (and of q's and O's channels); the
//   two threads of a row trade their maxima, so that both hold the same references; warp 4 fetches pages by TMA as
//   above; warps 5 and 6 issue S = Q K^T (Q from TMEM) and O += P V (P from TMEM); warps 7 and 12-18 turn v's codes into
//   f16 core matrices of 8 keys x 8 channels (its channels stay contiguous, so nothing is transposed).
// k's codes are operands as they arrive: the e4m3 product takes q as two e4m3 terms (e4m3.cuh: exact down to 2^-9 of the
// row's largest value, below that off by at most 2^-17 of it, far less than the largest's own bf16 rounding) at twice
// the f16 rate.  With k converted too, a tile moved 192 KB through shared memory and took 2.0 us, its converters the
// longest wait; P stays f16, since two e4m3 terms of it would lose the keys below 2^-18 of a row's largest, whose sum
// counts in a long cache.
// Exponents, scales and their references as in the 16-row kernel, with the references raised only when a row's maximum
// passes them by 2^raise, since moving O means a pass through TMEM; P is 2^top at its reference, top + raise = 15, and a
// key is off by at most 2^-(25 + top) of the row's largest.
// A CTA takes whole units, and the last ones (fewer than CTAs) are cut into equal ranges of tiles: at most one part a
// CTA, joined as above.
// Measured: five chunks of up to 256 tokens, 10 heads of 256, 2048 keys each: 45 us with the launch and the join, 330
// TFLOP/s (one thread a row: 50 us).  The start takes 8 us, a tile 1.35, the output 3 and the join 6; without the
// exponentials, maxima and masks the call would still take 37.
constexpr int kWideThreads = 608, kSoftmax = 256;
constexpr float kRaise = 8.f;
constexpr int kNanTiles = 128;  // 8 warps' notes of the tiles that some rows of a unit see and others do not: at most 6 of them

template <int D>
struct WideCfg {
    static constexpr int kRing = 3;  // tiles of codes in flight
    static constexpr int kRaw = kKeyTile * D, kF16 = 2 * kRaw, kRawHalf = kKeyTile * 128;
    static constexpr int kOffRawK = 0, kOffRawV = kRing * kRaw, kOffV = 2 * kRing * kRaw;
    static constexpr int kOffStage = kOffV + 2 * kF16;     // per softmax warp: 32 rows x 32 channels of O on their way out
    static constexpr int kSmem = kOffStage + 8 * 4096 + 1024;
    static_assert(4 * 32 * 2 * D <= 2 * kF16, "the rows of q pass through v's operands' place");
    static constexpr uint32_t kColO = 0, kColQ = 256, kColS = 384, kColP = 448;
};

struct Segment {  // a unit, or a range of its tiles
    int head, row0, ctx, row, rows, pos0, pos1, lo, hi, seq;
    int tile0, tiles;          // the range: first tile (of the positions), tiles
    int parts, part;           // 1, 0: the whole unit
};

// Wide units of a sequence.
__device__ __forceinline__ int wide_units(const AttendArgs &p, const paged::Seq &s)
{
    return p.b.Hkv * (int)(((long long)s.n * (p.b.H / p.b.Hkv) + kWideRows - 1) / kWideRows);
}

template <int D>
__global__ void __launch_bounds__(kWideThreads, 1)
rglru_paged_attention_wide_kernel(const AttendArgs p, const __grid_constant__ CUtensorMap tm_k,
                                  const __grid_constant__ CUtensorMap tm_v)
{
    using namespace sm100;
    using C = WideCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Meta meta[kMeta];
    constexpr int kRing = C::kRing;
    __shared__ uint64_t k_full[kRing], k_free[kRing], rv_full[kRing], rv_free[kRing], v_full[2], v_free[2];
    __shared__ uint64_t q_full, s_full, s_free, p_full[2], pv_done[2], drain[2];
    __shared__ uint32_t tmem_holder;
    __shared__ long long scan[kWideThreads / 32];
    __shared__ int nan_count, nan_key0[kNanTiles], lost;
    __shared__ int sent[2];  // tiles of k and v asked for by a warp 4 that gave up
    __shared__ Plan plan;
    __shared__ Segment seg_s;
    __shared__ float2 trade[2][2][kWideRows];  // what the two threads of a row give each other
    const Batch &b = p.b;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = b.H / b.Hkv, cta = blockIdx.x, n_ctas = gridDim.x;
    Plan *plans = reinterpret_cast<Plan *>(reinterpret_cast<char *>(b.ws) + kWsHeaderBytes);
    float *parts = reinterpret_cast<float *>(reinterpret_cast<char *>(b.ws) + kWsHeaderBytes + align_up_d(kPlanBytes, 256));
    griddep_launch_dependents();

    if (warp == 5) {
        tmem_alloc(&tmem_holder, 512);
        if (lane == 0) {
            for (int i = 0; i < kRing; ++i)
                mbar_init(k_full + i, 1), mbar_init(k_free + i, 1), mbar_init(rv_full + i, 1), mbar_init(rv_free + i, 8);
            for (int i = 0; i < 2; ++i) {
                mbar_init(v_full + i, 8), mbar_init(v_free + i, 1);
                mbar_init(p_full + i, kSoftmax), mbar_init(pv_done + i, 1), mbar_init(drain + i, 1);
            }
            mbar_init(&q_full, kSoftmax), mbar_init(&s_full, 1), mbar_init(&s_free, kSoftmax);
            lost = 0, sent[0] = -1, plan = {0, 0, 0, 0, 0};
            mbar_fence_init();
        }
    }
    // this thread's sequences and the units before them
    const int per = (b.S + kWideThreads - 1) / kWideThreads, s0 = min(b.S, tid * per), s1 = min(b.S, s0 + per);
    long long mine = 0;
    for (int i = s0; i < s1; ++i) mine += wide_units(p, paged::load_seq(b, i));
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    long long all = 0, before = inc - mine;
    for (int w = 0; w < kWideThreads / 32; ++w) {
        if (w < warp) before += scan[w];
        all += scan[w];
    }
    // More units than the rows hold: sequences that name rows twice (cu goes back between them, so load_seq has recorded
    // it); refused here too, so that the counts stay within the host's bounds.
    int units = (int)all;
    if (all > (long long)b.H * b.rows / kWideRows + (long long)b.S * b.Hkv) {
        units = 0;
        paged::record_invalid(b.ws);
    }
    const uint32_t tmem = tmem_holder;
    const int whole = units / n_ctas * n_ctas, rest = units - whole, cuts = rest > 0 ? n_ctas / rest : 1;

    int n = 0;          // tiles done before this segment: the phase of every barrier
    bool alive = true;
    for (int round = 0; round <= units / n_ctas; ++round) {
        int unit = round * n_ctas + cta, part = 0;
        if (round == units / n_ctas) {  // what is left, cut
            if (cta / cuts >= rest) break;
            unit = whole + cta / cuts, part = cta % cuts;
        }
        __syncthreads();  // the last segment is done with
        if (unit >= before && unit < before + mine) {
            int at = (int)before;
            for (int i = s0; i < s1; ++i) {
                const paged::Seq s = paged::load_seq(b, i);
                const int u = wide_units(p, s);
                if (unit < at + u) {
                    const int per_head = u / b.Hkv;
                    Segment g;
                    g.seq = i, g.row0 = s.row0, g.ctx = s.ctx;
                    g.head = (unit - at) / per_head;
                    g.row = (unit - at) % per_head * kWideRows;
                    g.rows = (int)min((long long)kWideRows, (long long)s.n * G - g.row);
                    g.pos0 = s.ctx + g.row / G, g.pos1 = s.ctx + (g.row + g.rows - 1) / G;
                    g.lo = max(0, g.pos0 - p.window + 1), g.hi = g.pos1 + 1;
                    g.tile0 = g.lo / kKeyTile;
                    const int tiles = (g.hi - 1) / kKeyTile - g.tile0 + 1;
                    g.parts = round < units / n_ctas ? 1 : max(1, min(cuts, tiles / kMinTiles));
                    g.part = part;
                    g.tiles = 0;
                    if (part < g.parts) {
                        const int from = (int)((long long)tiles * part / g.parts);
                        g.tiles = (int)((long long)tiles * (part + 1) / g.parts) - from;
                        g.tile0 += from;
                    }
                    seg_s = g;
                    break;
                }
                at += u;
            }
        }
        if (tid == 0) nan_count = 0;
        __syncthreads();
        const Segment seg = seg_s;
        if (seg.tiles == 0) continue;
        const int tiles = seg.tiles;

        if (warp == 4) {
            // ------------------------------------------------------------ pages by TMA
            const int page_shift = 31 - __clz(b.page), box = min(b.page, kKeyTile);
            for (int t0 = 0; t0 < tiles && alive; t0 += 8) {
                const int q = lane & 3, key0 = (seg.tile0 + t0 + (lane >> 2)) * kKeyTile, key = key0 + 16 * q;
                int page = -1;
                float ks = 0.f, vs = 0.f;
                const int bk = key & ~(box - 1);  // the box's first key
                if (t0 + (lane >> 2) < tiles && bk + box > seg.lo && bk < seg.hi) {
                    page = b.table[(size_t)seg.seq * b.max_pages + (key >> page_shift)];
                    if (page < 0 || page >= b.num_pages) {
                        paged::record_invalid(b.ws);
                        page = -1;
                    }
                }
                const size_t at = (size_t)max(page, 0) * b.Hkv + seg.head;
                if (page >= 0) ks = p.ks[at], vs = p.vs[at];
                const bool ok = page >= 0 && key + 16 > seg.lo && key < seg.hi, leads = page >= 0 && key == bk;
                const uint32_t oks = __ballot_sync(0xffffffffu, ok), leaders = __ballot_sync(0xffffffffu, leads);
                const int c1 = (int)((at << page_shift) + (key & (b.page - 1)));
                for (int t = 0; t < min(8, tiles - t0); ++t) {
                    const int i = n + t0 + t, slot = i % kRing;
                    const uint32_t parity = (uint32_t)(i / kRing - 1) & 1u, bytes = (uint32_t)__popc(leaders & (0xfu << (4 * t))) * box * D;
                    const bool lead = leads && (lane >> 2) == t;
                    alive = __all_sync(0xffffffffu, i < kRing || wait(k_free + slot, parity, b.ws, &lost, 10));
                    if (!alive) {
                        if (lane == 0) sent[0] = sent[1] = i;
                        break;
                    }
                    if (lane == 0) mbar_expect(k_full + slot, bytes);
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < D / 128; ++x)
                        if (lead) tma_load_2d(smem + C::kOffRawK + slot * C::kRaw + x * C::kRawHalf + q * 2048, &tm_k, k_full + slot, x * 128, c1);
                    if ((lane >> 2) == t) {
                        Meta &mt = meta[i % kMeta];
                        mt.ks[q] = ks;
                        mt.lv[q] = ok ? log2f(vs) : 0.f;
                        if (q == 0) mt.ok = (int)((oks >> (4 * t)) & 0xfu), mt.key0 = key0;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(k_full + slot);
                    alive = __all_sync(0xffffffffu, i < kRing || wait(rv_free + slot, parity, b.ws, &lost, 11));
                    if (!alive) {
                        if (lane == 0) sent[0] = i + 1, sent[1] = i;
                        break;
                    }
                    if (lane == 0) mbar_expect(rv_full + slot, bytes);
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < D / 128; ++x)
                        if (lead) tma_load_2d(smem + C::kOffRawV + slot * C::kRaw + x * C::kRawHalf + q * 2048, &tm_v, rv_full + slot, x * 128, c1);
                    __syncwarp();
                    if (lane == 0 && !(i == 0 && p.withhold == cta + 1)) mbar_arrive(rv_full + slot);
                }
            }
        } else if (warp == 7 || warp >= 12) {
            // ------------------------------------------------------------ v's codes to f16 operands
            // a thread: one key, a quarter of its 16-channel chunks; lanes are consecutive keys, so every phase of a
            // read or write touches each bank once
            const int cw = warp == 7 ? 0 : warp - 11, row = (cw & 1) * 32 + lane, c0 = (cw >> 1) * (D / 64);
            for (int t = 0; t < tiles; ++t) {
                const int i = n + t, raw = i % kRing, slot = i & 1;
                if (alive) alive = wait(rv_full + raw, (uint32_t)(i / kRing) & 1u, b.ws, &lost, 12);
                if (t == 0 && alive) alive = wait(&q_full, (uint32_t)round & 1u, b.ws, &lost, 28);  // q has left this place
                if (i >= 2 && alive) alive = wait(v_free + slot, (uint32_t)(i / 2 - 1) & 1u, b.ws, &lost, 13);
                const Meta &mt = meta[i % kMeta];
                const int key0 = mt.key0, key = key0 + row;
                const bool in = ((mt.ok >> (row >> 4)) & 1) && key >= seg.lo && key < seg.hi;
                // rows that see different keys: a NaN must not reach those that do not see it
                const bool mixed = key0 < seg.pos1 - p.window + 1 || key0 + kKeyTile - 1 > seg.pos0;
                const uint8_t *src = smem + C::kOffRawV + raw * C::kRaw + row * 128;
                uint8_t *dst = smem + C::kOffV + slot * C::kF16 + (row >> 3) * 128 + (row & 7) * 16;
                uint32_t bad = 0;
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    const int c = c0 + x;
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (in) w = *reinterpret_cast<const uint4 *>(src + (c >> 3) * C::kRawHalf + (((c & 7) ^ (row & 7)) << 4));
                    uint32_t u[4] = {w.x, w.y, w.z, w.w}, h[8];
                    if (mixed) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t m = nan_bytes(u[e]);
                            bad |= m;
                            u[e] &= ~m;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) e4m3::to_f16x2x2(u[e], h[2 * e], h[2 * e + 1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e)  // octets of channels
                        *reinterpret_cast<uint4 *>(dst + (2 * c + e) * 1024) = make_uint4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]);
                }
                if (__any_sync(0xffffffffu, bad != 0) && lane == 0) {
                    const int at = atomicAdd(&nan_count, 1);
                    if (at < kNanTiles) nan_key0[at] = key0;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && alive) {
                    mbar_arrive(v_full + slot);
                    mbar_arrive(rv_free + raw);
                }
            }
        } else if (warp == 5) {
            // ------------------------------------------------------------ S = Q K^T
            const uint32_t idesc = umma_idesc_e4m3(kWideRows, kKeyTile);
            for (int t = 0; t < tiles; ++t) {
                const int i = n + t, slot = i % kRing;
                if (t == 0 && alive) alive = wait(&q_full, (uint32_t)round & 1u, b.ws, &lost, 16);
                if (alive) alive = wait(k_full + slot, (uint32_t)(i / kRing) & 1u, b.ws, &lost, 17);
                if (i >= 1 && alive) alive = wait(&s_free, (uint32_t)(i - 1) & 1u, b.ws, &lost, 18);
                alive = __all_sync(0xffffffffu, alive);
                if (!alive) break;
                tc_fence_after();
                const uint64_t kd = umma_desc_sw128(smem_u32(smem + C::kOffRawK + slot * C::kRaw));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {  // the first terms, then the second
                    const int c = kk % (D / 32);       // 32 channels: 32 bytes into 128-byte rows, 128 channels a half
                    umma_ts_e4m3_warp(tmem + C::kColS, tmem + C::kColQ + (uint32_t)kk * 8,
                                      kd + (uint64_t)(((c >> 2) * C::kRawHalf + (c & 3) * 32) >> 4), idesc, kk > 0);
                }
                umma_commit_warp(&s_full);
                umma_commit_warp(k_free + slot);
                __syncwarp();
            }
        } else if (warp == 6) {
            // ------------------------------------------------------------ O += P V
            const uint32_t idesc = umma_idesc_f16(kWideRows, D) | (1u << 16);  // v's channels are contiguous
            for (int t = 0; t < tiles; ++t) {
                const int i = n + t, slot = i & 1;
                if (alive) alive = wait(p_full + slot, (uint32_t)(i / 2) & 1u, b.ws, &lost, 19);
                if (alive) alive = wait(v_full + slot, (uint32_t)(i / 2) & 1u, b.ws, &lost, 20);
                alive = __all_sync(0xffffffffu, alive);
                if (!alive) break;
                tc_fence_after();
                const uint64_t vd = umma_desc_mn_noswizzle(smem_u32(smem + C::kOffV + slot * C::kF16), 128, 1024);
#pragma unroll
                for (int kk = 0; kk < kKeyTile / 16; ++kk)
                    umma_ts_warp(tmem + C::kColO, tmem + C::kColP + (uint32_t)(slot * 32 + kk * 8), vd + (uint64_t)((kk * 256) >> 4),
                                 idesc, (t > 0 || kk > 0) ? 1u : 0u);
                umma_commit_warp(pv_done + slot);
                umma_commit_warp(v_free + slot);
                __syncwarp();
            }
        } else {
            // ------------------------------------------------------------ softmax, two threads a row
            const int quarter = warp & 3, half = warp >> 3, r = quarter * 32 + lane;
            const bool live = r < seg.rows;
            const int row = seg.row + (live ? r : 0), pos = seg.ctx + row / G;
            // rows behind the unit's see everything: they are not written, and their tiles need no mask
            const int lo = live ? max(0, pos - p.window + 1) : 0, hi = live ? pos : INT_MAX;
            const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
            uint8_t *stage = smem + C::kOffStage + (quarter + 4 * half) * 4096, *rows_q = smem + C::kOffV + quarter * 64 * D;
            // the other thread's value; two turns of the place, so that one barrier is enough
            int turn = 0;
            auto swap = [&](float2 v) {
                trade[turn][half][r] = v;
                asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
                const float2 u = trade[turn][half ^ 1][r];
                turn ^= 1;
                return u;
            };
            float qs;
            {
                // The row as two e4m3 terms, times a power of two that brings its largest exponent to 2^7.  A warp
                // fetches 16 whole rows (a thread fetching its own touches 32 lines an instruction: 4 us), which meet
                // their lane in shared memory, 16-byte piece x of row r at x ^ r: in the place of v's operands, whose
                // converters wait for q.
                constexpr int kPerRow = D / 8, kRowsAtOnce = 32 / kPerRow;  // 16-byte pieces; rows of an instruction
                const int sub = lane / kPerRow, piece = lane % kPerRow;
                uint4 q[16 / kRowsAtOnce];
#pragma unroll
                for (int k = 0; k < 16 / kRowsAtOnce; ++k) {
                    const int at = half * 16 + k * kRowsAtOnce + sub, gr = seg.row + quarter * 32 + at;
                    q[k] = quarter * 32 + at < seg.rows
                               ? __ldg(reinterpret_cast<const uint4 *>(
                                     p.q + ((size_t)(seg.row0 + gr / G) * b.H + seg.head * G + gr % G) * D) + piece)
                               : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < 16 / kRowsAtOnce; ++k) {
                    const int at = half * 16 + k * kRowsAtOnce + sub;
                    *reinterpret_cast<uint4 *>(rows_q + at * 2 * D + ((piece ^ (at & (kPerRow - 1))) << 4)) = q[k];
                }
                asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
                auto mine_q = [&](int k) {  // of this thread's half of the channels
                    k += half * (D / 16);
                    return *reinterpret_cast<const uint4 *>(rows_q + lane * 2 * D + ((k ^ (lane & (kPerRow - 1))) << 4));
                };
                uint32_t top = 0;
#pragma unroll 8
                for (int k = 0; k < D / 16; ++k) {
                    const uint4 u = mine_q(k);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) top = max(top, max((w[x] << 16) & 0x7f800000u, w[x] & 0x7f800000u));
                }
                top = max(top, __float_as_uint(swap(make_float2(__uint_as_float(top), 0.f)).x));
                int e = max(-126, (int)(top >> 23) - 127 - 7);
                if (top == 0) e = 0;
                const float f = __uint_as_float((uint32_t)(127 - e) << 23);
                qs = p.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
                if (top == 0x7f800000u) qs = __uint_as_float(0x7fc00000u);  // as above (the codes saturate)
#pragma unroll 2
                for (int g = 0; g < D / 64; ++g) {  // 32 channels: 8 columns of each term
                    uint32_t hi[8], lo_[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 q4 = mine_q(4 * g + k);
                        const uint32_t u[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t h0, l0, h1, l1;
                            e4m3::split2(pack_f16(bf_lo(u[2 * x]) * f, bf_hi(u[2 * x]) * f), h0, l0);
                            e4m3::split2(pack_f16(bf_lo(u[2 * x + 1]) * f, bf_hi(u[2 * x + 1]) * f), h1, l1);
                            hi[2 * k + x] = h0 | (h1 << 16), lo_[2 * k + x] = l0 | (l1 << 16);
                        }
                    }
                    const uint32_t col = (uint32_t)(half * (D / 8) + g * 8);
                    tmem_st8(tmem + lane_off + C::kColQ + col, hi);
                    tmem_st8(tmem + lane_off + C::kColQ + D / 4 + col, lo_);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&q_full);
            }
            float m = -INFINITY, mv = -INFINITY, l = 0.f;  // l: of this thread's keys
#pragma unroll 1
            for (int t = 0; t < tiles; ++t) {
                const int i = n + t, pb = i & 1;
                if (alive) alive = wait(&s_full, (uint32_t)i & 1u, b.ws, &lost, 21);
                __syncwarp();
                tc_fence_after();
                const Meta &mt = meta[i % kMeta];
                const int key0 = mt.key0 + 32 * half, okm = mt.ok >> (2 * half);
                f2_t v[16];  // pairs of scores
                {
                    uint32_t ra[32];
                    tmem_ld32(tmem + lane_off + C::kColS + (uint32_t)(32 * half), ra);
                    tmem_wait_ld();
                    tc_fence_before();
                    mbar_arrive(&s_free);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = f2_make(__uint_as_float(ra[2 * e]), __uint_as_float(ra[2 * e + 1]));
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const f2_t c = f2_splat(qs * mt.ks[2 * half + g]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[8 * g + e] = f2_mul(v[8 * g + e], c);
                }
                const bool inside = (okm & 3) == 3 && key0 >= lo && key0 + 31 <= hi;
                if (!__all_sync(0xffffffffu, inside)) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const bool ok = (okm >> (e >> 3)) & 1;
                        const int k = key0 + 2 * e;
                        v[e] = f2_make(!ok || k < lo || k > hi ? -INFINITY : f2_lo(v[e]),
                                       !ok || k + 1 < lo || k + 1 > hi ? -INFINITY : f2_hi(v[e]));
                    }
                }
                float gm[2];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    gm[g] = fmaxf(f2_lo(v[8 * g]), f2_hi(v[8 * g]));
#pragma unroll
                    for (int e = 1; e < 8; ++e) gm[g] = fmaxf(gm[g], fmaxf(f2_lo(v[8 * g + e]), f2_hi(v[8 * g + e])));
                }
                const float2 og = swap(make_float2(gm[0], gm[1]));
                const float mt_max = fmaxf(fmaxf(gm[0], gm[1]), fmaxf(og.x, og.y));
                if (mt_max > m + kRaise || (m == -INFINITY && mt_max > m)) {  // l's own reference; mv is relative to it
                    if (m != -INFINITY) l *= ex2_approx(m - mt_max), mv += m - mt_max;
                    m = mt_max;
                }
                const float mz = finite_or_0(m);
                const float lv[2] = {mt.lv[2 * half], mt.lv[2 * half + 1]};
                const float top = fmaxf(fmaxf(gm[0] - mz + lv[0], gm[1] - mz + lv[1]),
                                        fmaxf(og.x - mz + mt.lv[2 - 2 * half], og.y - mz + mt.lv[3 - 2 * half]));
                float f = 1.f;
                bool move = false;
                if (top > mv + (p.raise + p.top) || (mv == -INFINITY && top > mv)) {
                    move = mv != -INFINITY;
                    if (move) f = ex2_approx(mv - top + p.top);
                    mv = top - p.top;
                }
                if (__any_sync(0xffffffffu, move)) {
                    // O holds the tiles before: wait for the last of them, then scale in place, half of the channels a
                    // thread (a row moves after its first tile)
                    if (alive) alive = wait(pv_done + ((i - 1) & 1), (uint32_t)((i - 1) / 2) & 1u, b.ws, &lost, 22);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
                        uint32_t o[32];
                        tmem_ld32(tmem + lane_off + C::kColO + (uint32_t)c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(tmem + lane_off + C::kColO + (uint32_t)c, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                uint32_t pk[2][8];
                f2_t l2[2];
                const float vz = finite_or_0(mv);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    // P = 2^(s - m + d), l sums 2^(s - m).  Where d is above 100 (values 2^100 apart), 2^(s - m) would
                    // underflow under a P that counts: then the exponential is taken at s - m + d - 100, at most 2^-92.
                    const float d = lv[g] - vz, over = fmaxf(0.f, d - 100.f);
                    const f2_t w = f2_splat(ex2_approx(d - over)), minus = f2_splat(over - mz);
                    f2_t lg[2];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const f2_t x = f2_add(v[8 * g + e], minus);
                        const f2_t q = f2_make(ex2_approx(f2_lo(x)), ex2_approx(f2_hi(x)));
                        lg[e & 1] = e < 2 ? q : f2_add(lg[e & 1], q);
                        const f2_t y = f2_mul(q, w);
                        pk[g][e] = pack_f16(f2_lo(y), f2_hi(y));
                    }
                    l2[g] = f2_mul(f2_add(lg[0], lg[1]), f2_splat(ex2_approx(-over)));
                }
                l2[0] = f2_add(l2[0], l2[1]);
                l += f2_lo(l2[0]) + f2_hi(l2[0]);
                // P's buffer was last read by the product of tile i - 2
                if (i >= 2 && alive) alive = wait(pv_done + pb, (uint32_t)(i / 2 - 1) & 1u, b.ws, &lost, 23);
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    tmem_st8(tmem + lane_off + C::kColP + (uint32_t)(pb * 32 + half * 16 + g * 8), pk[g]);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full + pb);
            }
            const int last = n + tiles - 1;
            if (alive) alive = wait(pv_done + (last & 1), (uint32_t)(last / 2) & 1u, b.ws, &lost, 24);
            __syncwarp();
            tc_fence_after();
            // Whether these 32 rows were held up.  A softmax thread that gave up goes on arriving (256 of them, whose
            // guards would cost 0.4 us), so `lost` counts too: it is set before an arrival that could mislead these rows.
            const bool mine_up = !alive || *(volatile int *)&lost != 0;
            const float2 other = swap(make_float2(l, mine_up ? 1.f : 0.f));
            l = half == 0 ? l + other.x : other.x + l;
            const bool held_up = __any_sync(0xffffffffu, mine_up || other.y != 0.f);
            const int bad = min(nan_count, kNanTiles);
            const bool is_whole = seg.parts == 1;
            float *slot = parts + (size_t)cta * part_floats(kWideRows, D);
            const float o_scale = l == 0.f ? 0.f : 1.f / l, o_scale2 = ex2_approx(finite_or_0(mv));
            if (!is_whole && live && !held_up && half == 0) *reinterpret_cast<float4 *>(slot + 4 * r) = make_float4(m, mv, l, 0.f);
#pragma unroll 1
            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
                uint32_t o[32];
                tmem_ld32(tmem + lane_off + C::kColO + (uint32_t)c, o);
                tmem_wait_ld();
                if (live && !held_up)
                    for (int k = 0; k < bad; ++k)  // channels of NaN values that this row sees (noted tiles only, a few)
                        for (int e = max(nan_key0[k], lo); e <= min(nan_key0[k] + kKeyTile - 1, hi); ++e) {
                            const int page = b.table[(size_t)seg.seq * b.max_pages + e / b.page];
                            if (page < 0 || page >= b.num_pages) continue;
                            const uint8_t *src = p.v + (((size_t)page * b.Hkv + seg.head) * b.page + e % b.page) * D + c;
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if ((src[x] & 0x7f) == 0x7f) o[x] = 0x7fc00000u;
                        }
                // through shared memory, so that a store covers whole lines: row r's 16-byte piece x at x ^ (r & 7)
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = is_whole ? __float_as_uint(__uint_as_float(o[4 * x + e]) * o_scale * o_scale2) : o[4 * x + e];
                    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((x ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) {  // four rows at a time, eight lanes each
                    const int rr = 4 * k + (lane >> 3), x = lane & 7, at = quarter * 32 + rr;
                    const uint4 w = *reinterpret_cast<const uint4 *>(stage + rr * 128 + ((x ^ (rr & 7)) << 4));
                    if (at < seg.rows && !held_up) {
                        if (is_whole) {
                            const int gr = seg.row + at;
                            *reinterpret_cast<uint2 *>(
                                p.out + ((size_t)(seg.row0 + gr / G) * b.H + seg.head * G + gr % G) * D + c + 4 * x) =
                                make_uint2(pack_bf16(__uint_as_float(w.x), __uint_as_float(w.y)),
                                           pack_bf16(__uint_as_float(w.z), __uint_as_float(w.w)));
                        } else {
                            *reinterpret_cast<uint4 *>(slot + 4 * kWideRows + (size_t)at * D + c + 4 * x) = w;
                        }
                    }
                }
            }
            if (tid == 0 && !is_whole && seg.part == 0) plan = {(short)seg.parts, (short)seg.rows, seg.row0, seg.row, seg.head};
            tc_fence_before();
        }
        n += tiles;
    }
    // no copy, product or read of TMEM is in flight when the CTA ends
    __syncwarp();
    if (warp == 5 || warp == 6) {
        umma_commit_warp(drain + (warp - 5));
        drain_wait(drain + (warp - 5), 0);
    }
    if (warp == 4) {
        const int k_sent = sent[0] < 0 ? n : sent[0], v_sent = sent[0] < 0 ? n : sent[1];
        for (int i = max(0, k_sent - kRing); i < k_sent; ++i) drain_wait(k_full + i % kRing, (uint32_t)(i / kRing) & 1u);
        for (int i = max(0, v_sent - kRing); i < v_sent; ++i) drain_wait(rv_full + i % kRing, (uint32_t)(i / kRing) & 1u);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (lost && tid < kWideRows)
        *reinterpret_cast<float4 *>(parts + (size_t)cta * part_floats(kWideRows, D) + 4 * tid) = make_float4(0.f, 0.f, 0.f, 1.f);
    if (tid == 0) plans[cta] = lost ? Plan{0, 0, 0, 0, 0} : plan;
    if (warp == 5) tmem_dealloc(tmem, 512);
}

template <int D, int R>
rglru_status launch_join(const AttendArgs &p, int grid, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSms), cfg.blockDim = dim3(kJoinThreads), cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, rglru_paged_combine_kernel<D, R>, p, grid));
}

template <int D>
rglru_status launch(const AttendArgs &p, cudaStream_t stream)
{
    using C = Cfg<D>;
    using W = WideCfg<D>;
    static PerDeviceFlag flag, wide_flag;
    CUtensorMap tm_k, tm_v;
    if (!encode_pool(&tm_k, p.k, p.b) || !encode_pool(&tm_v, p.v, p.b)) return RGLRU_ERR_CUDA;
    // A tile takes the 128-row kernel about 1.3 us an SM whatever its rows, the 16-row one 0.9 for each unit of 16 rows.  256
    // sequences of 32 rows over 2048 keys: 125 us and 112, of 48 rows 126 and 156; 64 sequences of 32 rows 43 and 44, of 48
    // rows 42 and 57; 5 sequences of 48 rows 26 and 23, of 96 rows 27 and 26.  Short runs in the same batch go along with the
    // long ones (a second launch and its join cost 6 us).
    if ((int64_t)p.b.max_new * (p.b.H / p.b.Hkv) <= 2 * kRowTile) {
        const rglru_status st = set_smem_limit_once(reinterpret_cast<const void *>(rglru_paged_attention_kernel<D>), C::kSmem, flag);
        if (st != RGLRU_OK) return st;
        // A third CTA an SM pays when there is much to do (5280 tiles, 160 sequences: 50.5 us against 52.3; 8448: the figures
        // at Cfg); with little, more pieces can be more to join (one sequence over 131072 keys, 2049 tiles: 444 pieces 30.5
        // us, 296 29.1; 96 sequences, 3168 tiles: 39.4 and 38.7; but 64 sequences, 2112 tiles: 31.4 and 32.6).
        const int reach = p.window < p.b.max_total - p.b.max_new ? p.window + p.b.max_new : p.b.max_total;
        const int64_t tiles = (int64_t)p.b.S * p.b.Hkv * (reach / kKeyTile + 1);
        const int grid = kSms * (tiles < kManyTiles * kSms * C::kCtasPerSm ? 2 : C::kCtasPerSm);
        rglru_paged_attention_kernel<D><<<grid, kThreads, C::kSmem, stream>>>(p, tm_k, tm_v);
        if (cudaGetLastError() != cudaSuccess) return RGLRU_ERR_CUDA;
        return launch_join<D, kRowTile>(p, grid, stream);
    }
    const rglru_status st = set_smem_limit_once(reinterpret_cast<const void *>(rglru_paged_attention_wide_kernel<D>), W::kSmem, wide_flag);
    if (st != RGLRU_OK) return st;
    // What keys below f16's range lose is at most 2^-(25 + top) a key: over 2^20 keys 2^-12 of the largest with a raise of
    // 2^8, so beyond them the reference follows every maximum (2^-10 over 2^30 keys).  Five chunks of up to 256 tokens over
    // 2048 keys: 45.1 us against 49.
    const int64_t reach = (int64_t)p.window + p.b.max_new < p.b.max_total ? (int64_t)p.window + p.b.max_new : p.b.max_total;
    AttendArgs a = p;
    a.raise = reach <= (1 << 20) ? 8.f : 0.f;
    a.top = kTop - a.raise;
    rglru_paged_attention_wide_kernel<D><<<kSms, kWideThreads, W::kSmem, stream>>>(a, tm_k, tm_v);
    if (cudaGetLastError() != cudaSuccess) return RGLRU_ERR_CUDA;
    return launch_join<D, kWideRows>(p, kSms, stream);
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
                          window, scale, 0.f, 0.f, debug_withheld, static_cast<const __nv_bfloat16 *>(q), static_cast<const uint8_t *>(k_cache),
                          static_cast<const uint8_t *>(v_cache), k_scale, v_scale, static_cast<__nv_bfloat16 *>(out)};
    const size_t need = rglru_paged_attention_workspace_size(H, Hkv, head_dim);
    const rglru_status c = paged::check_batch(p.b, k_cache, k_scale, v_cache, v_scale, workspace_bytes, need);
    if (c != RGLRU_OK) return c;
    if ((int64_t)num_pages * Hkv * page_size > INT32_MAX) return RGLRU_ERR_UNSUPPORTED;  // rows of a tensor map
    if (!args::al16(q) || !args::al16(out) || window < 1 || !(scale > 0.f) || scale > 1e30f) return RGLRU_ERR_INVALID_ARG;
    // counts of rows and of a CTA's tiles stay below 2^31
    const int64_t span = (int64_t)(max_total < (int64_t)window + max_new ? max_total : (int64_t)window + max_new) / kKeyTile + 2;
    const int64_t units = (int64_t)rows * H / kRowTile + (int64_t)S * Hkv;
    if ((int64_t)rows * H > INT32_MAX || units / kSms + 1 > INT32_MAX / span) return RGLRU_ERR_UNSUPPORTED;
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
