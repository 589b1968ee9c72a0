// Attention of a step's rows over the paged cache. See sv_cache.cu for the mathematics.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "sv_cache.cuh"

namespace sv_cache {

constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kLn2 = 0x1.62e430p-1f;
constexpr int kMaxPlace = 1 << 30;  // places of a request
constexpr int kTile = 128;          // keys of a tile, at most

// A part of a group that ends at a CTA's last tile, to be joined with those of the CTAs behind: the CTAs that
// hold parts of the group, the first one's slot, and the group's rows. first < 0: none.
struct Part {
    int first, last, slot, row0, from, count, head, unused;
};

// How places are cut into tiles: `span` places each, whole pages where a page has at most 128 places (parts 1), or
// each page in `parts` tiles of `box` places (the last may have fewer). Copies by tensor map bring boxes of `box` places
// that lie in one page; box 0: keys are loaded one by one, whatever the pages are.
struct Cut {
    int span, box, parts, boxes, q_box;
};

struct AttentionParams {
    Step s;
    const unsigned char *q;
    unsigned char *out;
    i64 q_row, q_head, out_row, out_head;  // bytes
    Cache kc, vc;
    const float *k_scale, *v_scale;
    float *lse;
    float scale;  // times log2 e
    int window, hq, hk, group;
    bool bf16;            // type of the rows
    Cut cut;
    Divider by_group, by_span, by_parts;
#ifdef SV_DEBUG_BOUNDS
    int patience;
#endif
    float *sums;          // workspace: [ctas][2][rows of a tile][dim], then [ctas][2][rows of a tile][2], then Part [ctas]
    float2 *stats;
    Part *parts;
};

struct TensorMaps {
    CUtensorMap q, k, v;
};

// Whether the CTA's work has been given up.
struct Given {
    int up;        // some wait of the CTA ran out
#ifdef SV_DEBUG_BOUNDS
    int patience;  // (the checked build's tests let waits run out)
#endif
};

// SV_ERR_WAIT once some CTA of the device has given up.
static __device__ unsigned g_cache_error;

enum : int { kFirst = 1, kLast = 2, kPartial = 4, kSlot = 8, kOpen = 16, kEdge = 32 };

// A tile is up to 128 keys. Both products have the keys or the elements in the 128 rows of the tensor cores' memory and
// the query rows (N, 16 to 64) in its columns: scores^T = K Q^T, and out^T += V^T weights^T. So few query rows
// waste nothing, and every key is read from shared memory once for all of them. Roles, each a warp or more: weights
// (twice four warps; a thread has one key's scores of half of the rows), the first product, the second, a plan (the tiles
// and their pages, ahead of the others), queries and keys, values. Keys and values come by tensor map, or, where they are
// 8 bits or the pages small, by eight or sixteen warps that copy (and widen) them vector by vector.
template <int KIND, int D, int N, bool LOADS>  // KIND: type of the cache, SV_BF16, SV_F16 or SV_E4M3
struct Tile {
    static constexpr bool bf16 = KIND == SV_BF16;    // type of the products
    static constexpr int bytes_of = KIND == SV_E4M3 ? 1 : 2;
    static constexpr int rows = N;
    static constexpr int halves = D / 64;            // pieces of 64 elements, 128 bytes a key: the copies' swizzle
    static constexpr int piece = kTile * 128;
    static constexpr int slot = halves * piece;      // keys or values of a tile
    static constexpr int q_bytes = N * D * 2;
    static constexpr int weights = kTile * N * 2;
    static constexpr int q_buffers = (D == 256 && N > 16) || N == 64 ? 1 : 2;
    static constexpr int heads = D == 256 && N > 16 ? 2 : 8;  // descriptions of tiles that are kept
    // 8-bit keys and values are copied to `staged` rooms of a tile before they are widened
    static constexpr int staged = bytes_of == 2 ? 0 : D == 64 ? 4 : D == 128 ? 2 : 1, rooms = staged ? staged : 1, staging = staged * 2 * kTile * D;
    static constexpr int fit = ((heads == 8 ? 223400 : 229376) - q_buffers * q_bytes - 2 * weights - staging) / slot;
    static constexpr int slots = fit > 12 ? 12 : fit;
    static constexpr int k_slots = slots / 2, v_slots = slots - slots / 2;  // rings of their own: each is filled in turn
    static constexpr int blocks = D == 256 ? 2 : 1;  // of 128 elements
    static constexpr int columns_used = (2 + blocks) * N;
    static constexpr int columns = columns_used <= 64 ? 64 : columns_used <= 128 ? 128 : 256;
    static constexpr bool slots_told = D < 256;
    // Factors of the queries of `kept` segments: when those of a segment are written, the weights of all but the two tiles before
    // the last scores are done, and so those of the segment whose place they take.
    static constexpr int kept = q_buffers + 2;
    static constexpr int loaders = bytes_of == 1 ? 16 : LOADS ? 8 : 1;  // warps that widen or copy vector by vector, half of them keys; or that of the values
    static constexpr int threads = 32 * (12 + loaders);
    static constexpr int mine = N / 2;                // rows of a weights warp
    static_assert(slots >= 2 && columns_used <= 256, "room");
    struct Head {
        int p0, first, count, from, head, length, flags, segment;
        int part_first, part_last, part_slot, slot, started;
        uint32_t seen[4];
        int page[kTile];                            // of each box, or of each key
        uint16_t key_slot[slots_told ? kTile : 2];  // of each key
    };
    struct Shared {
        u64 k_full[k_slots], k_empty[k_slots], v_full[v_slots], v_empty[v_slots], scores[2], weighed[2], done[2], q_full[2], q_empty[2], told[heads],
            used[heads], raw_full[2][rooms], raw_empty[2][rooms];  // (of 8-bit keys and values before they are widened)
        u64 ended;  // (of a call that is given up) all products
        Head head[heads];
        alignas(16) float less[N];    // minus the reference of each row's weights (plus the offset)
        alignas(16) float factor[N];  // what a new reference makes of the old sums; of the result
        alignas(16) float scale[bytes_of == 1 ? N : 4];  // of the scores
        union {
            alignas(16) float most[4][N];  // by warps: largest scores, sums of weights
            uint32_t scan[32];  // before the first tile
        };
        uint32_t start[2], total;  // the first tile's request and its number there; tiles of the step
        float top[N];                 // the reference, times log2 e
        i64 row_at[N];                // where a row's result goes, in bytes from its array's start; -1: nowhere
        float q_scale[kept][bytes_of == 1 ? N : 1];  // of queries held in binary16
        uint32_t tensor_at;
        Given given;
        int asked[3];  // tiles of keys, tiles of values, segments of queries asked for by tensor map
    };
    static constexpr int bytes = slots * slot + staging + q_buffers * q_bytes + 2 * weights + static_cast<int>(sizeof(Shared));
    static_assert(bytes <= 232448, "shared memory");
};

// Weights relative to a reference that is the row's largest score when it is set, and is set anew when some score is
// `slack` doublings above it: in bf16 (range of binary32) rarely, in binary16 so that weights stay below 2^15, held
// `offset` doublings up, so that the smallest step of a weight is 2^-35.
template <bool BF16>
struct Weights {
    static constexpr float offset = BF16 ? 0.0f : 11.0f, slack = BF16 ? 8.0f : 4.0f;
};

__device__ __forceinline__ uint32_t shared_address(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(void *to, const void *from, bool there)
{
    there = there && SV_CACHE_INSIDE(from, 16, false);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(shared_address(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger number; NaN if one is.
__device__ __forceinline__ float larger(float a, float b)
{
    float c;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
    return c;
}

// ---------------------------------------------------------------------------------------
// which tiles there are
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ int tile_of(const AttentionParams &P, int p)
{
    if (P.cut.parts == 1) return P.by_span(p);
    const int c = P.s.by_page(p);
    return c * P.cut.parts + P.by_span(p - c * P.s.page);  // (a tile's span is its box)
}
// CTA k's first tile of `total` (below 2^31): total k / ctas, rounded down.
__device__ __forceinline__ uint32_t share_of(uint32_t total, uint32_t k, uint32_t ctas) { return total / ctas * k + total % ctas * k / ctas; }
// The last CTA whose first tile is not behind this one.
__device__ __forceinline__ int sharer_of(uint32_t total, uint32_t number, uint32_t ctas) { return static_cast<int>((static_cast<u64>(number) * ctas + ctas - 1) / total); }

// A sum that does not pass 2^32 - 1.
__device__ __forceinline__ uint32_t sum_of(uint32_t a, uint32_t b)
{
    const uint32_t s = a + b;
    return s < a ? ~0u : s;
}

// All tiles of the step in order: request, rows of a tile, key head, tokens. CTA c takes those from c W / ctas
// to (c + 1) W / ctas, so every CTA gets as many whatever the lengths are. A group is the tiles of a request's N query
// rows and a key head: at least one tile; keys at places [start, end) are seen by one of its rows.
template <int N>
struct Walk {
    const AttentionParams &P;
    int i, first, rows, length;  // the request: its first row, its rows times the group, its length
    int from, count, head, t;    // the group: its first row within the request, its rows; the tile
    int t0, t1, start, end;
    uint32_t base;               // number of the group's first tile

    __device__ __forceinline__ Walk(const AttentionParams &P) : P(P) {}
    __device__ __forceinline__ void request(int k)
    {
        i = k;
        rows = i < P.s.n ? request_rows(P.s, i, first) * P.group : 0;
        length = rows ? ld(P.s.lengths + i) : 0;
    }
    __device__ __forceinline__ void group(int at)
    {
        from = at;
        count = min(N, rows - at);
        const int cap = P.s.width * P.s.page;  // (at most kMaxPlace)
        // places up to that of the last row
        end = length < 0 ? 0 : static_cast<int>(min(static_cast<i64>(length) + (P.by_group(at + count - 1) + 1), static_cast<i64>(cap)));
        start = 0;
        if (P.window > 0 && length >= 0) start = static_cast<int>(min(max(0ll, static_cast<i64>(length) + P.by_group(at) + 1 - P.window), static_cast<i64>(cap)));
        if (start >= end) start = end = 0;
        t0 = start ? tile_of(P, start) : 0;
        t1 = end ? tile_of(P, end - 1) + 1 : 1;
        t = t0;
    }
    __device__ __forceinline__ int tiles() const { return t1 - t0; }
    __device__ __forceinline__ uint32_t request_tiles(int k)
    {
        request(k);
        uint32_t sum = 0;
#pragma unroll 1
        for (int at = 0; at < rows; at += N) {
            group(at);
            sum += tiles() * P.hk;  // (below 2^31: the host sees to it for the rows that there are)
        }
        return sum;
    }
    // To tile `skip` of request k, the step's tile `number`.
    __device__ __forceinline__ void seek(int k, uint32_t skip, uint32_t number)
    {
        request(k);
        base = number - skip;
#pragma unroll 1
        for (int at = 0; at < rows; at += N) {
            group(at);
            const uint32_t here = tiles() * P.hk;
            if (skip < here) break;
            skip -= here;
            base += here;
        }
        head = static_cast<int>(skip / static_cast<uint32_t>(tiles()));
        t += static_cast<int>(skip) - head * tiles();
        base += head * tiles();
    }
    __device__ __forceinline__ void next()
    {
        if (++t < t1) return;
        base += tiles();
        t = t0;
        if (++head < P.hk) return;
        head = 0;
        if (from + N < rows) return group(from + N);
        do
            request(i + 1);
        while (rows == 0 && i < P.s.n);
        if (rows) group(0);
    }
};

// ---------------------------------------------------------------------------------------
// barriers, copies, products
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void barrier_init(u64 *b, int count) { asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(shared_address(b)), "r"(count) : "memory"); }
__device__ __forceinline__ void barrier_expect(u64 *b, int bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(shared_address(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void barrier_arrive(u64 *b) { asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(shared_address(b)) : "memory"); }
// Waits for a phase to end, not for ever: false if after kPatience looks (seconds) it has not, or some other wait of the CTA ran
// out before. All lanes of a warp get the same answer. Who gets false leaves its work where it is: it arrives
// at no barrier and writes no description any more, so every phase that does end stands for what it says, and the others come to the
// end of their work or to a wait that gives up as well. (The weights' warps, which meet, leave together; see there.) Whoever waits has seen
// the phase before end, so that a parity names one phase.
constexpr int kPatience = 1 << 22;
__device__ __forceinline__ bool barrier_try(u64 *b, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared.b64 p, [%1], %2;\nselp.b32 %0, 1, 0, p;\n}" : "=r"(done) : "r"(shared_address(b)), "r"(parity) : "memory");
    return done != 0;
}
#ifndef SV_DEBUG_BOUNDS
__device__ __forceinline__ bool barrier_wait(u64 *b, uint32_t parity, Given *given)
{
    uint32_t there;
    asm volatile(
        "{\n.reg .pred p;\n.reg .b32 k, l;\nmov.b32 k, %4;\nmov.b32 %0, 1;\n"
        "$AGAIN_%=: mbarrier.try_wait.parity.shared.b64 p, [%1], %2;\nvote.sync.all.pred p, p, 0xffffffff;\n@p bra $DONE_%=;\n"
        "ld.volatile.shared.b32 l, [%3];\nsetp.ne.b32 p, l, 0;\nvote.sync.any.pred p, p, 0xffffffff;\n@p bra $LEAVE_%=;\n"
        "sub.u32 k, k, 1;\nsetp.ne.b32 p, k, 0;\n@p bra $AGAIN_%=;\n"
        "mov.b32 l, 1;\nst.volatile.shared.b32 [%3], l;\n$LEAVE_%=: mov.b32 %0, 0;\n$DONE_%=:\n}"
        : "=r"(there)
        : "r"(shared_address(b)), "r"(parity), "r"(shared_address(&given->up)), "n"(kPatience)
        : "memory");
    return there != 0;
}
#else
// The same with looks that do not last, as many as the call says.
__device__ __forceinline__ bool barrier_wait(u64 *b, uint32_t parity, Given *given)
{
    volatile Given *const g = given;
    for (int k = g->patience;;) {
        uint32_t done;
        asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared.b64 p, [%1], %2;\nselp.b32 %0, 1, 0, p;\n}" : "=r"(done) : "r"(shared_address(b)), "r"(parity) : "memory");
        if (__all_sync(~0u, done)) return true;
        if (__any_sync(~0u, g->up)) return false;
        if (--k <= 0) break;
    }
    g->up = 1;
    return false;
}
#endif
// The last `slots` phases, at most, of `count` that a ring's barriers were asked for: waits for them on the way out (again not for ever).
__device__ __forceinline__ void barrier_drain(u64 *b, int slots, int count)
{
#pragma unroll 1
    for (int it = max(0, count - slots); it < count; ++it)
#pragma unroll 1
        for (int k = 0; k < kPatience && !barrier_try(b + it % slots, it / slots & 1); ++k) {
        }
}
// A box of an array of heads, [1][1][box][64 elements], to shared memory (swizzled by 128 bytes).
__device__ __forceinline__ void copy_box(uint32_t to, const CUtensorMap *map, u64 *b, int element, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(to), "l"(map),
                 "r"(shared_address(b)), "r"(element), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// Description of a matrix in shared memory: address, the two strides in bytes, and the swizzle (2: 128 bytes, 0: none). The
// address is in the lower word, in steps of 16 bytes.
__device__ __forceinline__ u64 matrix_at(uint32_t at, uint32_t lead, uint32_t stride, u64 swizzle)
{
    return static_cast<u64>((at & 0x3ffff) >> 4) | static_cast<u64>(lead >> 4) << 16 | static_cast<u64>(stride >> 4) << 32 | u64{1} << 46 | swizzle << 61;
}
// Shape of a product of 16-bit elements, 128 x N, into binary32; whether A and B have their rows contiguous.
__host__ __device__ constexpr uint32_t product_of(bool bf16, int n, bool turned)
{
    return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (turned ? 3u : 0u) << 15 | static_cast<uint32_t>(n >> 3) << 17 | 8u << 24;
}
// One lane of a warp, always the same.
__device__ __forceinline__ uint32_t elected()
{
    uint32_t one;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.b32 %0, 1, 0, p;\n}" : "=r"(one));
    return one;
}
// d (+)= A B, issued by the elected lane of a warp whose lanes all call it: with operands that are the same in the whole warp
// a product is issued every 40 to 50 cycles, by a lane on its own path (and descriptions put together anew) every 75 to 115.
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t a_high, uint32_t b, uint32_t b_high, uint32_t shape, bool add, uint32_t leader)
{
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 x, y;\nmov.b64 x, {%1, %2};\nmov.b64 y, {%3, %4};\nsetp.ne.b32 p, %6, 0;\nsetp.ne.b32 q, %7, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n}" ::"r"(d),
        "r"(a), "r"(a_high), "r"(b), "r"(b_high), "r"(shape), "r"(static_cast<int>(add)), "r"(leader)
        : "memory");
}
// An arrival at b when all products that the elected lane has issued so far have ended.
__device__ __forceinline__ void products_close(u64 *b, uint32_t leader)
{
    asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"l"(
                     static_cast<u64>(shared_address(b))),
                 "r"(leader)
                 : "memory");
}
__device__ __forceinline__ void tensor_load8(float *v, uint32_t at)
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at)
                 : "memory");
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r[k]);
}
__device__ __forceinline__ void tensor_store8(uint32_t at, const float *v)
{
    uint32_t r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = __float_as_uint(v[k]);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
                 "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tensor_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tensor_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tensor_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void shared_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// The eight warps of the weights among themselves.
__device__ __forceinline__ void weights_meet() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool weights_any(bool x)
{
    int any;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\nbar.red.or.pred q, 2, 256, p;\nselp.b32 %0, 1, 0, q;\n}" : "=r"(any) : "r"(static_cast<int>(x)) : "memory");
    return any != 0;
}

// They meet, and know whether one of them has given up (behind the one above, which such a warp makes true).
__device__ __forceinline__ bool weights_gone(bool x)
{
    int any;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\nbar.red.or.pred q, 1, 256, p;\nselp.b32 %0, 1, 0, q;\n}" : "=r"(any) : "r"(static_cast<int>(x)) : "memory");
    return any != 0;
}

// The boxes of a tile's keys or values, by a warp, once the slot is free; false if that is given up.
template <typename S>
__device__ __forceinline__ bool boxes_to(const CUtensorMap *map, u64 *full, u64 *empty, bool wait, uint32_t parity, uint32_t to, const Cut &cut, int slot, int head,
                                         const int *page, int lane, Given *given)
{
    if (wait && !barrier_wait(empty, parity, given)) return false;
    if (lane == 0) barrier_expect(full, cut.boxes * cut.box * 128 * S::halves);
    __syncwarp();
#pragma unroll 1
    for (int k = lane; k < cut.boxes * S::halves; k += 32) {
        const int b = k / S::halves, e = k % S::halves;
        copy_box(to + e * S::piece + b * cut.box * 128, map, full, e * 64, slot, head, page[b]);
    }
    return true;
}
template <typename E, typename T>
__device__ __forceinline__ E from_bits(T v)
{
    static_assert(sizeof(E) == 2 && sizeof(T) == 2);
    E e;
    memcpy(&e, &v, 2);
    return e;
}

// The largest of 8 columns' numbers over a warp, or their sums: lane l gets that of column l % 8 (a NaN stays one).
template <bool SUM>
__device__ __forceinline__ float columns_joined(float *v, int lane)
{
    auto join = [](float a, float b) { return SUM ? a + b : larger(a, b); };
#pragma unroll
    for (int half = 4; half; half /= 2)
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const bool upper = lane & half;
            const float other = __shfl_xor_sync(~0u, upper ? v[k] : v[k + half], half);
            v[k] = join(upper ? v[k + half] : v[k], other);
        }
    v[0] = join(v[0], __shfl_xor_sync(~0u, v[0], 8));
    return join(v[0], __shfl_xor_sync(~0u, v[0], 16));
}

// Registers of a warp's roles in the kernels with many warps, of four warps each: 2 x 104 + 3 x 56 are within the launch's
// 5 x 96, 2 x 104 + 5 x 56 within 7 x 72. (The checked
// build spills instead: its calls in these loops need more than there are.)
#ifdef SV_DEBUG_BOUNDS
#define SV_CACHE_REGISTERS(way, count) (void)0
#else
#define SV_CACHE_REGISTERS(way, count) asm volatile("setmaxnreg." way ".sync.aligned.u32 " #count ";")
#endif

// NaN for the rows of a CTA that gave up, or for their parts (told as those of a CTA that did not), by its first 256 threads.
template <int N, int D, typename E>
__device__ __forceinline__ void rows_lost(const AttentionParams &P, const uint32_t *start, uint32_t total)
{
    const uint32_t ctas = min(total, gridDim.x), cta = blockIdx.x, u0 = share_of(total, cta, ctas), u1 = share_of(total, cta + 1, ctas);
    const int n = static_cast<int>(u1 - u0);  // (some: who has no tile waits for nothing)
    Walk<N> walk(P);
    const float nan = __int_as_float(0x7fffffff);
    walk.seek(static_cast<int>(start[0]), start[1], u0);
    int here = 0;  // tiles of the group
#pragma unroll 1
    for (int it = 0; it < n; it += here) {
        here = min(walk.t1 - walk.t, n - it);
        const bool open = here < walk.t1 - walk.t, partial = walk.base < u0 || walk.base + walk.tiles() > u1;
        const i64 part = (static_cast<i64>(cta) * 2 + (walk.base > u0 ? 1 : 0)) * N;
#pragma unroll 1
        for (int x = threadIdx.x; x < walk.count * D; x += 256) {
            const int r = x / D, e = x % D, at_row = walk.from + r, j = P.by_group(at_row), qh = walk.head * P.group + at_row - j * P.group;
            const i64 row = static_cast<i64>(walk.first) + j;
            if (partial) {
                st(P.sums + (part + r) * D + e, nan);
                if (e == 0) st(P.stats + part + r, make_float2(nan, nan));
            } else {
                st(reinterpret_cast<E *>(P.out + row * P.out_row + qh * P.out_head) + e, from_bits<E>(static_cast<uint16_t>(0x7fff)));  // (a NaN in either type)
                if (e == 0 && P.lse) st(P.lse + row * P.hq + qh, nan);
            }
        }
        if (P.parts && threadIdx.x == 0 && it + here == n) {
            const uint32_t k = sharer_of(total, walk.base, ctas);
            st(reinterpret_cast<int4 *>(P.parts + cta),
               make_int4(open ? static_cast<int>(k) : -1, sharer_of(total, walk.base + walk.tiles() - 1, ctas), share_of(total, k, ctas) < walk.base, walk.first));
            st(reinterpret_cast<int4 *>(P.parts + cta) + 1, make_int4(walk.from, walk.count, walk.head, 0));
        }
        walk.t = walk.t1 - 1;
        walk.next();
    }
}

// (LOADS: keys vector by vector, not by tensor map. Kernels of their own, since the size of the code counts.)
template <int KIND, int D, int N, bool LOADS>
__global__ void __launch_bounds__((Tile<KIND, D, N, LOADS>::threads), 1) sv_cache_attention_kernel(const AttentionParams P, const __grid_constant__ TensorMaps maps)
{
    using S = Tile<KIND, D, N, LOADS>;
    constexpr bool kBf16 = S::bf16, kWide = KIND == SV_E4M3;  // 8 bits are widened to binary16
    using E = std::conditional_t<kBf16, __nv_bfloat16, __half>;
    using W = Weights<kBf16>;
    extern __shared__ __align__(1024) unsigned char room[];
    unsigned char *const staging = room + S::slots * S::slot, *const q_room = staging + S::staging, *const w_room = q_room + S::q_buffers * S::q_bytes;
    auto &sh = *reinterpret_cast<typename S::Shared *>(w_room + 2 * S::weights);
    const uint32_t room_at = shared_address(room), q_at = shared_address(q_room), w_at = shared_address(w_room);
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid / 32, 0), lane = tid & 31;
    const int cta = blockIdx.x;
    constexpr bool loads = LOADS, many = loads || kWide;

    // -- barriers and memory, while the work before this call ends
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_address(&sh.tensor_at)), "n"(S::columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        const int filled = many ? S::loaders / 2 : 1;  // arrivals at a slot: of the loading warps, or of the thread that names the bytes
#pragma unroll 1
        for (int k = 0; k < S::v_slots; ++k) {
            if (k < S::k_slots) barrier_init(sh.k_full + k, filled), barrier_init(sh.k_empty + k, 1);
            barrier_init(sh.v_full + k, filled), barrier_init(sh.v_empty + k, 1);
        }
#pragma unroll 1
        for (int k = 0; k < 2 * S::staged; ++k) barrier_init(&sh.raw_full[0][0] + k, 1), barrier_init(&sh.raw_empty[0][0] + k, S::loaders / 2);
#pragma unroll 1
        for (int k = 0; k < S::heads; ++k) barrier_init(sh.told + k, 1), barrier_init(sh.used + k, 2);  // (used: by the second product, and by the warp of the queries)
#pragma unroll 1
        for (int k = 0; k < 2; ++k)
            barrier_init(sh.scores + k, 2), barrier_init(sh.weighed + k, 256), barrier_init(sh.done + k, 1), barrier_init(sh.q_full + k, 1), barrier_init(sh.q_empty + k, 1);
        barrier_init(&sh.ended, 2);
        sh.given.up = 0;
#ifdef SV_DEBUG_BOUNDS
        sh.given.patience = P.patience;
#endif
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 12 * 32 && !loads) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.v) : "memory");
        if (!kWide) asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.q) : "memory");
    }
    if constexpr (!loads) {  // places of a slot that no copy writes: zeros for good
        // (8 bits: of the rooms that they are copied to before they are widened)
        constexpr int kPieces = kWide ? 2 * S::staged : S::slots * S::halves, kPiece = kWide ? kTile * D : S::piece, kKey = kWide ? D : 128;
        const int filled = P.cut.boxes * P.cut.box, piece = (kTile - filled) * (kKey / 16);
#pragma unroll 1
        for (int x = tid; x < kPieces * piece; x += S::threads)
            *reinterpret_cast<uint4 *>((kWide ? staging : room) + x / piece * kPiece + filled * kKey + x % piece * 16) = make_uint4(0, 0, 0, 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // -- this CTA's tiles
    Walk<N> walk(P);
    const int per = (P.s.n + S::threads - 1) / S::threads;
    uint32_t mine = 0;
#pragma unroll 1
    for (int k = tid * per; k < min(P.s.n, (tid + 1) * per); ++k) mine = sum_of(mine, walk.request_tiles(k));
    auto running = [lane](uint32_t x) {
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t up = __shfl_up_sync(~0u, x, d);
            if (lane >= d) x = sum_of(x, up);
        }
        return x;
    };
    uint32_t before = running(mine);
    if (lane == 31) sh.scan[warp] = before;
    tensor_before();
    __syncthreads();
    tensor_after();
    const uint32_t warps = running(lane < S::threads / 32 ? sh.scan[lane] : 0u), all = __shfl_sync(~0u, warps, 31);
    // (2^31 tiles or more come only of requests that overlap, by prefix sums that are none: such a step is left out)
    const uint32_t total = all < 1u << 31 ? all : 0;
    if (tid == 0) sh.total = total;
    before += (warp ? __shfl_sync(~0u, warps, (warp - 1) & 31) : 0u) - mine;
    const uint32_t tensor = __shfl_sync(~0u, sh.tensor_at, 0);
    const uint32_t ctas = min(total, gridDim.x);  // (each with a tile at least)
    int n = 0;
    uint32_t u0 = 0, u1 = 0;
    if (cta < static_cast<int>(ctas)) {
        u0 = share_of(total, cta, ctas), u1 = share_of(total, cta + 1, ctas);
        n = __shfl_sync(~0u, static_cast<int>(u1 - u0), 0);
        if (u0 >= before && u0 < before + mine) {
            uint32_t at = before;
            int k = tid * per;
            if (per > 1)
#pragma unroll 1
                for (; k < min(P.s.n, (tid + 1) * per) - 1; ++k) {
                    const uint32_t here = walk.request_tiles(k);
                    if (u0 < at + here) break;
                    at += here;
                }
            sh.start[0] = static_cast<uint32_t>(k);
            sh.start[1] = u0 - at;
        }
    } else if (P.parts && tid == 0) {
        st(&P.parts[cta].first, -1);
    }
    __syncthreads();
    Given *const given = &sh.given;

    if (warp < 8) {
        if constexpr (many) SV_CACHE_REGISTERS("inc", 104);
        // -- weights: this thread has key `key0` of every tile, the elements key0 and key0 + 128 of the outputs, and rows r0 to r0 + M - 1
        constexpr int M = S::mine;
        const int key0 = tid & 127, r0 = warp / 4 * M;
        const uint32_t lanes = tensor + (static_cast<uint32_t>(warp & 3) << 21);  // (lane 32 * (warp % 4) of the tensor memory, in bits 16 and up)
        float sum[M];
        float scale = 0;
        // A warp whose wait for scores is given up says so at the tile's first meeting, whatever the tile is: that is `weights_any`, and the
        // meeting behind it where that is true, `weights_gone`, tells the others to leave with it. Whether a wait within a tile was given up does not
        // matter: what the tile makes is overwritten at the kernel's end, and its weights are in their room all the same.
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            const int b = it & 1;
            const uint32_t turn = it >> 1 & 1;
            auto &h = sh.head[it % S::heads];
            if (__builtin_expect(!barrier_wait(sh.scores + b, turn, given), 0)) {
                weights_any(true);
                weights_gone(true);
                break;
            }
            tensor_after();
            const int flags = h.flags;
            if (it >= 2) barrier_wait(sh.done + b, turn ^ 1, given);  // (the weights' room is free, and the values before the last have come)
            int r_lo = 0, r_hi = key0 < P.cut.span ? M : 0;  // the rows, from r0 on, that see this thread's key
            const bool masks = flags & kEdge || (key0 | 31) >= P.cut.span;  // (the same in a warp)
            if (flags & kFirst) {
                const int head = h.head;
                scale = P.scale * (P.k_scale ? ld(P.k_scale + head) : 1.0f);
#pragma unroll
                for (int r = 0; r < M; ++r) sum[r] = 0;
                if constexpr (kWide) {
                    const int segment = h.segment;
                    if (tid < N) sh.scale[tid] = scale * sh.q_scale[segment % S::kept][tid];
                    if (__builtin_expect(weights_any(false), 0)) {
                        weights_gone(false);
                        break;
                    }
                }
            }
            if (__builtin_expect(flags & kEdge, 0)) {
                const i64 d = static_cast<i64>(h.p0) + key0 - h.length;  // it is the d-th new token's place
                const i64 lo = d <= 0 ? 0 : d * P.group - h.from - r0, hi = P.window > 0 ? (d + P.window) * P.group - h.from - r0 : M;
                r_lo = static_cast<int>(min(max(lo, 0ll), static_cast<i64>(M)));
                r_hi = static_cast<int>(min(max(hi, 0ll), static_cast<i64>(M)));
                if (!(h.seen[key0 / 32] >> (key0 & 31) & 1)) r_hi = 0;
                // A weight of 0 times a value that is not finite would be NaN. Such elements, if any, are set to 0 in shared
                // memory, and what they make of the rows that see them is added by hand.
                const int vslot = it % S::v_slots;
                if (S::v_slots == 1 && it > 0) barrier_wait(sh.done + (b ^ 1), (it - 1) >> 1 & 1, given);
                barrier_wait(sh.v_full + vslot, it / S::v_slots & 1, given);
                unsigned char *const v = room + (S::k_slots + vslot) * S::slot;
                auto chunk = [&](int key, int c) { return reinterpret_cast<uint4 *>(v + c / 8 * S::piece + key * 128 + (((c & 7) ^ (key & 7)) << 4)); };
                constexpr uint32_t mask = kBf16 ? 0x7f80u : 0x7c00u;
                bool odd = false;
#pragma unroll 2
                for (int c = warp / 4; c < D / 8; c += 2) {
                    const uint4 x = *chunk(key0, c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t w = k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w;
                        odd |= (w & mask) == mask || (w >> 16 & mask) == mask;
                    }
                }
                if (__builtin_expect(weights_any(odd), 0)) {
                    // (rare: one row at a time, every element over all keys)
                    if (it > 0) barrier_wait(sh.done + (b ^ 1), (it - 1) >> 1 & 1, given);
                    tensor_after();
#pragma unroll 1
                    for (int e = 0; e < S::blocks; ++e)
#pragma unroll 1
                        for (int r = r0; r < r0 + M; ++r) {
                            const uint32_t at = lanes + (2 + e) * N + r;
                            uint32_t w;
                            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(w) : "r"(at) : "memory");
                            tensor_loaded();
                            float x = flags & kFirst ? 0.0f : __uint_as_float(w);
                            const int element = e * 128 + key0;
#pragma unroll 1
                            for (int key = 0; key < kTile && element < D; ++key) {
                                const i64 dk = static_cast<i64>(h.p0) + key - h.length;
                                if (!(h.seen[key / 32] >> (key & 31) & 1) || (dk > 0 && r < dk * P.group - h.from) || (P.window > 0 && r >= (dk + P.window) * P.group - h.from)) continue;
                                const float y = static_cast<float>(reinterpret_cast<const E *>(chunk(key, element / 8))[element & 7]);
                                if (!(fabsf(y) < kInf)) x += y;
                            }
                            __syncwarp();
                            asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(at), "r"(__float_as_uint(x)) : "memory");
                        }
                    tensor_stored();
                    tensor_before();
                    if (weights_gone(false)) break;
#pragma unroll 1
                    for (int c = warp / 4; c < D / 8; c += 2) {
                        uint32_t *x = reinterpret_cast<uint32_t *>(chunk(key0, c));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((x[k] & mask) == mask) x[k] &= 0xffff0000u;
                            if ((x[k] >> 16 & mask) == mask) x[k] &= 0xffffu;
                        }
                    }
                    shared_to_async();
                    if (tid == 0) h.started = 1;
                }
            }

            // -- the scores relative to the reference; a new one where some score is too far above it
            const uint32_t scores_at = lanes + b * N + r0;
            float s[M];
            auto relative = [&] {
#pragma unroll
                for (int c = 0; c < M; c += 8) tensor_load8(s + c, scores_at + c);
                tensor_loaded();
#pragma unroll
                for (int r = 0; r < M; r += 4) {
                    const float4 less = *reinterpret_cast<const float4 *>(sh.less + r0 + r);
                    const float4 by = kWide ? *reinterpret_cast<const float4 *>(sh.scale + r0 + r) : make_float4(scale, scale, scale, scale);
                    s[r] = fmaf(s[r], by.x, less.x), s[r + 1] = fmaf(s[r + 1], by.y, less.y);
                    s[r + 2] = fmaf(s[r + 2], by.z, less.z), s[r + 3] = fmaf(s[r + 3], by.w, less.w);
                }
                if (__builtin_expect(masks, 0)) {
#pragma unroll
                    for (int r = 0; r < M; ++r)
                        if (r < r_lo || r >= r_hi) s[r] = -kInf;
                }
            };
            bool renew = flags & kFirst;
            if (!renew) {
                relative();
                float far[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
                for (int r = 0; r < M; ++r) far[r & 3] = fmaxf(far[r & 3], s[r]);
                renew = weights_any(fmaxf(fmaxf(far[0], far[1]), fmaxf(far[2], far[3])) > W::offset + W::slack);
            }
            if (__builtin_expect(renew, 0)) {
#pragma unroll 1
                for (int c = 0; c < M; c += 8) {
                    float v[8];
                    tensor_load8(v, scores_at + c);
                    tensor_loaded();
#pragma unroll
                    for (int r = 0; r < 8; ++r) v[r] = c + r < r_lo || c + r >= r_hi ? -kInf : v[r] * (kWide ? sh.scale[r0 + c + r] : scale);
                    const float most = columns_joined<false>(v, lane);
                    if (lane < 8) sh.most[warp & 3][r0 + c + lane] = most;
                }
                const bool opens = !kWide && (flags & (kFirst | kEdge)) == kFirst;  // (the tile's first meeting)
                if (opens ? weights_any(false) : weights_gone(false)) {
                    if (opens) weights_gone(false);
                    break;
                }
                if (tid < N) {
                    const float old = flags & kFirst ? -kInf : sh.top[tid];
                    const float top = larger(larger(larger(sh.most[0][tid], sh.most[1][tid]), larger(sh.most[2][tid], sh.most[3][tid])), old);
                    sh.factor[tid] = top == old ? 1.0f : exp2_fast(old - top);
                    sh.top[tid] = top;
                    sh.less[tid] = top == -kInf ? 0x1.fffffep127f : W::offset - top;  // (no key yet: any score is far above, -1e38 too)
                }
                weights_meet();
                if (!(flags & kFirst)) {
                    barrier_wait(sh.done + (b ^ 1), (it - 1) >> 1 & 1, given);
                    tensor_after();
#pragma unroll 1
                    for (int e = 0; e < S::blocks; ++e)
#pragma unroll 1
                        for (int c = 0; c < M; c += 8) {
                            float o[8];
                            tensor_load8(o, lanes + (2 + e) * N + r0 + c);
                            tensor_loaded();
#pragma unroll
                            for (int r = 0; r < 8; ++r) o[r] *= sh.factor[r0 + c + r];
                            tensor_store8(lanes + (2 + e) * N + r0 + c, o);
                        }
                    tensor_stored();
                    tensor_before();
#pragma unroll
                    for (int r = 0; r < M; r += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(sh.factor + r0 + r);
                        sum[r] *= f.x, sum[r + 1] *= f.y, sum[r + 2] *= f.z, sum[r + 3] *= f.w;
                    }
                }
                relative();
            }
            // -- weights, to shared memory as the product wants them: eight rows of a key side by side. Rounded to the type of the values, since a product
            // of 16 bits takes both operands so: 2^-8 (bf16) or 2^-11 of each, which over many keys adds about as much as the output's own
            // rounding does (errors against 64 bits 1.0 to 1.5 times those of binary32 weights). Their sums are taken before.
            unsigned char *const to = w_room + b * S::weights + r0 / 8 * (kTile * 16) + key0 * 16;
#pragma unroll
            for (int r = 0; r < M; r += 8) {
                float e[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    e[k] = exp2_fast(s[r + k]);
                    sum[r + k] += e[k];
                }
                *reinterpret_cast<uint4 *>(to + r / 8 * (kTile * 16)) = make_uint4(pack<E>(e[0], e[1]), pack<E>(e[2], e[3]), pack<E>(e[4], e[5]), pack<E>(e[6], e[7]));
            }
            shared_to_async();
            tensor_before();
            int head = 0, from = 0, count = 0, first_row = 0, part_first = 0, part_last = 0, part_slot = 0;
            if (flags & kLast) {  // (before others may take the description's room)
                head = h.head, from = h.from, count = h.count, first_row = h.first;
                part_first = h.part_first, part_last = h.part_last, part_slot = h.part_slot;
            }
            barrier_arrive(sh.weighed + b);
            if (__builtin_expect(!(flags & kLast), 1)) continue;

            // -- a segment's end: the sums over the keys, and the result or the part written
#pragma unroll
            for (int c = 0; c < M; c += 8) {
                const float z = columns_joined<true>(sum + c, lane);
                if (lane < 8) sh.most[warp & 3][r0 + c + lane] = z;
            }
            weights_meet();
            const bool partial = flags & kPartial;
            if (tid < N) {
                const float top = sh.top[tid];
                const float z = top == -kInf ? 0.0f : (sh.most[0][tid] + sh.most[1][tid]) + (sh.most[2][tid] + sh.most[3][tid]);
                const int at_row = from + tid, j = P.by_group(at_row), qh = head * P.group + at_row - j * P.group;
                const i64 part = (static_cast<i64>(cta) * 2 + (flags & kSlot ? 1 : 0)) * N + tid;
                sh.factor[tid] = z == 0 ? 0.0f : partial ? 1.0f : (P.v_scale ? ld(P.v_scale + head) : 1.0f) / z;
                sh.row_at[tid] = tid >= count ? -1 : partial ? part * (D * 4) : static_cast<i64>(first_row + j) * P.out_row + static_cast<i64>(qh) * P.out_head;
                if (tid < count) {
                    if (partial)
                        st(P.stats + part, make_float2(top, z));
                    else if (P.lse)
                        st(P.lse + static_cast<i64>(first_row + j) * P.hq + qh, z == 0 ? -kInf : (top - W::offset + log2f(z)) * kLn2);
                }
            }
            if (tid == 128 && P.parts && it == n - 1) {
                st(reinterpret_cast<int4 *>(P.parts + cta), make_int4(flags & kOpen ? part_first : -1, part_last, part_slot, first_row));
                st(reinterpret_cast<int4 *>(P.parts + cta) + 1, make_int4(from, count, head, 0));
            }
            weights_meet();
            barrier_wait(sh.done + b, turn, given);
            tensor_after();
            if (D >= 128 || key0 < D) {
                unsigned char *const array = partial ? reinterpret_cast<unsigned char *>(P.sums) : P.out;
#pragma unroll 1
                for (int e = 0; e < S::blocks; ++e)
#pragma unroll 1
                    for (int c = 0; c < M; c += 8) {
                        float o[8];
                        tensor_load8(o, lanes + (2 + e) * N + r0 + c);
                        tensor_loaded();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const i64 at = sh.row_at[r0 + c + k];
                            const float f = sh.factor[r0 + c + k], y = f == 0 ? 0.0f : o[k] * f;
                            if (at < 0) continue;
                            if (partial)
                                st(reinterpret_cast<float *>(array + at) + e * 128 + key0, y);
                            else
                                st(reinterpret_cast<E *>(array + at) + e * 128 + key0, kWide && P.bf16 ? from_bits<E>(__float2bfloat16_rn(y)) : from_bits<E>(static_cast<E>(y)));
                        }
                    }
            }
            tensor_before();
        }
    } else if (warp < 12) {
        if constexpr (many) SV_CACHE_REGISTERS("dec", 56);
        if (warp == 8) {
            // -- scores^T = K Q^T
            const uint32_t leader = elected();
            constexpr uint32_t kShape = product_of(kBf16, N, false);
#pragma unroll 1
            for (int it = 0; it < n; ++it) {
                const int s = it % S::k_slots;
                if (it >= 2 && !barrier_wait(sh.weighed + (it & 1), (it >> 1 & 1) ^ 1, given)) break;  // (its scores have been read)
                if (!barrier_wait(sh.told + it % S::heads, it / S::heads & 1, given)) break;
                const auto &h = sh.head[it % S::heads];
                const int flags = __shfl_sync(~0u, h.flags, 0), segment = __shfl_sync(~0u, h.segment, 0), qb = segment % S::q_buffers;
                if (flags & kFirst && !barrier_wait(sh.q_full + qb, segment / S::q_buffers & 1, given)) break;
                if (!barrier_wait(sh.k_full + s, it / S::k_slots & 1, given)) break;
                tensor_after();
                const u64 a = matrix_at(room_at + s * S::slot, 16, 1024, 2), q = matrix_at(q_at + qb * S::q_bytes, 16, 1024, 2);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    product(tensor + (it & 1) * N, static_cast<uint32_t>(a) + (k / 4 * S::piece + k % 4 * 32) / 16, static_cast<uint32_t>(a >> 32),
                            static_cast<uint32_t>(q) + (k / 4 * (N * 128) + k % 4 * 32) / 16, static_cast<uint32_t>(q >> 32), kShape, k > 0, leader);
                products_close(sh.scores + (it & 1), leader);
                if (leader) barrier_arrive(sh.scores + (it & 1));  // (and with it what this warp has seen: the description, the queries' factors)
                products_close(sh.k_empty + s, leader);
                if (flags & kLast) products_close(sh.q_empty + qb, leader);
            }
        } else if (warp == 9) {
            // -- out^T += V^T weights^T
            const uint32_t leader = elected();
            constexpr uint32_t kShape = product_of(kBf16, N, true);
#pragma unroll 1
            for (int it = 0; it < n; ++it) {
                const int s = it % S::v_slots, b = it & 1;
                if (!barrier_wait(sh.v_full + s, it / S::v_slots & 1, given)) break;
                if (!barrier_wait(sh.weighed + b, it >> 1 & 1, given)) break;
                tensor_after();
                const auto &h = sh.head[it % S::heads];
                const bool first = __shfl_sync(~0u, h.flags & kFirst && !h.started, 0);
                // 64 elements of 8 keys are 1024 bytes; the next 64 elements are a piece further (with 64 in all: the same again,
                // into rows of the memory that nobody reads)
                const u64 a = matrix_at(room_at + (S::k_slots + s) * S::slot, D == 64 ? 0 : S::piece, 1024, 2), w = matrix_at(w_at + b * S::weights, 128, kTile * 16, 0);
#pragma unroll
                for (int e = 0; e < S::blocks; ++e)
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        product(tensor + (2 + e) * N, static_cast<uint32_t>(a) + (e * 2 * S::piece + k * 2048) / 16, static_cast<uint32_t>(a >> 32),
                                static_cast<uint32_t>(w) + k * 256 / 16, static_cast<uint32_t>(w >> 32), kShape, k > 0 || !first, leader);
                products_close(sh.done + b, leader);
                products_close(sh.v_empty + s, leader);
                products_close(sh.used + it % S::heads, leader);
            }
        } else if (warp == 10 && n > 0) {
            // -- plan: this lane has places lane, 32 + lane, ... of each tile
            walk.seek(static_cast<int>(sh.start[0]), sh.start[1], u0);
            int segment = -1;
#pragma unroll 1
            for (int it = 0; it < n; ++it) {
                // the tile's places: p0 and `places` more; a tile in parts of a page starts at its slot `slot0`
                int p0 = walk.t * P.cut.span, places = P.cut.span, c0 = walk.t * P.cut.boxes, slot0 = 0;
                if (P.cut.parts > 1) {
                    c0 = P.by_parts(walk.t);
                    slot0 = (walk.t - c0 * P.cut.parts) * P.cut.box;
                    p0 = c0 * P.s.page + slot0;
                    places = min(P.cut.box, P.s.page - slot0);
                }
                int page[4], in[4], at[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int k = w * 32 + lane, p = p0 + k, c = P.s.by_page(p);
                    page[w] = -1;
                    in[w] = loads ? k : P.cut.parts > 1 ? 0 : c - c0;  // its box, and the box's places
                    at[w] = p - c * P.s.page;
                    const int lo = loads ? p : P.cut.parts > 1 ? p0 : c * P.s.page, hi = loads ? p + 1 : P.cut.parts > 1 ? p0 + places : lo + P.s.page;
                    if (walk.rows && k < places && lo < walk.end && hi > walk.start) page[w] = ld(P.s.table + walk.i * P.s.table_stride + c);
                    if (!loads && p != lo) in[w] = -1;  // (the box's first place speaks for it)
                }
                const int k = it % S::heads;
                if (it >= S::heads && !barrier_wait(sh.used + k, (it / S::heads - 1) & 1, given)) break;
                auto &h = sh.head[k];
                bool all = true;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int p = p0 + w * 32 + lane;
                    bool there = page[w] >= 0 && page[w] < P.s.pages;
#ifdef SV_DEBUG_BOUNDS
                    const int sl = p - P.s.by_page(p) * P.s.page;
                    if (there && w * 32 + lane < places)
                        there = inside(P.kc.at + page[w] * P.kc.page + sl * P.kc.slot + walk.head * P.kc.head, D * S::bytes_of, false) &&
                                inside(P.vc.at + page[w] * P.vc.page + sl * P.vc.slot + walk.head * P.vc.head, D * S::bytes_of, false);
#endif
                    const uint32_t seen = __ballot_sync(~0u, there && w * 32 + lane < places && p >= walk.start && p < walk.end);
                    const int in_word = places - w * 32;  // (places of a tile that are none do not count)
                    all = all && seen == (in_word >= 32 ? ~0u : in_word <= 0 ? 0u : (1u << in_word) - 1);
                    if (lane == 0) h.seen[w] = seen;
                    if (in[w] >= 0 && w * 32 + lane < places) h.page[in[w]] = there ? page[w] : loads ? -1 : P.s.pages;  // (a page behind the last: zeros)
                }
                if constexpr (S::slots_told) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) h.key_slot[w * 32 + lane] = static_cast<uint16_t>(at[w]);
                }
                const bool opens = walk.t == walk.t0, ends = walk.t + 1 == walk.t1;
                const bool first = it == 0 || opens, last = it == n - 1 || ends;
                if (first) ++segment;
                if (lane == 0) {
                    const int j0 = P.by_group(walk.from), j1 = P.by_group(walk.from + walk.count - 1);
                    const bool part = walk.base < u0 || walk.base + walk.tiles() > u1;
                    all = all && places == P.cut.span && static_cast<i64>(p0) + places - 1 <= static_cast<i64>(walk.length) + j0 &&
                          (P.window <= 0 || static_cast<i64>(p0) > static_cast<i64>(walk.length) + j1 - P.window);
                    h.p0 = p0;
                    h.first = walk.first;
                    h.count = walk.count;
                    h.from = walk.from;
                    h.head = walk.head;
                    h.length = walk.length;
                    h.segment = segment;
                    h.slot = slot0;
                    h.started = 0;  // (1: sums of the segment are there before its first product)
                    h.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (part ? kPartial : 0) | (walk.base > u0 ? kSlot : 0) | (last && !ends ? kOpen : 0) | (all ? 0 : kEdge);
                    if (last && !ends) {  // the CTAs that have tiles of the group
                        h.part_first = sharer_of(total, walk.base, ctas);
                        h.part_last = sharer_of(total, walk.base + walk.tiles() - 1, ctas);
                        h.part_slot = share_of(total, h.part_first, ctas) < walk.base;
                    }
                }
                __syncwarp();
                if (lane == 0) barrier_arrive(sh.told + k);
                walk.next();
            }
        } else if (warp == 11) {
            // -- keys by boxes, and queries
            int s = 0, asked = 0, asked_q = 0;
            uint32_t turn = 0;  // times the ring has been gone round, as the parity waited for
#pragma unroll 1
            for (int it = 0; it < n; ++it) {
                if (!barrier_wait(sh.told + it % S::heads, it / S::heads & 1, given)) break;
                const auto &h = sh.head[it % S::heads];
                const int flags = h.flags, head = h.head;
                if constexpr (!many) {
                    if (!boxes_to<S>(&maps.k, sh.k_full + s, sh.k_empty + s, it >= S::k_slots, turn ^ 1, room_at + s * S::slot, P.cut, h.slot, head, h.page, lane, given)) break;
                    ++asked;
                    if (++s == S::k_slots) s = 0, turn ^= 1;
                }
                if (flags & kFirst) {
                const int segment = h.segment, qb = segment % S::q_buffers, from = h.from, count = h.count, first = h.first;
                if (segment >= S::q_buffers && !barrier_wait(sh.q_empty + qb, (segment / S::q_buffers - 1) & 1, given)) break;
                if constexpr (!kWide) {
                    ++asked_q;
                    if (lane == 0) barrier_expect(sh.q_full + qb, S::q_bytes);
                    __syncwarp();
                    const int box = P.cut.q_box;  // rows of one token side by side, so that no box has two tokens
#pragma unroll 1
                    for (int r = lane * box; r < N; r += 32 * box) {
                        const int at_row = from + r, j = P.by_group(at_row);
                        const int row = r < count ? first + j : P.s.rows;  // (a row behind the last: zeros)
#pragma unroll 1
                        for (int e = 0; e < S::halves; ++e)
                            copy_box(q_at + qb * S::q_bytes + e * (N * 128) + r * 128, &maps.q, sh.q_full + qb, e * 64, head * P.group + at_row - j * P.group, row, 0);
                    }
                } else {
                    // queries in binary16: bf16 ones times a power of two that takes the row's largest to [2^13, 2^14), exact down
                    // to 2^-28 of it
                    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;  // lanes of a row, rows at once
                    const int c = lane % kLanes;
#pragma unroll 1
                    for (int r = lane / kLanes; r < N; r += 4 * kAtOnce) {
                        uint4 x[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int rr = r + k * kAtOnce, at_row = from + min(rr, count - 1), j = P.by_group(at_row);
                            x[k] = make_uint4(0, 0, 0, 0);
                            if (rr < count)
                                x[k] = ld(reinterpret_cast<const uint4 *>(P.q + static_cast<i64>(first + j) * P.q_row + static_cast<i64>(head * P.group + at_row - j * P.group) * P.q_head) + c);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int rr = r + k * kAtOnce;
                            float less = 1.0f;
                            if (P.bf16) {
                                uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                                float most = 0;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float2 f = pair_of<__nv_bfloat16>(w[e]);
                                    most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
                                }
#pragma unroll
                                for (int d = kLanes / 2; d; d /= 2) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
                                const int up = min(110, 13 - (static_cast<int>(__float_as_uint(most) >> 23) - 127));
                                const float more = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                                less = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float2 f = pair_of<__nv_bfloat16>(w[e]);
                                    w[e] = pack<__half>(f.x * more, f.y * more);
                                }
                                x[k] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                            if (rr < N) {
                                *reinterpret_cast<uint4 *>(q_room + qb * S::q_bytes + c / 8 * (N * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = x[k];
                                if (c == 0) sh.q_scale[segment % S::kept][rr] = less;
                            }
                        }
                    }
                    shared_to_async();
                    __syncwarp();
                    if (lane == 0) barrier_arrive(sh.q_full + qb);
                }
                }
                __syncwarp();
                if (lane == 0) barrier_arrive(sh.used + it % S::heads);
            }
            if (lane == 0) {
                if (!many) sh.asked[0] = asked;
                sh.asked[2] = asked_q;
            }
        }
    } else {
        if constexpr (many) SV_CACHE_REGISTERS("dec", 56);
        if constexpr (!many) {
            if (warp == 12) {
                // -- values by boxes
                int s = 0, asked = 0;
                uint32_t turn = 0;
#pragma unroll 1
                for (int it = 0; it < n; ++it) {
                    if (!barrier_wait(sh.told + it % S::heads, it / S::heads & 1, given)) break;
                    const auto &h = sh.head[it % S::heads];
                    if (!boxes_to<S>(&maps.v, sh.v_full + s, sh.v_empty + s, it >= S::v_slots, turn ^ 1, room_at + (S::k_slots + s) * S::slot, P.cut, h.slot, h.head, h.page, lane, given)) break;
                    ++asked;
                    if (++s == S::v_slots) s = 0, turn ^= 1;
                }
                if (lane == 0) sh.asked[1] = asked;
            }
        } else {
            // -- keys (half of the warps) and values vector by vector: copied to their slot, or to a room of the thread's
            // own and widened from there. A tile is given on when kLag more have been asked for. 8 bits in pages that boxes can
            // bring: the first warp of each half has them copied by tensor map, and every thread widens its vectors of the tile.
            constexpr bool kRaw = kWide && !loads;
            constexpr int kSide = 16 * S::loaders;  // threads
            const bool values = warp >= 12 + S::loaders / 2;
            constexpr int kRow = D * S::bytes_of / 16, kEvery = kSide / kRow, kEach = kTile / kEvery;  // vectors of a key; keys at once; a thread's vectors
            constexpr int kLag = kWide ? S::staged - 1 : S::k_slots > 2 ? S::k_slots - 2 : S::k_slots - 1;
            const int x = (tid - 384) % kSide, c = x % kRow, key0 = x / kRow, slots = values ? S::v_slots : S::k_slots;
            const Cache &cache = values ? P.vc : P.kc;
            // (strides in vectors of 16 bytes, below 2^32)
            const uint32_t by_page = static_cast<uint32_t>(cache.page >> 4), by_slot = static_cast<uint32_t>(cache.slot >> 4);
            u64 *const fulls = values ? sh.v_full : sh.k_full, *const empties = values ? sh.v_empty : sh.k_empty;
            unsigned char *const ring = room + (values ? S::k_slots * S::slot : 0);
            auto place_of = [&](unsigned char *slot, int chunk, int key) { return slot + chunk / 8 * S::piece + key * 128 + (((chunk & 7) ^ (key & 7)) << 4); };
            auto own = [&](int it, int k) { return staging + (((it % S::rooms * 2 + values) * kEach + k) * kSide + x) * 16; };
            int asked = 0, passed = 0, boxes = 0;  // slots; tiles asked for by tensor map
            uint32_t asked_turn = 0, passed_turn = 0;
#pragma unroll 1
            for (int it = 0; it < n + kLag; ++it) {
                if (kRaw && it < n && warp == (values ? 12 + S::loaders / 2 : 12)) {
                    const int r = it % S::rooms;
                    if (!barrier_wait(sh.told + it % S::heads, it / S::heads & 1, given)) break;
                    if (it >= S::rooms && !barrier_wait(&sh.raw_empty[values][r], (it / S::rooms - 1) & 1, given)) break;
                    ++boxes;
                    const auto &h = sh.head[it % S::heads];
                    if (lane == 0) barrier_expect(&sh.raw_full[values][r], P.cut.boxes * P.cut.box * D);
                    __syncwarp();
                    if (lane < P.cut.boxes)  // (at most 16)
                        copy_box(shared_address(staging + (r * 2 + values) * (kTile * D) + lane * P.cut.box * D), values ? &maps.v : &maps.k, &sh.raw_full[values][r], 0, h.slot, h.head, h.page[lane]);
                }
                if (!kRaw && it < n) {
                    if (!barrier_wait(sh.told + it % S::heads, it / S::heads & 1, given)) break;
                    if (!kWide && it >= slots && !barrier_wait(empties + asked, asked_turn ^ 1, given)) break;
                    const auto &h = sh.head[it % S::heads];
                    const uint4 *const at = reinterpret_cast<const uint4 *>(cache.at + static_cast<i64>(h.head) * cache.head) + c;
                    constexpr int kPart = kEach < 8 ? kEach : 8;
#pragma unroll 1
                    for (int k0 = 0; k0 < kEach; k0 += kPart) {
                        const uint4 *from[kPart];
                        uint32_t there = 0;
#pragma unroll
                        for (int k = 0; k < kPart; ++k) {
                            const int key = key0 + (k0 + k) * kEvery, page = h.page[key], p = h.p0 + key;
                            const uint32_t slot = S::slots_told ? h.key_slot[S::slots_told ? key : 0] : static_cast<uint32_t>(p - P.s.by_page(p) * P.s.page);
                            from[k] = page >= 0 ? at + (static_cast<u64>(static_cast<uint32_t>(page)) * by_page + static_cast<u64>(slot) * by_slot) : at;
                            there |= static_cast<uint32_t>(page >= 0) << k;
                        }
#pragma unroll
                        for (int k = 0; k < kPart; ++k)
                            copy16(kWide ? own(it, k0 + k) : place_of(ring + asked * S::slot, c, key0 + (k0 + k) * kEvery), from[k], there >> k & 1);
                    }
                    if (++asked == slots) asked = 0, asked_turn ^= 1;
                }
                if (!kRaw) copies_close();
                if (it < kLag) continue;
                if (!kRaw) copies_wait<kLag>();
                const int raw = kRaw ? (it - kLag) % S::rooms : 0;
                if (kRaw && !barrier_wait(&sh.raw_full[values][raw], (it - kLag) / S::rooms & 1, given)) break;
                if constexpr (kWide) {
                    if (it - kLag >= slots && !barrier_wait(empties + passed, passed_turn ^ 1, given)) break;
                    // (of the lanes of a key those of the upper half write their second vector first: eight lanes, eight banks)
                    const bool second = kRow == 8 ? c >> 2 : kRow == 4 ? 0 : c >> 2 & 1;
                    constexpr int kPart = kEach < 4 ? kEach : 4;
#pragma unroll 1
                    for (int k0 = 0; k0 < kEach; k0 += kPart) {
                        uint4 v[kPart];
#pragma unroll
                        for (int k = 0; k < kPart; ++k) v[k] = *reinterpret_cast<const uint4 *>(kRaw ? staging + ((raw * 2 + values) * kTile + key0 + (k0 + k) * kEvery) * D + c * 16 : own(it - kLag, k0 + k));
#pragma unroll
                        for (int k = 0; k < kPart; ++k) {
                            const uint4 lo = make_uint4(half2_of_e4m3(v[k].x), half2_of_e4m3(v[k].x >> 16), half2_of_e4m3(v[k].y), half2_of_e4m3(v[k].y >> 16));
                            const uint4 hi = make_uint4(half2_of_e4m3(v[k].z), half2_of_e4m3(v[k].z >> 16), half2_of_e4m3(v[k].w), half2_of_e4m3(v[k].w >> 16));
                            const int key = key0 + (k0 + k) * kEvery;
                            *reinterpret_cast<uint4 *>(place_of(ring + passed * S::slot, 2 * c + second, key)) = second ? hi : lo;
                            *reinterpret_cast<uint4 *>(place_of(ring + passed * S::slot, 2 * c + !second, key)) = second ? lo : hi;
                        }
                    }
                }
                shared_to_async();
                __syncwarp();
                if (kRaw && lane == 0) barrier_arrive(&sh.raw_empty[values][raw]);
                if (lane == 0) barrier_arrive(fulls + passed);
                if (++passed == slots) passed = 0, passed_turn ^= 1;
            }
            if (kRaw && lane == 0 && warp == (values ? 12 + S::loaders / 2 : 12)) sh.asked[values] = boxes;
        }
    }
    tensor_before();
    __syncthreads();
    if (__builtin_expect(*reinterpret_cast<volatile int *>(&given->up), 0)) {  // (all threads see the same: no one waits any more)
        // -- given up: what is on the way ends before the block does, and the rows that it had get NaN
        if (loads) asm volatile("cp.async.wait_all;" ::: "memory");
        if (warp == 8 || warp == 9) products_close(&sh.ended, elected());
        if (tid == 0) {
            atomicOr(&g_cache_error, SV_ERR_WAIT);
            if constexpr (!loads) {
                barrier_drain(kWide ? &sh.raw_full[0][0] : sh.k_full, kWide ? S::rooms : S::k_slots, sh.asked[0]);
                barrier_drain(kWide ? &sh.raw_full[1][0] : sh.v_full, kWide ? S::rooms : S::v_slots, sh.asked[1]);
            }
            if constexpr (!kWide) barrier_drain(sh.q_full, S::q_buffers, sh.asked[2]);
            barrier_drain(&sh.ended, 1, 1);
        }
        if (warp < 8) rows_lost<N, D, E>(P, sh.start, sh.total);  // (these have registers for it)
        __syncthreads();
    }
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tensor), "n"(S::columns) : "memory");
}

// Joins the parts of the groups that more than one CTA has. A group over k + 1 CTAs has k CTAs here, which share its
// outputs; a few lanes take the parts of four elements, up to four parts of a lane at once. What it takes is three trips to
// memory, one after the other.
constexpr int kJoinThreads = 512;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) sv_cache_join_kernel(const AttentionParams P, int rows, float offset)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 a = ld(reinterpret_cast<const int4 *>(P.parts + blockIdx.x)), b = ld(reinterpret_cast<const int4 *>(P.parts + blockIdx.x) + 1);
    const int first = a.x, last = a.y, row0 = a.w, from = b.x, count = b.y, head = b.z;
    if (first < 0) return;
    const int share = last - first, mine = static_cast<int>(blockIdx.x) - first, items = count * (D / 4);
    const int lo = items * mine / share, hi = items * (mine + 1) / share;
    // as many lanes as there is room for, and no more than there are parts
    int lanes = 1;
    while (lanes < 32 && lanes <= share && (hi - lo) * lanes * 2 <= kJoinThreads) lanes *= 2;
    const int each = kJoinThreads / lanes, lane = threadIdx.x & (lanes - 1), nth = threadIdx.x / lanes;
    const float vs = P.v_scale ? ld(P.v_scale + head) : 1.0f;
#pragma unroll 1
    for (int base = lo; base < hi; base += each) {
        const int item = base + nth;
        const bool there = item < hi;
        const int r = there ? item / (D / 4) : 0, c = there ? item % (D / 4) * 4 : 0;
        float most = -kInf, z = 0;
        float4 y = make_float4(0, 0, 0, 0);
#pragma unroll 1
        for (int k0 = lane; k0 <= share; k0 += 4 * lanes) {
            float2 s[4];
            float4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int q = k0 + k * lanes;
                const i64 part = (static_cast<i64>(first + q) * 2 + (q == 0 ? a.z : 0)) * rows + r;
                s[k] = make_float2(-kInf, 0);
                v[k] = make_float4(0, 0, 0, 0);
                if (q <= share) s[k] = ld(P.stats + part), v[k] = ld(reinterpret_cast<const float4 *>(P.sums + part * D + c));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float up = larger(most, s[k].x), at = up == -kInf ? 0.0f : up;
                const float f = exp2_fast(most - at), g = s[k].x == up ? 1.0f : exp2_fast(s[k].x - at);
                z = z * f + s[k].y * g;
                y = make_float4(y.x * f + v[k].x * g, y.y * f + v[k].y * g, y.z * f + v[k].z * g, y.w * f + v[k].w * g);
                most = up;
            }
        }
#pragma unroll 1
        for (int d = lanes / 2; d; d /= 2) {
            const float up = larger(most, __shfl_xor_sync(~0u, most, d)), at = up == -kInf ? 0.0f : up, f = exp2_fast(most - at);
            auto add = [&](float &v) {
                v *= f;
                v += __shfl_xor_sync(~0u, v, d);
            };
            add(z), add(y.x), add(y.y), add(y.z), add(y.w);
            most = up;
        }
        if (!there || lane != 0) continue;
        const int at_row = from + r, j = P.by_group(at_row), qh = head * P.group + at_row - j * P.group;
        const float f = z == 0 ? 0.0f : vs / z;
        if (z == 0) y = make_float4(0, 0, 0, 0);
        const uint2 w = P.bf16 ? make_uint2(pack<__nv_bfloat16>(y.x * f, y.y * f), pack<__nv_bfloat16>(y.z * f, y.w * f))
                               : make_uint2(pack<__half>(y.x * f, y.y * f), pack<__half>(y.z * f, y.w * f));
        st(reinterpret_cast<uint2 *>(P.out + (row0 + j) * P.out_row + qh * P.out_head + c * 2), w);
        if (c == 0 && P.lse) st(P.lse + static_cast<i64>(row0 + j) * P.hq + qh, z == 0 ? -kInf : (most - offset + log2f(z)) * kLn2);
    }
}

}  // namespace sv_cache
