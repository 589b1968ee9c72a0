// Attention of a step's rows over the paged cache by the tensor cores' own memory (16-bit caches). See
// sv_cache.cu for the mathematics.
#pragma once

#include <cuda.h>

#include "sv_cache_attention.cuh"

namespace sv_cache {

// A tile is 128 keys. Both products have the keys or the elements in the 128 rows of the tensor cores' memory and
// the query rows (N, 16 to 64) in its columns: scores^T = K Q^T, and out^T += V^T weights^T. So few query rows
// waste nothing, and every key is read from shared memory once for all of them. Roles: four warps for the weights (a
// thread has one key's scores of all rows), one thread that issues the products, one warp that goes through the tiles
// and the page table ahead of the others, one that copies keys and queries and one that copies values.
template <int D, int N>
struct Tensor {
    static constexpr int tokens = 128;
    static constexpr int rows = N;
    static constexpr int halves = D / 64;            // pieces of 64 elements, 128 bytes a key: the copies' swizzle
    static constexpr int slot = tokens * D * 2;      // keys or values of a tile
    static constexpr int q_bytes = N * D * 2;
    static constexpr int weights = tokens * N * 2;
    static constexpr int q_buffers = D == 256 && N > 16 || N == 64 ? 1 : 2;
    static constexpr int heads = D == 256 && N > 16 ? 3 : 8;  // descriptions of tiles that are kept
    static constexpr int fit = (heads == 8 ? 225800 : 229376) - q_buffers * q_bytes - 2 * weights;
    static constexpr int slots = fit / slot > 12 ? 12 : fit / slot;
    static constexpr int k_slots = slots / 2, v_slots = slots - slots / 2;  // rings of their own: each has one warp that fills it
    static constexpr int blocks = D == 256 ? 2 : 1;  // of 128 elements
    static constexpr int columns_used = (2 + blocks) * N;
    static constexpr int columns = columns_used <= 64 ? 64 : columns_used <= 128 ? 128 : 256;
    static constexpr int threads = 256;
    static_assert(slots >= 2 && columns_used <= 256, "room");
    struct Head {
        int p0, first, count, from, row0, head, length, flags;
        int part_first, part_last, part_slot, segment;
        uint32_t seen[4];
        int page[tokens];  // of each box
    };
    struct Shared {
        u64 k_full[k_slots], k_empty[k_slots], v_full[v_slots], v_empty[v_slots], scores[2], weighed[2], done[2], q_empty[2], told[heads], used[heads];
        Head head[heads];
        alignas(16) float less[N];    // minus the reference of each row's weights (plus the offset)
        alignas(16) float top[N];     // the reference, times log2 e
        alignas(16) float factor[N];  // what a new reference makes of the old sums
        alignas(16) float most[4][N];
        float sum[N];
        i64 scan[threads / 32];
        i64 start[2];
        uint32_t tensor_at;
        int lost;
    };
    static constexpr int bytes = slots * slot + q_buffers * q_bytes + 2 * weights + static_cast<int>(sizeof(Shared));
    static_assert(bytes <= 232448, "shared memory");
};

enum : int { kEdge = 32 };

// ---------------------------------------------------------------------------------------
// barriers, copies, products
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void barrier_init(u64 *b, int count) { asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(shared_address(b)), "r"(count) : "memory"); }
__device__ __forceinline__ void barrier_expect(u64 *b, int bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(shared_address(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void barrier_arrive(u64 *b) { asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(shared_address(b)) : "memory"); }
// Waits for a phase to end, not for ever: after kPatience looks the call is given up (`lost`), every later wait
// returns at once, and the rows get NaN.
constexpr int kPatience = 1 << 22;
__device__ __forceinline__ bool barrier_try(u64 *b, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared.b64 p, [%1], %2;\nselp.b32 %0, 1, 0, p;\n}" : "=r"(done) : "r"(shared_address(b)), "r"(parity) : "memory");
    return done != 0;
}
__device__ __forceinline__ void barrier_wait(u64 *b, uint32_t parity, int *lost)
{
    if (barrier_try(b, parity)) return;
    for (int k = 0; k < kPatience; ++k) {
        if (barrier_try(b, parity)) return;
        if (*reinterpret_cast<volatile int *>(lost)) return;
    }
    *reinterpret_cast<volatile int *>(lost) = 1;
}
// A box of the cache, [slots][64 elements], to shared memory (swizzled by 128 bytes).
__device__ __forceinline__ void copy_box(uint32_t to, const CUtensorMap *map, u64 *b, int element, int slot, int head, int page)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(to), "l"(map),
                 "r"(shared_address(b)), "r"(element), "r"(slot), "r"(head), "r"(page)
                 : "memory");
}
__device__ __forceinline__ void copy_row(uint32_t to, const CUtensorMap *map, u64 *b, int element, int head, int row)
{
    copy_box(to, map, b, element, head, row, 0);
}
// Description of a matrix in shared memory: address, the two strides in bytes, and the swizzle (2: 128 bytes, 0: none).
__device__ __forceinline__ u64 matrix_at(uint32_t at, uint32_t lead, uint32_t stride, u64 swizzle)
{
    return static_cast<u64>((at & 0x3ffff) >> 4) | static_cast<u64>(lead >> 4) << 16 | static_cast<u64>(stride >> 4) << 32 | u64{1} << 46 | swizzle << 61;
}
// Shape of a product of 16-bit elements, 128 x N, into binary32; whether A and B have their rows contiguous.
__host__ __device__ constexpr uint32_t product_of(bool bf16, int n, bool turned)
{
    return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (turned ? 3u : 0u) << 15 | static_cast<uint32_t>(n >> 3) << 17 | 8u << 24;
}
__device__ __forceinline__ void product(uint32_t d, u64 a, u64 b, uint32_t shape, bool add)
{
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(shape),
                 "r"(static_cast<int>(add))
                 : "memory");
}
// An arrival at b when all products issued so far have ended.
__device__ __forceinline__ void products_close(u64 *b)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"l"(static_cast<u64>(shared_address(b))) : "memory");
}
__device__ __forceinline__ void tensor_load16(float *v, uint32_t at)
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
}
__device__ __forceinline__ void tensor_store16(uint32_t at, const float *v)
{
    uint32_t r[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(v[k]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]),
        "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(at)
        : "memory");
}
__device__ __forceinline__ void tensor_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tensor_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tensor_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void shared_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// The four warps of the weights among themselves.
__device__ __forceinline__ void weights_meet() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool weights_any(bool x)
{
    int any;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\nbar.red.or.pred q, 2, 128, p;\nselp.b32 %0, 1, 0, q;\n}" : "=r"(any) : "r"(static_cast<int>(x)) : "memory");
    return any != 0;
}
// The larger number; NaN if one is.
__device__ __forceinline__ float larger(float a, float b)
{
    float c;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
    return c;
}
// The largest of a warp's numbers (as whole numbers of the same order), NaN if one is.
__device__ __forceinline__ float warp_largest(float x)
{
    int i = __float_as_int(x);
    i ^= i >> 31 & 0x7fffffff;
    i = __reduce_max_sync(~0u, i);
    return __int_as_float(i ^ (i >> 31 & 0x7fffffff));
}

struct TensorMaps {
    CUtensorMap q, k, v;
};

// Weights relative to a reference that is the row's largest score when it is set, and is set anew when some score is
// kSlack doublings above it: in bf16 (range of binary32) rarely, in binary16 so that weights stay below 2^15, with
// kOffset doublings up, so that the smallest step of a weight is 2^-35.
template <bool BF16>
struct Weights {
    static constexpr float offset = BF16 ? 0.0f : 11.0f, slack = BF16 ? 8.0f : 4.0f;
};

template <bool BF16, int D, int N>
__global__ void __launch_bounds__(256, 1) sv_cache_tensor_kernel(const AttentionParams P, const __grid_constant__ TensorMaps maps, const int box)
{
    using S = Tensor<D, N>;
    using E = std::conditional_t<BF16, __nv_bfloat16, __half>;
    using W = Weights<BF16>;
    extern __shared__ __align__(1024) unsigned char room[];
    unsigned char *const q_room = room + S::slots * S::slot, *const w_room = q_room + S::q_buffers * S::q_bytes;
    auto &sh = *reinterpret_cast<typename S::Shared *>(w_room + 2 * S::weights);
    const uint32_t room_at = shared_address(room), q_at = shared_address(q_room), w_at = shared_address(w_room);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    const int cta = blockIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // -- this CTA's tiles, barriers, memory
    if (tid == 0) {
        for (int k = 0; k < S::k_slots; ++k) barrier_init(sh.k_full + k, 1), barrier_init(sh.k_empty + k, 1);
        for (int k = 0; k < S::v_slots; ++k) barrier_init(sh.v_full + k, 1), barrier_init(sh.v_empty + k, 1);
        for (int k = 0; k < 2; ++k) barrier_init(sh.scores + k, 1), barrier_init(sh.weighed + k, 128), barrier_init(sh.done + k, 1), barrier_init(sh.q_empty + k, 1);
        for (int k = 0; k < S::heads; ++k) barrier_init(sh.told + k, 1), barrier_init(sh.used + k, 1);
        sh.lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        shared_to_async();
    }
    Walk<S> walk(P);
    const int per = (P.s.n + S::threads - 1) / S::threads;
    i64 mine = 0;
    for (int k = tid * per; k < min(P.s.n, (tid + 1) * per); ++k) mine += walk.request_tiles(k);
    i64 before = mine;
    for (int d = 1; d < 32; d *= 2) {
        const i64 up = __shfl_up_sync(~0u, before, d);
        if (lane >= d) before += up;
    }
    if (lane == 31) sh.scan[warp] = before;
    __syncthreads();
    i64 total = 0, ahead = 0;
    for (int w = 0; w < S::threads / 32; ++w) {
        if (w == warp) ahead = total;
        total += sh.scan[w];
    }
    before += ahead - mine;
    const int ctas = static_cast<int>(min(total, static_cast<i64>(gridDim.x)));  // (each with a tile at least)
    if (cta >= ctas) {
        if (P.parts && tid == 0) st(&P.parts[cta].first, -1);
        return;
    }
    if (warp == 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_address(&sh.tensor_at)), "n"(S::columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const i64 u0 = total * cta / ctas, u1 = total * (cta + 1) / ctas;
    const int n = static_cast<int>(u1 - u0);
    if (u0 >= before && u0 < before + mine) {
        i64 at = before;
        for (int k = tid * per; k < min(P.s.n, (tid + 1) * per); ++k) {
            const i64 here = walk.request_tiles(k);
            if (u0 < at + here) {
                sh.start[0] = k;
                sh.start[1] = u0 - at;
                break;
            }
            at += here;
        }
    }
    tensor_before();
    __syncthreads();
    tensor_after();
    const uint32_t tensor = sh.tensor_at;
    int *const lost = &sh.lost;

    if (warp == 5) {
        // -- descriptions of the tiles: this lane has places lane, 32 + lane, ... of each
        walk.seek(static_cast<int>(sh.start[0]), sh.start[1], u0);
        int segment = -1;
        int page[4];
        auto look_up = [&] {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int p = walk.t * S::tokens + w * 32 + lane;
                // (all places of a box that some row sees a place of)
                const int in = p & ~(box - 1);
                page[w] = -1;
                if (walk.rows && in < walk.range.end && in + box > walk.range.start) {
                    const int c = p < (1 << 22) ? static_cast<int>((static_cast<u64>(p) * P.s.page_magic) >> 42) : p / P.s.page;
                    page[w] = ld(P.s.table + walk.i * P.s.table_stride + c);
#ifdef SV_DEBUG_BOUNDS
                    const int pg = page[w], slot = p - c * P.s.page;
                    if (pg >= 0 && pg < P.s.pages)
                        inside(P.kc.at + pg * P.kc.page + slot * P.kc.slot + walk.head * P.kc.head, D * 2, false),
                            inside(P.vc.at + pg * P.vc.page + slot * P.vc.slot + walk.head * P.vc.head, D * 2, false);
#endif
                }
            }
        };
        look_up();
        for (int it = 0; it < n; ++it) {
            const int k = it % S::heads;
            if (it >= S::heads) barrier_wait(sh.used + k, (it / S::heads - 1) & 1, lost);
            auto &h = sh.head[k];
            const int p0 = walk.t * S::tokens;
            bool all = true;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int p = p0 + w * 32 + lane;
                const bool there = page[w] >= 0 && page[w] < P.s.pages;
                const uint32_t seen = __ballot_sync(~0u, there && p >= walk.range.start && p < walk.range.end);
                all = all && seen == ~0u;
                if (lane == 0) h.seen[w] = seen;
                if ((p & (box - 1)) == 0) h.page[(w * 32 + lane) / box] = there ? page[w] : P.s.pages;  // (a page behind the last: zeros)
            }
            const bool opens = walk.t == walk.range.t0, ends = walk.t + 1 == walk.range.t1;
            const bool first = it == 0 || opens, last = it == n - 1 || ends;
            if (first) ++segment;
            if (lane == 0) {
                const int j0 = walk.from / P.group, j1 = (walk.from + walk.count - 1) / P.group;
                const bool part = walk.base < u0 || walk.base + walk.tiles() > u1;
                all = all && static_cast<i64>(p0) + S::tokens - 1 <= static_cast<i64>(walk.length) + j0 &&
                      (P.window <= 0 || static_cast<i64>(p0) > static_cast<i64>(walk.length) + j1 - P.window);
                h.p0 = p0;
                h.first = walk.first;
                h.count = walk.count;
                h.from = walk.from;
                h.head = walk.head;
                h.length = walk.length;
                h.segment = segment;
                h.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (part ? kPartial : 0) | (walk.base > u0 ? kSlot : 0) | (last && !ends ? kOpen : 0) | (all ? 0 : kEdge);
                if (last && !ends) {  // the CTAs that have tiles of the group
                    h.part_first = static_cast<int>(((walk.base + 1) * ctas - 1) / total);
                    h.part_last = static_cast<int>(((walk.base + walk.tiles()) * ctas - 1) / total);
                    h.part_slot = total * h.part_first / ctas < walk.base;
                }
            }
            __syncwarp();
            if (lane == 0) barrier_arrive(sh.told + k);
            walk.next();
            if (it + 1 < n) look_up();
        }
    } else if (warp >= 6) {
        // -- copies: keys (and queries) or values, by boxes of `box` places, a power of two that divides the page
        const bool values = warp == 7;
        const CUtensorMap *const map = values ? &maps.v : &maps.k;
        const int boxes = S::tokens / box;
        const int slots = values ? S::v_slots : S::k_slots;
        u64 *const fulls = values ? sh.v_full : sh.k_full, *const empties = values ? sh.v_empty : sh.k_empty;
        const uint32_t ring = room_at + (values ? S::k_slots * S::slot : 0);
        int s = 0;
        uint32_t turn = 0;  // times the ring has been gone round, as the parity waited for
        for (int it = 0; it < n; ++it) {
            const int k = it % S::heads;
            u64 *const full = fulls + s;
            barrier_wait(sh.told + k, it / S::heads & 1, lost);
            const auto &h = sh.head[k];
            const int flags = h.flags, head = h.head, p0 = h.p0;
            if (it >= slots) barrier_wait(empties + s, turn ^ 1, lost);
            if (lane == 0) barrier_expect(full, S::slot + (flags & kFirst && !values ? S::q_bytes : 0));
            __syncwarp();
            for (int b = lane; b < boxes; b += 32) {
                const int p = p0 + b * box, c = p < (1 << 22) ? static_cast<int>((static_cast<u64>(p) * P.s.page_magic) >> 42) : p / P.s.page;
                const int page = h.page[b];
#pragma unroll
                for (int e = 0; e < S::halves; ++e)
                    copy_box(ring + s * S::slot + e * (S::tokens * 128) + b * box * 128, map, full, e * 64, p - c * P.s.page, head, page);
            }
            if (flags & kFirst && !values) {
                const int segment = h.segment, qb = segment % S::q_buffers, from = h.from, count = h.count, first = h.first;
                if (segment >= S::q_buffers) barrier_wait(sh.q_empty + qb, (segment / S::q_buffers - 1) & 1, lost);
                __syncwarp();
                for (int r = lane; r < N; r += 32) {
                    const int at_row = from + r, j = at_row / P.group;
                    const int row = r < count ? first + j : P.s.rows;  // (a row behind the last: zeros)
#pragma unroll
                    for (int e = 0; e < S::halves; ++e)
                        copy_row(q_at + qb * S::q_bytes + e * (N * 128) + r * 128, &maps.q, full, e * 64, head * P.group + at_row - j * P.group, row);
                }
            }
            if (++s == slots) s = 0, turn ^= 1;
        }
        if (*reinterpret_cast<volatile int *>(lost))  // copies in flight end before the block does
            for (int it = max(0, n - slots); it < n; ++it)
                for (int k = 0; k < kPatience && !barrier_try(fulls + it % slots, it / slots & 1); ++k) {
                }
    } else if (warp == 4) {
        // -- products
        if (lane == 0) {
            constexpr uint32_t kScores = product_of(BF16, N, false), kOut = product_of(BF16, N, true);
            int qb = 0;
            auto scores = [&](int it) {
                const int s = it % S::k_slots;
                barrier_wait(sh.k_full + s, it / S::k_slots & 1, lost);
                tensor_after();
                const auto &h = sh.head[it % S::heads];
                const int flags = h.flags;
                qb = h.segment % S::q_buffers;
                const uint32_t k_at = room_at + s * S::slot, qa = q_at + qb * S::q_bytes;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    product(tensor + (it & 1) * N, matrix_at(k_at + k / 4 * (S::tokens * 128) + k % 4 * 32, 16, 1024, 2),
                            matrix_at(qa + k / 4 * (N * 128) + k % 4 * 32, 16, 1024, 2), kScores, k > 0);
                products_close(sh.scores + (it & 1));
                products_close(sh.k_empty + s);
                if (flags & kLast) products_close(sh.q_empty + qb);
            };
            scores(0);
            for (int it = 0; it < n; ++it) {
                if (it + 1 < n) scores(it + 1);
                const int s = it % S::v_slots, b = it & 1;
                barrier_wait(sh.weighed + b, it >> 1 & 1, lost);
                barrier_wait(sh.v_full + s, it / S::v_slots & 1, lost);
                tensor_after();
                const bool first = sh.head[it % S::heads].flags & kFirst;
                const uint32_t v_at = room_at + (S::k_slots + s) * S::slot, wa = w_at + b * S::weights;
                // 64 elements of 8 keys are 1024 bytes; the next 64 elements are a piece further (with 64 in all: the same again,
                // into rows of the memory that nobody reads)
#pragma unroll
                for (int e = 0; e < S::blocks; ++e)
#pragma unroll
                    for (int k = 0; k < S::tokens / 16; ++k)
                        product(tensor + (2 + e) * N, matrix_at(v_at + e * 2 * (S::tokens * 128) + k * 2048, D == 64 ? 0 : S::tokens * 128, 1024, 2),
                                matrix_at(wa + k * 256, 128, 2048, 0), kOut, k > 0 || !first);
                products_close(sh.done + b);
                products_close(sh.v_empty + s);
                products_close(sh.used + it % S::heads);
            }
        }
        __syncwarp();
    } else {
        // -- weights: this thread has the key `tid` of every tile, and the elements tid and tid + 128 of the outputs
        const uint32_t lanes = static_cast<uint32_t>(warp) << 21;  // (lane 32 * warp of the tensor memory, in bits 16 and up)
        float sum[N];
        float scale = 0;
        for (int it = 0; it < n; ++it) {
            const int b = it & 1;
            barrier_wait(sh.told + it % S::heads, it / S::heads & 1, lost);
            barrier_wait(sh.scores + b, it >> 1 & 1, lost);
            tensor_after();
            const auto &h = sh.head[it % S::heads];
            const int flags = h.flags, head = h.head, from = h.from, count = h.count, first_row = h.first;
            float s[N];
#pragma unroll
            for (int c = 0; c < N; c += 16) tensor_load16(s + c, tensor + lanes + b * N + c);
            if (flags & kFirst) {
                scale = P.scale * (P.k_scale ? ld(P.k_scale + head) : 1.0f);
#pragma unroll
                for (int r = 0; r < N; ++r) sum[r] = 0;
            }
            tensor_loaded();
            int r_lo = 0, r_hi = N;  // the rows that see this thread's key
            if (flags & kEdge) {
                const i64 d = static_cast<i64>(h.p0) + tid - h.length;  // it is the d-th new token's place
                const i64 lo = d <= 0 ? 0 : d * P.group - from, hi = P.window > 0 ? (d + P.window) * P.group - from : N;
                r_lo = static_cast<int>(min(max(lo, 0ll), static_cast<i64>(N)));
                r_hi = static_cast<int>(min(max(hi, 0ll), static_cast<i64>(N)));
                if (!(h.seen[tid / 32] >> (tid & 31) & 1)) r_hi = 0;
                // A weight of 0 times a value that is not finite would be NaN. Such elements, if any, are set to 0 in shared
                // memory, and what they make of the rows that see them is added by hand.
                const int vslot = it % S::v_slots;
                barrier_wait(sh.v_full + vslot, it / S::v_slots & 1, lost);
                unsigned char *const v = room + (S::k_slots + vslot) * S::slot;
                auto chunk = [&](int key, int c) { return reinterpret_cast<uint4 *>(v + c / 8 * (S::tokens * 128) + key * 128 + ((c & 7 ^ key & 7) << 4)); };
                constexpr uint32_t mask = BF16 ? 0x7f80u : 0x7c00u;
                bool odd = false;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 x = *chunk(tid, c);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t w = k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w;
                        odd |= (w & mask) == mask || (w >> 16 & mask) == mask;
                    }
                }
                if (weights_any(odd)) {
                    // (rare: one row at a time, every element over all keys)
                    if (it > 0) barrier_wait(sh.done + (b ^ 1), (it - 1) >> 1 & 1, lost);
                    tensor_after();
                    for (int e = 0; e < S::blocks; ++e)
                        for (int r = 0; r < N; ++r) {
                            const uint32_t at = tensor + lanes + (2 + e) * N + r;
                            uint32_t w;
                            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(w) : "r"(at) : "memory");
                            tensor_loaded();
                            float x = flags & kFirst ? 0.0f : __uint_as_float(w);
                            const int element = e * 128 + tid;
                            for (int key = 0; key < S::tokens && element < D; ++key) {
                                const i64 dk = static_cast<i64>(h.p0) + key - h.length;
                                if (!(h.seen[key / 32] >> (key & 31) & 1) || (dk > 0 && r < dk * P.group - from) || (P.window > 0 && r >= (dk + P.window) * P.group - from)) continue;
                                const float y = static_cast<float>(reinterpret_cast<const E *>(chunk(key, element / 8))[element & 7]);
                                if (!(fabsf(y) < kInf)) x += y;
                            }
                            __syncwarp();
                            asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(at), "r"(__float_as_uint(x)) : "memory");
                        }
                    tensor_stored();
                    tensor_before();
                    weights_meet();
                    for (int c = 0; c < D / 8; ++c) {
                        uint32_t *x = reinterpret_cast<uint32_t *>(chunk(tid, c));
                        for (int k = 0; k < 4; ++k) {
                            if ((x[k] & mask) == mask) x[k] &= 0xffff0000u;
                            if ((x[k] >> 16 & mask) == mask) x[k] &= 0xffffu;
                        }
                    }
                    shared_to_async();
                    if (tid == 0) sh.head[it % S::heads].flags = flags & ~kFirst;  // (the sums have been started)
                }
            }

            // the scores relative to the reference; a new one where some score is too far above it
            float far = -kInf;
            auto relative = [&] {
#pragma unroll
                for (int r = 0; r < N; r += 4) {
                    const float4 less = *reinterpret_cast<const float4 *>(sh.less + r);
                    s[r] = fmaf(s[r], scale, less.x), s[r + 1] = fmaf(s[r + 1], scale, less.y);
                    s[r + 2] = fmaf(s[r + 2], scale, less.z), s[r + 3] = fmaf(s[r + 3], scale, less.w);
                }
                if (flags & kEdge) {
#pragma unroll
                    for (int r = 0; r < N; ++r)
                        if (r < r_lo || r >= r_hi) s[r] = -kInf;
                }
            };
            bool renew = flags & kFirst;
            if (!renew) {
                relative();
#pragma unroll
                for (int r = 0; r < N; ++r) far = fmaxf(far, s[r]);
                renew = weights_any(far > W::offset + W::slack);
                if (renew) {  // (the scores once more)
#pragma unroll
                    for (int c = 0; c < N; c += 16) tensor_load16(s + c, tensor + lanes + b * N + c);
                    tensor_loaded();
                }
            }
            if (renew) {
                float own[N / 16 > 2 ? 2 : 1];
                own[0] = 0;
                if constexpr (N > 32) own[1] = 0;
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    const float most = warp_largest(r < r_lo || r >= r_hi ? -kInf : s[r] * scale);
                    if (lane == (r & 31)) own[r / 32] = most;
                }
                if (lane < N) sh.most[warp][lane] = own[0];
                if constexpr (N > 32) {
                    if (lane < N - 32) sh.most[warp][lane + 32] = own[1];
                }
                weights_meet();
                if (tid < N) {
                    const float old = flags & kFirst ? -kInf : sh.top[tid];
                    const float top = larger(larger(larger(sh.most[0][tid], sh.most[1][tid]), larger(sh.most[2][tid], sh.most[3][tid])), old);
                    sh.factor[tid] = top == old ? 1.0f : exp2_fast(old - top);
                    sh.top[tid] = top;
                    sh.less[tid] = top == -kInf ? 0x1p120f : W::offset - top;  // (no key yet: any score is far above)
                }
                weights_meet();
                if (!(flags & kFirst)) {
                    barrier_wait(sh.done + (b ^ 1), (it - 1) >> 1 & 1, lost);
                    tensor_after();
#pragma unroll 1
                    for (int c = 0; c < S::blocks * N; c += 16) {
                        float o[16];
                        tensor_load16(o, tensor + lanes + 2 * N + c);
                        tensor_loaded();
#pragma unroll
                        for (int r = 0; r < 16; ++r) o[r] *= sh.factor[(c % N) + r];
                        tensor_store16(tensor + lanes + 2 * N + c, o);
                    }
                    tensor_stored();
                    tensor_before();
#pragma unroll
                    for (int r = 0; r < N; ++r) sum[r] *= sh.factor[r];
                }
                relative();
            }
            // weights, to shared memory as the product wants them: eight rows of a key side by side
            if (it >= 2) barrier_wait(sh.done + b, ((it - 2) >> 1) & 1, lost);
            unsigned char *const to = w_room + b * S::weights + tid * 16;
#pragma unroll
            for (int r = 0; r < N; r += 8) {
                float e[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    e[k] = exp2_fast(s[r + k]);
                    sum[r + k] += e[k];
                }
                *reinterpret_cast<uint4 *>(to + r / 8 * 2048) = make_uint4(pack<E>(e[0], e[1]), pack<E>(e[2], e[3]), pack<E>(e[4], e[5]), pack<E>(e[6], e[7]));
            }
            shared_to_async();
            tensor_before();
            barrier_arrive(sh.weighed + b);

            // -- a segment's end: the sums over the keys, and the result or the part written
            if (flags & kLast) {
                const int part_first = h.part_first, part_last = h.part_last, part_slot = h.part_slot;
                barrier_wait(sh.done + b, it >> 1 & 1, lost);
                if (it > 0) barrier_wait(sh.done + (b ^ 1), (it - 1) >> 1 & 1, lost);
                tensor_after();
                float *const all = reinterpret_cast<float *>(w_room);  // (both rooms for weights are free)
#pragma unroll
                for (int r = 0; r < N; ++r) all[r * 128 + tid] = sum[r];
                weights_meet();
                for (int r = warp; r < N; r += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(all + r * 128 + lane * 4);
                    float z = (x.x + x.y) + (x.z + x.w);
#pragma unroll
                    for (int d = 16; d; d /= 2) z += __shfl_xor_sync(~0u, z, d);
                    if (lane == 0) sh.sum[r] = z;
                }
                weights_meet();
                const float vs = P.v_scale ? ld(P.v_scale + head) : 1.0f;
                const i64 part = static_cast<i64>(cta) * 2 + (flags & kSlot ? 1 : 0);
                const float poison = *reinterpret_cast<volatile int *>(lost) ? __int_as_float(0x7fffffff) : 1.0f;
#pragma unroll 1
                for (int c = 0; c < S::blocks * N; c += 16) {
                    float o[16];
                    tensor_load16(o, tensor + lanes + 2 * N + c);
                    tensor_loaded();
                    const int e = (c < N ? 0 : 128) + tid, r0 = c % N;
                    int j = (from + r0) / P.group, g = from + r0 - j * P.group;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int r = r0 + k;
                        if (r < count && (D >= 128 || e < D)) {
                            const float z = sh.sum[r];
                            const bool none = sh.top[r] == -kInf;
                            if (flags & kPartial) {
                                st(P.sums + (part * S::rows + r) * D + e, none ? 0.0f : o[k] * poison);
                            } else {
                                const float y = none ? 0.0f : o[k] * poison * (vs / z);
                                st(reinterpret_cast<E *>(P.out + static_cast<i64>(first_row + j) * P.out_row + static_cast<i64>(head * P.group + g) * P.out_head) + e, static_cast<E>(y));
                            }
                        }
                        if (++g == P.group) g = 0, ++j;
                    }
                }
                if (tid < count) {
                    const float top = sh.top[tid], z = top == -kInf ? 0.0f : sh.sum[tid];
                    const int at_row = from + tid, j = at_row / P.group;
                    if (flags & kPartial)
                        st(P.stats + part * S::rows + tid, make_float2(top, z));
                    else if (P.lse)
                        st(P.lse + static_cast<i64>(first_row + j) * P.hq + head * P.group + at_row - j * P.group, z == 0 ? -kInf : (top - W::offset + log2f(z)) * kLn2);
                }
                if (tid == 0 && P.parts && it == n - 1) {
                    const bool open = flags & kOpen;
                    st(reinterpret_cast<int4 *>(P.parts + cta), make_int4(open ? part_first : -1, part_last, part_slot, first_row));
                    st(reinterpret_cast<int4 *>(P.parts + cta) + 1, make_int4(from, count, head, 0));
                }
                tensor_before();
                weights_meet();  // (the sums' room takes weights again)
            }
        }
    }
    tensor_before();
    __syncthreads();
    if (warp == 4) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tensor), "n"(S::columns) : "memory");
}

}  // namespace sv_cache
