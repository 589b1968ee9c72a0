// Attention of a step's rows over the paged cache. See sv_cache_attention.cu for the mathematics.
#pragma once

#include <type_traits>

#include "sv_cache.cuh"

namespace sv_cache {

constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kLn2 = 0x1.62e430p-1f;
constexpr int kSlices = 4;             // warps that share a tile's tokens
constexpr int kMaxPlace = 1 << 30;     // places of a request

// A part of a group that ends at a CTA's last tile, to be joined with those of the CTAs behind: the CTAs that
// hold parts of the group, the first one's slot, and the group's rows. first < 0: none.
struct Part {
    int first, last, slot, row0, from, count, head, unused;
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
    float *sums;          // workspace: [ctas][2][rows of a tile][dim], then [ctas][2][rows of a tile][2], then Part [ctas]
    float2 *stats;
    Part *parts;
};

// What a kernel's tile is. ES bytes of a cached element, D elements of a head, RG groups of warps, each with MT
// tiles of 16 rows.
template <int ES, int D, int RG, int MT>
struct Tile {
    static constexpr int row = D * ES;                              // bytes of a key
    static constexpr int chunks = row / 16;
    static constexpr int tokens = row <= 128 ? 128 : 64;
    static constexpr int sub = tokens / (16 * kSlices);             // groups of 16 tokens a warp
    static constexpr int rows = 16 * RG * MT;
    static constexpr int threads = 32 * kSlices * RG;
    static constexpr int kv = tokens * row;
    static constexpr int stage = 2 * kv + rows * D * 2;
    static constexpr int resident = RG == 1 && stage <= 37000 ? 2 : 1;  // CTAs on an SM
    static constexpr bool q_held = MT == 1;                         // the queries' fragments stay in registers,
    static constexpr int q_bytes = q_held ? 0 : rows * D * 2;       // or the queries in shared memory
    static constexpr int fit = ((tokens == 128 ? 220000 : 226000) - q_bytes) / stage;
    static constexpr int stages = resident == 2 ? (stage > 30000 ? 3 : 5) : fit > 6 ? 6 : fit;
    static constexpr int buffers = 2 * rows * D * 4 <= 2 * kv ? 2 : 1;
    static_assert(stages >= 2 && rows * D * 4 <= 2 * kv, "room");
    // shared memory behind the stages
    struct Head {
        int p0, first, count, from, row0, head, length, flags;      // see describe()
        int part_first, part_last, part_slot, unused;
        uint32_t seen[tokens / 32];
    };
    struct Shared {
        int2 place[stages + 1][tokens];  // page, slot
        Head head[stages + 1];
        float2 stat[kSlices][rows];
        float2 joined[rows];
        i64 scan[threads / 32 + 1];
        i64 start[2];
    };
    static constexpr int bytes = stages * stage + q_bytes + static_cast<int>(sizeof(Shared));
    static_assert(bytes <= (resident == 2 ? 115712 : 232448), "shared memory");
};

enum : int { kFirst = 1, kLast = 2, kPartial = 4, kSlot = 8, kOpen = 16 };

__device__ __forceinline__ uint32_t shared_address(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void copy16(uint32_t to, const unsigned char *from, bool there)
{
    there = there && SV_CACHE_INSIDE(from, 16, false);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void matrices(uint32_t *r, uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void matrices_turned(uint32_t *r, uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void multiply(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The tiles of a group (rows `from` to from + count - 1 of request i with one key head): [t0, t1), at least one; keys
// at places [start, end) are seen by one of its rows.
struct Range {
    int t0, t1, start, end;
};
__device__ __forceinline__ Range range_of(const AttentionParams &P, int tokens, int length, int j0, int j1)
{
    const i64 cap = static_cast<i64>(P.s.width) * P.s.page;
    i64 end = length < 0 ? 0 : min(static_cast<i64>(length) + j1 + 1, cap);
    i64 start = P.window > 0 && length >= 0 ? max(0ll, static_cast<i64>(length) + j0 + 1 - P.window) : 0;
    if (start >= end) start = end = 0;
    Range r;
    r.start = static_cast<int>(start);
    r.end = static_cast<int>(end);
    r.t0 = r.start / tokens;
    r.t1 = max(r.t0 + 1, (r.end + tokens - 1) / tokens);
    return r;
}

// All tiles of the step in order: request, rows of a tile, key head, tokens. CTA c takes those from c W / ctas
// to (c + 1) W / ctas, so every CTA gets as many whatever the lengths are.
template <typename Shape>
struct Walk {
    const AttentionParams &P;
    int i, first, rows, length;  // the request: its first row, its rows times the group, its length
    int from, count, head, t;    // the group: its first row within the request, its rows; the tile
    Range range;
    i64 base;                    // number of the group's first tile

    __device__ Walk(const AttentionParams &P) : P(P) {}
    __device__ void request(int k)
    {
        i = k;
        rows = i < P.s.n ? request_rows(P.s, i, first) * P.group : 0;
        length = rows ? ld(P.s.lengths + i) : 0;
    }
    __device__ void group(int at)
    {
        from = at;
        count = min(Shape::rows, rows - at);
        range = range_of(P, Shape::tokens, length, at / P.group, (at + count - 1) / P.group);
        t = range.t0;
    }
    __device__ int tiles() const { return range.t1 - range.t0; }
    __device__ i64 request_tiles(int k)
    {
        request(k);
        i64 sum = 0;
        for (int at = 0; at < rows; at += Shape::rows) {
            group(at);
            sum += static_cast<i64>(tiles()) * P.hk;
        }
        return sum;
    }
    // To tile `skip` of request k.
    __device__ void seek(int k, i64 skip, i64 number)
    {
        request(k);
        base = number - skip;
        for (int at = 0; at < rows; at += Shape::rows) {
            group(at);
            const i64 here = static_cast<i64>(tiles()) * P.hk;
            if (skip < here) break;
            skip -= here;
            base += here;
        }
        head = static_cast<int>(skip / tiles());
        t += static_cast<int>(skip - static_cast<i64>(head) * tiles());
        base += static_cast<i64>(head) * tiles();
    }
    __device__ void next()
    {
        if (++t < range.t1) return;
        base += tiles();
        t = range.t0;
        if (++head < P.hk) return;
        head = 0;
        if (from + Shape::rows < rows) return group(from + Shape::rows);
        do
            request(i + 1);
        while (rows == 0 && i < P.s.n);
        if (rows) group(0);
    }
};

// Address of a 16-byte chunk of a key in a stage: chunks of eight keys in a row fall into different banks.
template <int CHUNKS>
__device__ __forceinline__ uint32_t swizzled(int token, int chunk)
{
    return CHUNKS >= 8 ? token * (CHUNKS * 16) + ((chunk ^ (token & 7)) << 4) : token * (CHUNKS * 16) + ((chunk ^ (token >> 1 & 3)) << 4);
}

// The fragments of a 16 x 16 piece of the queries. For 16-bit caches as the product wants them; for e4m3, whose
// bytes come four neighbours to a lane, with the elements of a piece in that order (4 t to 4 t + 3 in lane t of
// four), and bf16 queries as binary16 times their row's factor.
template <int ES, int D>
__device__ __forceinline__ void query_fragment(uint32_t *a, uint32_t q_at, int row0, int ks, int lane, bool convert, const float *factor)
{
    if constexpr (ES == 2) {
        const int r = row0 + (lane & 15), c = ks * 2 + (lane >> 4);
        matrices(a, q_at + swizzled<D / 8>(r, c));
    } else {
        const int t = lane & 3;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = row0 + lane / 4 + half * 8, e = ks * 16 + 4 * t;
            uint32_t lo, hi;
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(lo), "=r"(hi) : "r"(q_at + swizzled<D / 8>(r, e / 8) + (e & 7) * 2) : "memory");
            if (convert) {
                const float2 x = pair_of<__nv_bfloat16>(lo), y = pair_of<__nv_bfloat16>(hi);
                lo = pack<__half>(x.x * factor[half], x.y * factor[half]);
                hi = pack<__half>(y.x * factor[half], y.y * factor[half]);
            }
            a[half] = lo;
            a[2 + half] = hi;
        }
    }
}

template <bool BF16, int ES, int D, int RG, int MT>
__global__ void __launch_bounds__(Tile<ES, D, RG, MT>::threads, Tile<ES, D, RG, MT>::resident) sv_cache_attention_kernel(const AttentionParams P)
{
    using S = Tile<ES, D, RG, MT>;
    // Weights are rounded to the products' type relative to 1 (bf16) or 2^15 (binary16, whose smallest step
    // is then 2^-39 of the largest weight: without it 60000 weights of 2^-26 would be lost).
    constexpr float kOffset = BF16 ? 0.0f : 15.0f;
    extern __shared__ __align__(1024) unsigned char room[];
    auto &sh = *reinterpret_cast<typename S::Shared *>(room + S::stages * S::stage + S::q_bytes);
    const uint32_t stages_at = shared_address(room);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31, g = lane / 4, t4 = lane & 3;
    const int slice = warp % kSlices, rg = warp / kSlices;
    const int cta = blockIdx.x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // -- this CTA's tiles
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
    __syncthreads();
    walk.seek(static_cast<int>(sh.start[0]), sh.start[1], u0);

    // -- a tile's description: what is in it, and where its keys are
    int page = -1, slot = 0;
    auto look_up = [&](int) {  // this thread's key (its page arrives while a tile is computed)
        const int p = walk.t * S::tokens + tid;
        page = -1;
        if (walk.rows && tid < S::tokens && p >= walk.range.start && p < walk.range.end) {
            const int c = p < (1 << 22) ? static_cast<int>((static_cast<u64>(p) * P.s.page_magic) >> 42) : p / P.s.page;
            slot = p - c * P.s.page;
            page = ld(P.s.table + walk.i * P.s.table_stride + c);
        }
    };
    auto describe = [&](int d) {
        const int k = d % (S::stages + 1);
        if (tid < S::tokens) {
            const bool seen = page >= 0 && page < P.s.pages;
            sh.place[k][tid] = make_int2(seen ? page : -1, slot);
            const uint32_t all = __ballot_sync(~0u, seen);
            if (lane == 0) sh.head[k].seen[warp] = all;
        }
        if (tid == 0) {
            auto &h = sh.head[k];
            const bool opens = walk.t == walk.range.t0, ends = walk.t + 1 == walk.range.t1;
            // (a segment: the tiles of one group that this CTA has)
            const bool first = d == 0 || opens, last = d == n - 1 || ends;
            const bool part = walk.base < u0 || walk.base + walk.tiles() > u1;
            h.p0 = walk.t * S::tokens;
            h.first = walk.first;
            h.count = walk.count;
            h.from = walk.from;
            h.head = walk.head;
            h.length = walk.length;
            h.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (part ? kPartial : 0) | (walk.base > u0 ? kSlot : 0) | (last && !ends ? kOpen : 0);
            if (last && !ends) {  // the CTAs that have tiles of the group
                h.part_first = static_cast<int>(((walk.base + 1) * ctas - 1) / total);
                h.part_last = static_cast<int>(((walk.base + walk.tiles()) * ctas - 1) / total);
                h.part_slot = total * h.part_first / ctas < walk.base;
            }
        }
        walk.next();
    };
    auto issue = [&](int d) {
        const int k = d % (S::stages + 1);
        const uint32_t at = stages_at + (d % S::stages) * S::stage;
        const auto &h = sh.head[k];
        const i64 head = h.head;
        const unsigned char *keys = P.kc.at + head * P.kc.head, *values = P.vc.at + head * P.vc.head;
#pragma unroll 4
        for (int x = tid; x < S::tokens * S::chunks; x += S::threads) {
            const int token = x / S::chunks, c = x % S::chunks;
            const int2 w = sh.place[k][token];
            const bool there = w.x >= 0;
            const i64 pg = there ? w.x : 0, sl = there ? w.y : 0;
            const uint32_t to = at + swizzled<S::chunks>(token, c);
            copy16(to, keys + pg * P.kc.page + sl * P.kc.slot + c * 16, there);
            copy16(to + S::kv, values + pg * P.vc.page + sl * P.vc.slot + c * 16, there);
        }
        if (h.flags & kFirst)
            for (int x = tid; x < S::rows * (D / 8); x += S::threads) {
                const int r = x / (D / 8), c = x % (D / 8);
                const bool there = r < h.count;
                const int at_row = h.from + (there ? r : 0), j = at_row / P.group, qh = static_cast<int>(head) * P.group + at_row - j * P.group;
                copy16(at + 2 * S::kv + swizzled<D / 8>(r, c), P.q + (h.first + j) * P.q_row + qh * P.q_head + c * 16, there);
            }
    };

    for (int d = 0; d < S::stages && d < n; ++d) {
        look_up(d);
        describe(d);
    }
    __syncthreads();
    for (int d = 0; d < S::stages - 1; ++d) {
        if (d < n) issue(d);
        copies_close();
    }

    // -- the tiles
    uint32_t q[S::q_held ? D / 16 : 1][4];
    float o[MT][D / 8][4], top[MT][2], sum[MT][2], scale[MT][2], factor[MT][2];
    int hi[MT][2], lo[MT][2];
    bool part_written = false;
    for (int it = 0; it < n; ++it) {
        copies_wait<S::stages - 2>();
        __syncthreads();
        if (it + S::stages - 1 < n) issue(it + S::stages - 1);
        copies_close();
        const bool more = it + S::stages < n;
        if (more) look_up(it + S::stages);

        const auto &h = sh.head[it % (S::stages + 1)];
        const uint32_t at = stages_at + (it % S::stages) * S::stage, q_at = S::q_held ? at + 2 * S::kv : stages_at + S::stages * S::stage;
        const int flags = h.flags, p0 = h.p0, row_base = rg * MT * 16;
        if (flags & kFirst) {
            if constexpr (!S::q_held) {  // (the stage will hold other keys before the segment ends)
                const uint4 *from = reinterpret_cast<const uint4 *>(room + (it % S::stages) * S::stage + 2 * S::kv);
                for (int x = tid; x < S::q_bytes / 16; x += S::threads) reinterpret_cast<uint4 *>(room + S::stages * S::stage)[x] = from[x];
                __syncthreads();
            }
            const float ks = P.scale * (P.k_scale ? ld(P.k_scale + h.head) : 1.0f);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int e = 0; e < D / 8; ++e) o[m][e][0] = o[m][e][1] = o[m][e][2] = o[m][e][3] = 0;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int r = row_base + m * 16 + g + half * 8, j = (h.from + min(r, h.count - 1)) / P.group;
                    const i64 x = h.length < 0 ? -1 : static_cast<i64>(h.length) + j;
                    hi[m][half] = static_cast<int>(min(x, static_cast<i64>(kMaxPlace)));
                    lo[m][half] = P.window > 0 ? static_cast<int>(max(-1ll, min(x - P.window, static_cast<i64>(kMaxPlace)))) : -1;
                    top[m][half] = -kInf;
                    sum[m][half] = 0;
                    factor[m][half] = 1.0f;
                    scale[m][half] = ks;
                    if constexpr (ES == 1) {
                        if (P.bf16) {
                            // bf16 queries as binary16 times a power of two that takes the row's largest to [2^13, 2^14):
                            // exact down to 2^-28 of it
                            float most = 0;
#pragma unroll 4
                            for (int e = t4 * 4; e < D; e += 16) {
                                uint32_t x0, x1;
                                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x0), "=r"(x1) : "r"(q_at + swizzled<D / 8>(r, e / 8) + (e & 7) * 2) : "memory");
                                const float2 a = pair_of<__nv_bfloat16>(x0), b = pair_of<__nv_bfloat16>(x1);
                                most = fmaxf(fmaxf(most, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
                            }
                            most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
                            most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
                            const int up = min(110, 13 - (static_cast<int>(__float_as_uint(most) >> 23) - 127));
                            factor[m][half] = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                            scale[m][half] = ks * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
                        }
                    }
                }
                if constexpr (S::q_held) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) query_fragment<ES, D>(q[k], q_at, row_base + m * 16, k, lane, P.bf16, factor[m]);
                }
            }
        }

        // the tile's keys that this warp has
        const int token0 = slice * 16 * S::sub;
        uint32_t seen = h.seen[token0 / 32];
        if constexpr (S::sub == 1) seen = seen >> (token0 & 31) & 0xffffu;
        constexpr uint32_t kAll = S::sub == 1 ? 0xffffu : ~0u;
        if (seen) {
            float s[MT][S::sub][2][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int b = 0; b < S::sub; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[m][b][0][e] = s[m][b][1][e] = 0;
            if constexpr (ES == 2) {
                const int token = token0 + (lane >> 4) * 8 + (lane & 7), c = lane >> 3 & 1;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t b[S::sub][4];
#pragma unroll
                    for (int x = 0; x < S::sub; ++x) matrices(b[x], at + swizzled<S::chunks>(token + x * 16, k * 2 + c));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        uint32_t a[4];
                        if constexpr (!S::q_held) query_fragment<ES, D>(a, q_at, row_base + m * 16, k, lane, false, factor[m]);
                        const uint32_t *f = S::q_held ? q[S::q_held ? k : 0] : a;
#pragma unroll
                        for (int x = 0; x < S::sub; ++x) {
                            multiply<BF16>(s[m][x][0], f, b[x][0], b[x][1]);
                            multiply<BF16>(s[m][x][1], f, b[x][2], b[x][3]);
                        }
                    }
                }
            } else {
                const int token = token0 + (lane >> 3 & 1) * 8 + (lane & 7), c = lane >> 4;
#pragma unroll
                for (int k = 0; k < D / 16; k += 2) {
                    uint32_t b[S::sub][4];
#pragma unroll
                    for (int x = 0; x < S::sub; ++x) matrices(b[x], at + swizzled<S::chunks>(token + x * 16, k + c));
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        uint32_t w[S::sub][4];
#pragma unroll
                        for (int x = 0; x < S::sub; ++x) {
                            w[x][0] = half2_of_e4m3(b[x][2 * kk]);
                            w[x][1] = half2_of_e4m3(b[x][2 * kk] >> 16);
                            w[x][2] = half2_of_e4m3(b[x][2 * kk + 1]);
                            w[x][3] = half2_of_e4m3(b[x][2 * kk + 1] >> 16);
                        }
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            uint32_t a[4];
                            if constexpr (!S::q_held) query_fragment<ES, D>(a, q_at, row_base + m * 16, k + kk, lane, P.bf16, factor[m]);
                            const uint32_t *f = S::q_held ? q[S::q_held ? k + kk : 0] : a;
#pragma unroll
                            for (int x = 0; x < S::sub; ++x) {
                                multiply<BF16>(s[m][x][0], f, w[x][0], w[x][1]);
                                multiply<BF16>(s[m][x][1], f, w[x][2], w[x][3]);
                            }
                        }
                    }
                }
            }

            // which keys a row does not see: looked at in the tiles where some row may not see all
            const int first_key = p0 + token0, last_key = first_key + 16 * S::sub - 1;
            bool edge = seen != kAll;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int half = 0; half < 2; ++half) edge |= last_key > hi[m][half] || first_key <= lo[m][half];
            edge = __any_sync(~0u, edge);
            uint32_t w[MT][S::sub][4];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float up[2] = {top[m][0], top[m][1]};
#pragma unroll
                for (int x = 0; x < S::sub; ++x)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float v = s[m][x][b][e] * scale[m][e / 2];
                            if (edge) {
                                const int key = x * 16 + b * 8 + t4 * 2 + (e & 1), place = first_key + key;
                                if (!(seen >> key & 1) || place > hi[m][e / 2] || place <= lo[m][e / 2]) v = -kInf;
                            }
                            s[m][x][b][e] = v;
                            up[e / 2] = fmaxf(up[e / 2], v);
                        }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    up[half] = fmaxf(up[half], __shfl_xor_sync(~0u, up[half], 1));
                    up[half] = fmaxf(up[half], __shfl_xor_sync(~0u, up[half], 2));
                }
                if (__any_sync(~0u, up[0] > top[m][0] || up[1] > top[m][1])) {
                    float keep[2];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        keep[half] = up[half] == top[m][half] ? 1.0f : exp2_fast(top[m][half] - up[half]);
                        sum[m][half] *= keep[half];
                        top[m][half] = up[half];
                    }
#pragma unroll
                    for (int e = 0; e < D / 8; ++e)
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[m][e][c] *= keep[c / 2];
                }
                const float from[2] = {(up[0] == -kInf ? 0.0f : up[0]) - kOffset, (up[1] == -kInf ? 0.0f : up[1]) - kOffset};
#pragma unroll
                for (int x = 0; x < S::sub; ++x)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const float e0 = exp2_fast(s[m][x][b][2 * half] - from[half]), e1 = exp2_fast(s[m][x][b][2 * half + 1] - from[half]);
                            sum[m][half] += e0 + e1;
                            w[m][x][b * 2 + half] = BF16 ? pack<__nv_bfloat16>(e0, e1) : pack<__half>(e0, e1);
                        }
            }

            // weights times values
            const uint32_t v_at = at + S::kv;
            auto both = [&](int x, int n8, const uint32_t *b) {  // two pieces of eight elements
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (edge) {
                        // A weight of 0 times a value that is not finite is NaN in a product: such pieces, if any, by hand.
                        bool odd = false;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t mask = BF16 ? 0x7f80u : 0x7c00u;
                            odd |= (b[c] & mask) == mask || (b[c] >> 16 & mask) == mask;
                        }
                        if (__any_sync(~0u, odd)) {
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk)
#pragma unroll 1
                                for (int key = 0; key < 8; ++key) {
                                    // weights of the rows g and g + 8: in lane key / 2 of the four; values of the
                                    // elements 2 t4 and 2 t4 + 1: in the lanes 8 t4 + key / 2 and 4 behind
                                    const int in = key / 2, high = key & 1;
                                    using E = std::conditional_t<BF16, __nv_bfloat16, __half>;
                                    auto part = [&](uint32_t v, int from) {
                                        const float2 f = pair_of<E>(__shfl_sync(~0u, v, from));
                                        return high ? f.y : f.x;
                                    };
                                    const float w0 = part(w[m][x][kk * 2], (lane & ~3) | in), w1 = part(w[m][x][kk * 2 + 1], (lane & ~3) | in);
#pragma unroll
                                    for (int piece = 0; piece < 2; ++piece) {
                                        const float b0 = part(b[piece * 2 + kk], t4 * 8 + in), b1 = part(b[piece * 2 + kk], t4 * 8 + 4 + in);
                                        float *c = o[m][n8 + piece];
                                        if (w0 != 0) c[0] = fmaf(w0, b0, c[0]), c[1] = fmaf(w0, b1, c[1]);
                                        if (w1 != 0) c[2] = fmaf(w1, b0, c[2]), c[3] = fmaf(w1, b1, c[3]);
                                    }
                                }
                            continue;
                        }
                    }
                    multiply<BF16>(o[m][n8], w[m][x], b[0], b[1]);
                    multiply<BF16>(o[m][n8 + 1], w[m][x], b[2], b[3]);
                }
            };
            const int token = token0 + (lane >> 3 & 1) * 8 + (lane & 7);
#pragma unroll
            for (int x = 0; x < S::sub; ++x) {
                if constexpr (ES == 2) {
#pragma unroll
                    for (int e = 0; e < D / 16; ++e) {
                        uint32_t b[4];
                        matrices_turned(b, v_at + swizzled<S::chunks>(token + x * 16, e * 2 + (lane >> 4)));
                        both(x, 2 * e, b);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < D / 16; e += 2) {
                        uint32_t r[4];
                        matrices_turned(r, v_at + swizzled<S::chunks>(token + x * 16, e + (lane >> 4)));
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            // two keys, two neighbouring elements in each register: first both keys of the even element
                            const uint32_t a0 = __byte_perm(r[2 * c], 0, 0x3120), a1 = __byte_perm(r[2 * c + 1], 0, 0x3120);
                            const uint32_t b[4] = {half2_of_e4m3(a0), half2_of_e4m3(a1), half2_of_e4m3(a0 >> 16), half2_of_e4m3(a1 >> 16)};
                            both(x, 2 * (e + c), b);
                        }
                    }
                }
            }
        }

        // -- a segment's end: the slices joined, and the result or the part written
        if (flags & kLast) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    sum[m][half] += __shfl_xor_sync(~0u, sum[m][half], 1);
                    sum[m][half] += __shfl_xor_sync(~0u, sum[m][half], 2);
                    if (t4 == 0) sh.stat[slice][row_base + m * 16 + g + half * 8] = make_float2(top[m][half], sum[m][half]);
                }
            __syncthreads();  // (and every warp is through with the stage)
            float *buffer = reinterpret_cast<float *>(room + (it % S::stages) * S::stage);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int r = row_base + m * 16 + g + half * 8;
                    float most = -kInf, z = 0;
#pragma unroll
                    for (int w = 0; w < kSlices; ++w) most = fmaxf(most, sh.stat[w][r].x);
                    const float from = most == -kInf ? 0.0f : most;
#pragma unroll
                    for (int w = 0; w < kSlices; ++w) {
                        const float2 x = sh.stat[w][r];
                        z += x.y * (x.x == most ? 1.0f : exp2_fast(x.x - from));
                    }
                    const float keep = top[m][half] == most ? 1.0f : exp2_fast(top[m][half] - from);
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) o[m][e][2 * half] *= keep, o[m][e][2 * half + 1] *= keep;
                    if (slice == 0 && t4 == 0) sh.joined[r] = make_float2(most, z);
                }
            constexpr int kTurns = kSlices / S::buffers;
#pragma unroll
            for (int turn = 0; turn < kTurns; ++turn) {
                if (slice / S::buffers == turn) {
                    float *to = buffer + slice % S::buffers * S::rows * D;
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int r = row_base + m * 16 + g + half * 8;
#pragma unroll
                            for (int e = 0; e < D / 8; ++e) {
                                // (for e4m3 two pieces are the even and the odd elements of 16)
                                const int c0 = ES == 2 ? e * 8 + 2 * t4 : e / 2 * 16 + 4 * t4 + e % 2;
                                float *x = to + r * D + (c0 ^ (r & 7) << 3), *y = x + (ES == 2 ? 1 : 2);
                                *x = o[m][e][2 * half] + (turn ? *x : 0.0f);
                                *y = o[m][e][2 * half + 1] + (turn ? *y : 0.0f);
                            }
                        }
                }
                __syncthreads();
            }
            const float vs = P.v_scale ? ld(P.v_scale + h.head) : 1.0f;
            const i64 part = static_cast<i64>(cta) * 2 + (flags & kSlot ? 1 : 0);
            for (int x = tid; x < h.count * (D / 4); x += S::threads) {
                const int r = x / (D / 4), c = x % (D / 4) * 4, at_row = h.from + r, j = at_row / P.group;
                float4 v = *reinterpret_cast<const float4 *>(buffer + r * D + (c ^ (r & 7) << 3));
                if constexpr (S::buffers == 2) {
                    const float4 u = *reinterpret_cast<const float4 *>(buffer + (S::rows + r) * D + (c ^ (r & 7) << 3));
                    v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                }
                const float2 stat = sh.joined[r];
                if (flags & kPartial) {
                    st(reinterpret_cast<float4 *>(P.sums + (part * S::rows + r) * D + c), v);
                    if (c == 0) st(P.stats + part * S::rows + r, stat);
                } else {
                    const int qh = h.head * P.group + at_row - j * P.group;
                    const float f = stat.y == 0 ? 0.0f : vs / stat.y;
                    const float4 y = stat.y == 0 ? make_float4(0, 0, 0, 0) : make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
                    const bool bf16 = BF16 || P.bf16;
                    const uint2 w = bf16 ? make_uint2(pack<__nv_bfloat16>(y.x, y.y), pack<__nv_bfloat16>(y.z, y.w)) : make_uint2(pack<__half>(y.x, y.y), pack<__half>(y.z, y.w));
                    st(reinterpret_cast<uint2 *>(P.out + (h.first + j) * P.out_row + qh * P.out_head + c * 2), w);
                    if (c == 0 && P.lse) st(P.lse + static_cast<i64>(h.first + j) * P.hq + qh, stat.y == 0 ? -kInf : (stat.x - kOffset + log2f(stat.y)) * kLn2);
                }
            }
            if (flags & kOpen && tid == 0) {
                const Part x{h.part_first, h.part_last, h.part_slot, h.first, h.from, h.count, h.head, 0};
                st(reinterpret_cast<int4 *>(P.parts + cta), make_int4(x.first, x.last, x.slot, x.row0));
                st(reinterpret_cast<int4 *>(P.parts + cta) + 1, make_int4(x.from, x.count, x.head, 0));
            }
            part_written = flags & kOpen;
        }
        if (more) describe(it + S::stages);
    }
    if (!part_written && P.parts && tid == 0) st(&P.parts[cta].first, -1);
}

// Joins the parts of the groups that more than one CTA has. A group over k + 1 CTAs has k CTAs here, which share its
// outputs; a few lanes take the parts of four elements.
template <int D>
__global__ void __launch_bounds__(256) sv_cache_join_kernel(const AttentionParams P, int rows, float offset)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 a = ld_own(reinterpret_cast<const int4 *>(P.parts + blockIdx.x));
    const int first = a.x, last = a.y, row0 = a.w;
    if (first < 0) return;
    const int4 b = ld_own(reinterpret_cast<const int4 *>(P.parts + blockIdx.x) + 1);
    const int from = b.x, count = b.y, head = b.z;
    const int share = last - first, mine = static_cast<int>(blockIdx.x) - first, items = count * (D / 4);
    const int lo = static_cast<int>(static_cast<i64>(items) * mine / share), hi = static_cast<int>(static_cast<i64>(items) * (mine + 1) / share);
    int lanes = 1;
    while (lanes < 32 && lanes * 4 < share + 1) lanes *= 2;
    const int each = 256 / lanes, lane = threadIdx.x % lanes;
    const float vs = P.v_scale ? ld(P.v_scale + head) : 1.0f;
    for (int base = lo; base < hi; base += each) {
        const int item = base + threadIdx.x / lanes;
        const bool there = item < hi;
        const int r = there ? item / (D / 4) : 0, c = there ? item % (D / 4) * 4 : 0;
        auto part = [&](int k) { return (static_cast<i64>(first + k) * 2 + (k == 0 ? a.z : 0)) * rows + r; };
        float most = -kInf, z = 0;
        float4 y = make_float4(0, 0, 0, 0);
        for (int k = lane; k <= share; k += lanes) {
            const float2 s = ld_own(P.stats + part(k));
            const float4 v = ld_own(reinterpret_cast<const float4 *>(P.sums + part(k) * D + c));
            const float up = fmaxf(most, s.x), at = up == -kInf ? 0.0f : up;
            const float f = exp2_fast(most - at), g = s.x == up ? 1.0f : exp2_fast(s.x - at);
            z = z * f + s.y * g;
            y = make_float4(y.x * f + v.x * g, y.y * f + v.y * g, y.z * f + v.z * g, y.w * f + v.w * g);
            most = up;
        }
        for (int d = lanes / 2; d; d /= 2) {
            const float up = fmaxf(most, __shfl_xor_sync(~0u, most, d)), at = up == -kInf ? 0.0f : up, f = exp2_fast(most - at);
            auto add = [&](float &v) {
                v *= f;
                v += __shfl_xor_sync(~0u, v, d);
            };
            add(z), add(y.x), add(y.y), add(y.z), add(y.w);
            most = up;
        }
        if (!there || lane != 0) continue;
        const int at_row = from + r, j = at_row / P.group, qh = head * P.group + at_row - j * P.group;
        const float f = z == 0 ? 0.0f : vs / z;
        if (z == 0) y = make_float4(0, 0, 0, 0);
        const uint2 w = P.bf16 ? make_uint2(pack<__nv_bfloat16>(y.x * f, y.y * f), pack<__nv_bfloat16>(y.z * f, y.w * f))
                               : make_uint2(pack<__half>(y.x * f, y.y * f), pack<__half>(y.z * f, y.w * f));
        st(reinterpret_cast<uint2 *>(P.out + (row0 + j) * P.out_row + qh * P.out_head + c * 2), w);
        if (c == 0 && P.lse) st(P.lse + static_cast<i64>(row0 + j) * P.hq + qh, z == 0 ? -kInf : (most - offset + log2f(z)) * kLn2);
    }
}

}  // namespace sv_cache
