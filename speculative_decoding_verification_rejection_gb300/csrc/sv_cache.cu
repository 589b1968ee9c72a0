// Cache operators (spec_verify_cache_append, spec_verify_cache_attention of include/spec_verify.h): the rows
// of a step are appended to the paged cache of keys and values, turned by their positions, and attend
// over it.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "sv_cache.cuh"
#include "sv_cache_attention.cuh"

namespace {

using namespace sv_cache;

// ---------------------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------------------
// Every element is read once and written once; what is computed is a sine and cosine a pair and row (not
// a head: a warp turns all heads that it has of a row by one table in shared memory) and six operations a
// pair and head, so memory bounds it. A warp has a row, or a part of one where there are few rows, and asks for
// its first elements before it looks for the row's request, page and position: warps do not wait for one another.
//
// The angle in turns, modulo one: pos * frac(inv_freq / 2 pi) with the fraction in steps of 2^-64, one
// 64-bit product whose upper bits wrap away exactly the whole turns; what is left, 32 bits of a turn, is rounded to binary32 (by up to
// pi 2^-25) for sine and cosine. A binary32 angle of position 10^6 would be off by 0.03 radians.
struct AppendParams {
    Step s;
    const unsigned char *q, *k, *v;
    unsigned char *q_out;
    i64 q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head;  // bytes
    Cache kc, vc;
    const float *inv_freq, *k_scale, *v_scale;
    const int32_t *positions;
    i64 positions_stride;
    int hq, hk, dim, half, interleaved;
    int parts, items;  // parts of a row, 16-element items of a part
    Divider by_parts, by_items_a_head;
    uint32_t axes[SV_MAX_HEAD_DIM / 2 / 16];  // two bits a pair
};

constexpr int kAppendThreads = 256;
// Blocks of a call at most, twice what the device holds: those that start later ask for their rows while others write
// (16001 rows 55 us, with half of them 62).
constexpr int kAppendBlocks = 152 * 8;

// The 16 elements that a thread turns: two runs of 8 where the pairs are half a rotary dimension apart, else one run.
struct Item {
    int first, second;  // element of the first 8 and of the second 8
    int pair;           // the first one's pair, -1: not turned
};
__device__ __forceinline__ Item item_of(int c, int half, int interleaved)
{
    const int e = c * 16;
    if (e >= 2 * half) return Item{e, e + 8, -1};
    return interleaved ? Item{e, e + 8, c * 8} : Item{c * 8, half + c * 8, c * 8};
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &w, float *x)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 p = pair_of<T>(u[k]);
        x[2 * k] = p.x;
        x[2 * k + 1] = p.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float *x)
{
    return make_uint4(pack<T>(x[0], x[1]), pack<T>(x[2], x[3]), pack<T>(x[4], x[5]), pack<T>(x[6], x[7]));
}
// A head's scale as a divisor that many values have: the reciprocal in two numbers, known to 2^-47, whose products with a value give the
// binary32 quotient (Brisebarre, Muller and Raina, "Accelerating correctly rounded floating-point division when the divisor is known in advance",
// 2004). A product with one number takes quotients that are ties of two steps of 8 bits to the wrong one; divisions cost 36.6 us where this costs
// 35.2 and one product 34.2 (4 x 2048 rows of 28 query and 4 key heads of 128).
struct Scale {
    float by, less, scale;
    bool plain, none;  // divide (scales whose reciprocal is not within 2^100 and 2^-100); there is none
    __device__ __forceinline__ explicit Scale(const float *p) : scale(p ? ld(p) : 1.0f), none(!p)
    {
        plain = !(fabsf(scale) > 0x1p-100f && fabsf(scale) < 0x1p100f);
        by = __frcp_rz(scale);  // (so both have one sign, and -0 keeps its own)
        less = fmaf(-scale, by, 1.0f) * by;
    }
    __device__ __forceinline__ float operator()(float x) const
    {
        const float y = x * by;
        return fabsf(y) < 512.0f ? fmaf(x, by, x * less) : y;  // (beyond 448 it does not matter, and an infinity stays one)
    }
};
// 8 values, divided by their head's scale.
__device__ __forceinline__ uint2 pack8_e4m3(float *x, const Scale &scale)
{
    uint32_t h[4];
    if (__builtin_expect(scale.plain, 0)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] /= scale.scale;
    } else if (!scale.none) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = scale(x[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = e4m3_of(x[2 * k], x[2 * k + 1]);
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

constexpr int kAppendAtOnce = 2;  // items of a lane that are on the way at once

// A pair's share of a turn a position, frac(f / 2 pi) in steps of 2^-64. The product with 1 / 2 pi, known to 49 bits as two
// numbers, is one too: its error is below 2^-48 of it. (Binary64 runs at a sixtieth of the binary32 rate here: 256 x 6 rows
// took 30 us with it.)
__device__ __forceinline__ u64 turn_of(float f)
{
    const float hi = f * 0x1.45f306p-3f, lo = fmaf(f, 0x1.45f306p-3f, -hi) + f * 0x1.b9391p-28f;
    return (static_cast<u64>(__float2ll_rn((hi - truncf(hi)) * 0x1p63f)) << 1) + static_cast<u64>(__float2ll_rn(lo * 0x1p64f));
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads, 4) sv_cache_append_kernel(const AppendParams P)
{
    __shared__ float2 tables[kAppendThreads / 32][SV_MAX_HEAD_DIM / 2];
    __shared__ u64 turns[SV_MAX_HEAD_DIM / 2];
    __shared__ bool sound[SV_MAX_HEAD_DIM / 2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, per_head = P.dim / 16, all = (P.hq + 2 * P.hk) * per_head;
    float2 *const table = tables[warp];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int m = threadIdx.x; m < P.half; m += kAppendThreads) {
        const float f = ld(P.inv_freq + m);
        sound[m] = fabsf(f) < 0x1p20f;
        turns[m] = sound[m] ? turn_of(f) : 0;
    }
    __syncthreads();
    struct Where {
        const unsigned char *from;
        Item m;
        int head, kind;  // kind 0: queries, 1: keys, 2: values
    };
    auto where = [&](int r, int at) {
        const int head = P.by_items_a_head(at), c = at - head * per_head;
        Where w;
        w.kind = head < P.hq ? 0 : head < P.hq + P.hk ? 1 : 2;
        w.head = head - (w.kind == 0 ? 0 : w.kind == 1 ? P.hq : P.hq + P.hk);
        w.m = w.kind == 2 ? Item{c * 16, c * 16 + 8, -1} : item_of(c, P.half, P.interleaved);
        w.from = w.kind == 0 ? P.q + r * P.q_row + w.head * P.q_head : w.kind == 1 ? P.k + r * P.k_row + w.head * P.k_head : P.v + r * P.v_row + w.head * P.v_head;
        return w;
    };
    const i64 units = static_cast<i64>(P.s.rows) * P.parts;
#pragma unroll 1
    for (i64 u = static_cast<i64>(blockIdx.x) * (kAppendThreads / 32) + warp; u < units; u += static_cast<i64>(gridDim.x) * (kAppendThreads / 32)) {
        const int r = P.parts == 1 ? static_cast<int>(u) : P.by_parts(static_cast<int>(u)), part = P.parts == 1 ? 0 : static_cast<int>(u) - r * P.parts;
        const int lo = part * P.items, hi = min(lo + P.items, all);
        i64 page = -1;
        int slot = 0;
#pragma unroll 1
        for (int at0 = lo; at0 < hi; at0 += 32 * kAppendAtOnce) {
            uint4 a[kAppendAtOnce], b[kAppendAtOnce];
#pragma unroll
            for (int k = 0; k < kAppendAtOnce; ++k) {
                const int at = at0 + k * 32 + lane;
                if (at < hi) {
                    const Where w = where(r, at);
                    a[k] = ld(reinterpret_cast<const uint4 *>(w.from + w.m.first * 2));
                    b[k] = ld(reinterpret_cast<const uint4 *>(w.from + w.m.second * 2));
                }
            }
            if (at0 == lo) {
                const int i = request_of(P.s, r);
                const int length = i < 0 ? -1 : ld(P.s.lengths + i);
                if (length < 0) break;  // (the warp's lanes agree)
                int first;
                request_rows(P.s, i, first);
                const i64 x = static_cast<i64>(length) + (r - first);
                if (!place(P.s, i, x, page, slot)) page = -1;
                __syncwarp();  // (the table of the row before has been read)
#pragma unroll 1
                for (int m = lane; m < P.half; m += 32) {
                    const int axis = P.axes[m / 16] >> (m % 16 * 2) & 3;
                    const i64 pos = P.positions ? static_cast<i64>(ld(P.positions + axis * P.positions_stride + r)) : x;
                    const int half_turns = static_cast<int>((static_cast<u64>(pos) * turns[m]) >> 32);  // of 2^-31
                    float2 cs;
                    sincospif(static_cast<float>(half_turns) * 0x1p-31f, &cs.y, &cs.x);
                    table[m] = sound[m] ? cs : make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
                }
                __syncwarp();
            }
#pragma unroll
            for (int k = 0; k < kAppendAtOnce; ++k) {
                const int at = at0 + k * 32 + lane;
                if (at >= hi) continue;
                const Where x = where(r, at);
                if (x.kind && page < 0) continue;
                float y[8], w[8];
                unpack8<T>(a[k], y);
                unpack8<T>(b[k], w);
                if (x.m.pair >= 0) {
                    const float2 *t = table + x.m.pair;
                    if (P.interleaved) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 c = t[e], d = t[e + 4];
                            const float y0 = y[2 * e], y1 = y[2 * e + 1], w0 = w[2 * e], w1 = w[2 * e + 1];
                            y[2 * e] = y0 * c.x - y1 * c.y;
                            y[2 * e + 1] = y0 * c.y + y1 * c.x;
                            w[2 * e] = w0 * d.x - w1 * d.y;
                            w[2 * e + 1] = w0 * d.y + w1 * d.x;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 c = t[e];
                            const float y0 = y[e], w0 = w[e];
                            y[e] = y0 * c.x - w0 * c.y;
                            w[e] = y0 * c.y + w0 * c.x;
                        }
                    }
                }
                const Cache &c = x.kind == 2 ? P.vc : P.kc;
                if (E4M3 && x.kind) {
                    unsigned char *const to = c.at + page * c.page + slot * c.slot + x.head * c.head;
                    const float *scales = x.kind == 2 ? P.v_scale : P.k_scale;
                    const Scale scale(scales ? scales + x.head : nullptr);
                    st(reinterpret_cast<uint2 *>(to + x.m.first), pack8_e4m3(y, scale));
                    st(reinterpret_cast<uint2 *>(to + x.m.second), pack8_e4m3(w, scale));
                } else {
                    unsigned char *const to = x.kind ? c.at + page * c.page + slot * c.slot + x.head * c.head : P.q_out + r * P.out_row + x.head * P.out_head;
                    st(reinterpret_cast<uint4 *>(to + x.m.first * 2), pack8<T>(y));
                    st(reinterpret_cast<uint4 *>(to + x.m.second * 2), pack8<T>(w));
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

// Makes `dev` current for the call.
struct DeviceGuard {
    int prev = -1;
    bool ok = true, moved = false;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) {
            ok = false;
            return;
        }
        if (prev != dev) {
            ok = cudaSetDevice(dev) == cudaSuccess;
            moved = ok;
        }
    }
    ~DeviceGuard()
    {
        if (moved) cudaSetDevice(prev);
    }
    DeviceGuard(const DeviceGuard &) = delete;
    DeviceGuard &operator=(const DeviceGuard &) = delete;
};

// One kernel of the attention: what it needs, and how it is launched.
struct Kernel {
    const void *run, *join;
    int rows, threads, bytes, dim;
    float offset;
};

template <int KIND, int D, int N, bool LOADS>
Kernel kernel_of()
{
    using S = Tile<KIND, D, N, LOADS>;
    return Kernel{reinterpret_cast<const void *>(sv_cache_attention_kernel<KIND, D, N, LOADS>), reinterpret_cast<const void *>(sv_cache_join_kernel<D>), N, S::threads,
                  S::bytes, D, Weights<S::bf16>::offset};
}

template <int KIND, int D, bool LOADS>
Kernel kernel_of(int rows)
{
    if constexpr (D == 256)
        return rows == 16 ? kernel_of<KIND, D, 16, LOADS>() : kernel_of<KIND, D, 32, LOADS>();
    else
        return rows == 16   ? kernel_of<KIND, D, 16, LOADS>()
               : rows == 32 ? kernel_of<KIND, D, 32, LOADS>()
               : rows == 48 ? kernel_of<KIND, D, 48, LOADS>()
                            : kernel_of<KIND, D, 64, LOADS>();
}

template <int KIND, bool LOADS>
Kernel kernel_of(int dim, int rows)
{
    return dim == 64 ? kernel_of<KIND, 64, LOADS>(rows) : dim == 128 ? kernel_of<KIND, 128, LOADS>(rows) : kernel_of<KIND, 256, LOADS>(rows);
}

Kernel kernel_of(int cache_dtype, int dim, int rows, bool loads)
{
    if (cache_dtype == SV_E4M3) return loads ? kernel_of<SV_E4M3, true>(dim, rows) : kernel_of<SV_E4M3, false>(dim, rows);
    if (cache_dtype == SV_BF16) return loads ? kernel_of<SV_BF16, true>(dim, rows) : kernel_of<SV_BF16, false>(dim, rows);
    return loads ? kernel_of<SV_F16, true>(dim, rows) : kernel_of<SV_F16, false>(dim, rows);
}

constexpr int kMaxDevices = 64;
std::mutex g_cache_mutex;
bool g_cache_ready[kMaxDevices];
decltype(&cuTensorMapEncodeTiled) g_encode;

// Whether `dev` is a device the kernels run on; looked up once per device.
int cache_device(int dev)
{
    if (dev < 0 || dev >= kMaxDevices) return SV_EDEVICE;
    std::lock_guard<std::mutex> lock(g_cache_mutex);
    if (g_cache_ready[dev]) return SV_OK;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
        cudaGetLastError();
        return SV_EDEVICE;
    }
    if (major != 10 || minor != 3) return SV_EDEVICE;  // built for sm_103a only
    const DeviceGuard guard(dev);
    if (!guard.ok) return SV_EDEVICE;
    for (int cache : {SV_BF16, SV_F16, SV_E4M3})
        for (int dim : {64, 128, 256})
            for (int which = 0; which < 8; ++which) {
                const Kernel k = kernel_of(cache, dim, 16 + which / 2 * 16, which % 2 != 0);
                if (cudaFuncSetAttribute(k.run, cudaFuncAttributeMaxDynamicSharedMemorySize, k.bytes) != cudaSuccess) {
                    cudaGetLastError();
                    return SV_ECUDA;
                }
            }
    if (!g_encode) {
        cudaDriverEntryPointQueryResult found;
        void *f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess || found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return SV_ECUDA;
        }
        g_encode = reinterpret_cast<decltype(g_encode)>(f);
    }
    g_cache_ready[dev] = true;
    return SV_OK;
}

bool misaligned(const void *p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

using wide = __int128;

// An array of up to three strided dimensions of whole heads.
struct View {
    const void *at;
    int64_t size[3], stride[3];  // elements
    int inner, elem;

    // Strides that are whole vectors, none negative, and no offset beyond 2^62 bytes.
    bool sound() const
    {
        wide last = inner;
        for (int d = 0; d < 3; ++d) {
            if (size[d] <= 1) continue;
            if (stride[d] < 0 || stride[d] % (16 / elem) != 0) return false;
            last += static_cast<wide>(size[d] - 1) * stride[d];
        }
        return last * elem < (static_cast<wide>(1) << 62);
    }
#ifdef SV_DEBUG_BOUNDS
    int64_t bytes() const
    {
        int64_t last = inner;
        for (int d = 0; d < 3; ++d)
            if (size[d] > 1) last += (size[d] - 1) * stride[d];
        return last * elem;
    }
#endif
    // No two elements share memory (each stride reaches over all that is within it).
    bool distinct() const
    {
        int order[3] = {0, 1, 2};
        std::sort(order, order + 3, [this](int a, int b) { return stride[a] < stride[b]; });
        wide extent = inner;
        for (int d : order) {
            if (size[d] <= 1) continue;
            if (stride[d] < extent) return false;
            extent += static_cast<wide>(size[d] - 1) * stride[d];
        }
        return true;
    }
};

// The first address of a dimension is all there is where its size is 1: its stride is not looked at.
int64_t stride_of(int64_t size, int64_t stride, int elem) { return size > 1 ? stride * elem : 0; }

int elem_bytes(int dtype) { return dtype == SV_E4M3 ? 1 : 2; }

#ifdef SV_DEBUG_BOUNDS
// The arrays of one call, registered in g_spans (in stream order) before its launch. The environment
// variable SV_DEBUG_SHRINK leaves that many bytes of the end of the first (the cached keys) out, so
// that tests can check that the check fires on memory that is there.
struct SpanList {
    Spans l{};
    void add(const void *p, bool in, bool out, int64_t bytes)
    {
        if (p && bytes > 0 && l.n < kSpans) l.s[l.n++] = Span{reinterpret_cast<u64>(p), static_cast<u64>(bytes), in, out};
    }
    int push(cudaStream_t stream)
    {
        if (const char *e = getenv("SV_DEBUG_SHRINK")) l.s[0].bytes -= std::min<u64>(strtoull(e, nullptr, 10), l.s[0].bytes);
        return cudaMemcpyToSymbolAsync(g_spans, &l, sizeof(l), 0, cudaMemcpyHostToDevice, stream) == cudaSuccess ? SV_OK : SV_ECUDA;
    }
};

template <typename Args>
void add_step(SpanList &s, const Args &a)
{
    s.add(a.page_table, true, false, ((a.num_reqs - 1) * (a.num_reqs > 1 ? a.table_stride : 0) + a.pages_per_req) * 4);
    s.add(a.lengths, true, false, a.num_reqs * 4ll);
    s.add(a.cu_num_draft, true, false, (a.num_reqs + 1) * 4ll);
    s.add(a.k_scale, true, false, a.num_kv_heads * 4ll);
    s.add(a.v_scale, true, false, a.num_kv_heads * 4ll);
}
#endif

// What both entry points ask of the step and the caches. head_dim is checked by the caller.
template <typename Args>
int check_step(const Args &a, View &k, View &v)
{
    if (a.dtype != SV_BF16 && a.dtype != SV_F16) return SV_EDTYPE;
    if (a.cache_dtype != a.dtype && a.cache_dtype != SV_E4M3) return SV_EDTYPE;
    if (a.num_rows < 0 || a.num_reqs < 0 || a.num_kv_heads < 1 || a.num_pages < 0 || a.page_size < 1 || a.pages_per_req < 0) return SV_EINVAL;
    if (a.page_size > SV_MAX_PAGE) return SV_ECAPACITY;
    if (a.cache_dtype != SV_E4M3 && (a.k_scale || a.v_scale)) return SV_EINVAL;
    const int elem = elem_bytes(a.cache_dtype);
    k = View{a.k_cache, {a.num_pages, a.page_size, a.num_kv_heads}, {a.k_page_stride, a.k_slot_stride, a.k_cache_head_stride}, a.head_dim, elem};
    v = View{a.v_cache, {a.num_pages, a.page_size, a.num_kv_heads}, {a.v_page_stride, a.v_slot_stride, a.v_cache_head_stride}, a.head_dim, elem};
    if (!k.sound() || !v.sound()) return SV_EINVAL;
    if (a.num_rows == 0 || a.num_reqs == 0) return SV_OK;
    if (!a.lengths || (a.pages_per_req > 0 && !a.page_table) || (a.num_pages > 0 && (!a.k_cache || !a.v_cache))) return SV_EINVAL;
    if (a.num_reqs > 1 && (a.table_stride < a.pages_per_req || a.table_stride > (1ll << 40))) return SV_EINVAL;
    for (const void *p : {static_cast<const void *>(a.page_table), static_cast<const void *>(a.lengths), static_cast<const void *>(a.cu_num_draft),
                          static_cast<const void *>(a.k_scale), static_cast<const void *>(a.v_scale)})
        if (misaligned(p, 4)) return SV_EINVAL;
    if (misaligned(a.k_cache, 16) || misaligned(a.v_cache, 16)) return SV_EINVAL;
    return SV_OK;
}

template <typename Args>
Step step_of(const Args &a)
{
    return Step{a.page_table, a.lengths, a.cu_num_draft, a.num_reqs > 1 ? a.table_stride : 0, a.num_reqs, a.num_rows, a.num_pages, a.page_size,
                a.pages_per_req, Divider(static_cast<uint32_t>(a.page_size))};
}

Cache cache_of(const View &v)
{
    return Cache{static_cast<unsigned char *>(const_cast<void *>(v.at)), stride_of(v.size[0], v.stride[0], v.elem),
                 stride_of(v.size[1], v.stride[1], v.elem), stride_of(v.size[2], v.stride[2], v.elem)};
}

// Rows of heads: [rows, heads, head_dim] of 16-bit elements.
View rows_of(const void *at, int rows, int heads, int64_t row, int64_t head, int dim) { return View{at, {rows, heads, 1}, {row, head, 0}, dim, 2}; }

// The tensor map of an array of heads, [size2][size1][size0][inner], for copies of boxes of 64 elements of 16 bits, or of whole
// heads of 8, by `box` of the first dimension.
int map_of(CUtensorMap &map, bool bf16, const View &v, int box)
{
    const cuuint64_t sizes[4] = {static_cast<cuuint64_t>(v.inner), static_cast<cuuint64_t>(v.size[0]), static_cast<cuuint64_t>(v.size[1]), static_cast<cuuint64_t>(v.size[2])};
    cuuint64_t strides[3];
    for (int d = 0; d < 3; ++d) strides[d] = static_cast<cuuint64_t>(v.size[d] > 1 ? v.stride[d] : v.inner) * v.elem;
    const bool bytes = v.elem == 1;
    const cuuint32_t boxes[4] = {bytes ? static_cast<cuuint32_t>(v.inner) : 64, static_cast<cuuint32_t>(box), 1, 1}, steps[4] = {1, 1, 1, 1};
    return g_encode(&map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(v.at), sizes, strides, boxes, steps,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SV_OK
               : SV_ECUDA;
}

// Whether copies by tensor map can walk it: every stride in use above 0 (and below 2^36 bytes, which 32 bits hold in vectors).
bool walkable(const View &v)
{
    for (int d = 0; d < 3; ++d)
        if (v.size[d] > 1 && (v.stride[d] < 1 || v.stride[d] * v.elem >= (1ll << 36))) return false;
    return true;
}

int status_of(cudaError_t e)
{
    if (e == cudaSuccess) return SV_OK;
    cudaGetLastError();
    return SV_ECUDA;
}

// Places that a copy by tensor map brings to a tile: whole pages, or equal parts of a page above kTile.
int parts_of(int page) { return (page + kTile - 1) / kTile; }
int places_of(int page) { return page <= kTile ? kTile / page * page : (page + parts_of(page) - 1) / parts_of(page); }

// Copies by tensor map from pages of kSmallPage places on that fill seven eighths of a tile, others vector by vector into whole tiles.
// Measured, tensor map against vectors, us. 16 bits, 32 requests of 6 rows of heads of 128 over up to 16384 keys: pages of 4 places 300 / 225,
// 6 239 / 225, 8 205 / 226, 12 216 / 225, 64 194 / 224, 72 299 / 225 and 96 238 / 225, 112 218 / 225, 200 (two parts of 100) 233 / 225,
// 256 194 / 224; a window and heads of 64: 96 108 / 97, 112 97 / 98; heads of 256: 8 110 / 110, 16 93 / 111. 8 bits, 96 requests of 4 rows of heads of
// 128: 4 173 / 147, 8 142 / 146, 32 132 / 143, 96 168 / 142, 112 152 / 142, 120 146 / 142, 128 133 / 143; 256 of one row: 96 584 / 552, 112 509 / 550, 128 457 / 549.
// (Every place of a tile costs its share of the products, whether it holds a key or not, and each box its issue.) 8 bits also need boxes that start
// on 128 bytes.
constexpr int kSmallPage = 8;
bool by_loads(const spec_verify_cache_attention_args &a)
{
    if (a.page_size < kSmallPage || places_of(a.page_size) * 8 < kTile * 7) return true;
    return a.cache_dtype == SV_E4M3 && a.page_size <= kTile && a.page_size * a.head_dim % 128 != 0;
}

// The kernel for a call. Query rows of a key head of one request (on average: the rows of each are known on the device
// only) in tiles of 16: as few tiles over the keys as there can be, of as few rows.
Kernel kernel_for(const spec_verify_cache_attention_args &a)
{
    const int most = a.head_dim == 256 ? 2 : 4;
    const i64 rows = (static_cast<i64>(a.num_rows) + std::max(a.num_reqs, 1) - 1) / std::max(a.num_reqs, 1) * (a.num_q_heads / a.num_kv_heads);
    const i64 tiles = std::max<i64>(1, (rows + 15) / 16), passes = (tiles + most - 1) / most;
    return kernel_of(a.cache_dtype, a.head_dim, 16 * static_cast<int>((tiles + passes - 1) / passes), by_loads(a));
}

// Tiles of whole pages, or of parts of a page above 128 places, where copies are by tensor map.
Cut cut_of(const spec_verify_cache_attention_args &a, const Kernel &k)
{
    const int page = a.page_size, group = a.num_q_heads / a.num_kv_heads;
    int q_box = k.rows;
    while (group % q_box != 0) --q_box;  // a divisor of the group ...
    while (k.rows % q_box != 0) {        // ... and of the tile
        --q_box;
        while (group % q_box != 0) --q_box;
    }
    if (by_loads(a)) return Cut{kTile, 0, 1, kTile, q_box};
    const int places = places_of(page);
    return page <= kTile ? Cut{places, page, 1, kTile / page, q_box} : Cut{places, places, parts_of(page), 1, q_box};
}

// How many CTAs a call has: those that the device holds at once, or as many as there can be tiles.
i64 most_tiles(const spec_verify_cache_attention_args &a, const Kernel &k)
{
    const Cut cut = cut_of(a, k);
    return std::max<i64>(1, cut.parts > 1 ? static_cast<i64>(a.pages_per_req) * cut.parts : (static_cast<i64>(a.pages_per_req) * a.page_size + cut.span - 1) / cut.span);
}

i64 most_groups(const spec_verify_cache_attention_args &a, const Kernel &k)
{
    return (a.num_reqs + static_cast<i64>(a.num_rows) * (a.num_q_heads / a.num_kv_heads) / k.rows) * a.num_kv_heads;
}

i64 ctas_for(const spec_verify_cache_attention_args &a, const Kernel &k)
{
    const i64 groups = most_groups(a, k), tiles = most_tiles(a, k);
    return groups >= 152 || tiles >= 152 ? 152 : std::min<i64>(152, groups * tiles);
}

// Whether groups may have to be joined: not where each has one tile.
bool joins(const spec_verify_cache_attention_args &a, const Kernel &k) { return most_tiles(a, k) > 1; }

static_assert(SV_CACHE_WORKSPACE == 152 * (2 * 64 * (128 + 2) * 4 + sizeof(Part)), "the largest of the kernels'");

int64_t workspace_of(const spec_verify_cache_attention_args &a, const Kernel &k)
{
    return joins(a, k) ? ctas_for(a, k) * (2ll * k.rows * (k.dim + 2) * 4 + static_cast<int64_t>(sizeof(Part))) : 0;
}

int launch_after(const void *kernel, unsigned grid, unsigned block, int bytes, cudaStream_t stream, void **params)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return status_of(cudaLaunchKernelExC(&cfg, kernel, params));
}

// What an attention call asks beyond its step.
int check_attention(const spec_verify_cache_attention_args &a, View &k, View &v)
{
    if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return SV_EINVAL;
    const int rc = check_step(a, k, v);
    if (rc != SV_OK) return rc;
    if (a.num_q_heads < 1 || a.num_q_heads % a.num_kv_heads != 0 || a.window < 0 || !std::isfinite(a.scale)) return SV_EINVAL;
    if (static_cast<int64_t>(a.pages_per_req) * a.page_size > kMaxPlace) return SV_ECAPACITY;
    if (static_cast<int64_t>(a.num_rows) * (a.num_q_heads / a.num_kv_heads) >= (1ll << 31)) return SV_ECAPACITY;
    return SV_OK;
}

}  // namespace

extern "C" int spec_verify_cache_append(const spec_verify_cache_append_args *a, void *cuda_stream)
{
    const NvtxRange nvtx("spec_verify_cache_append");
    if (!a) return SV_EINVAL;
    if (a->head_dim < 16 || a->head_dim % 16 != 0 || a->rotary_dim < 0 || a->rotary_dim % 16 != 0 || a->rotary_dim > a->head_dim) return SV_EINVAL;
    if (a->head_dim > SV_MAX_HEAD_DIM) return SV_ECAPACITY;
    View kc, vc;
    const int rc = check_step(*a, kc, vc);
    if (rc != SV_OK) return rc;
    if (!kc.distinct() || !vc.distinct() || a->num_q_heads < 0) return SV_EINVAL;
    if (static_cast<i64>(a->num_q_heads) + 2ll * a->num_kv_heads > 65536) return SV_ECAPACITY;
    if (a->num_pages > 0 && a->k_cache == a->v_cache) return SV_EINVAL;
    if (a->rotary_dim > 0 && (!a->inv_freq || misaligned(a->inv_freq, 4))) return SV_EINVAL;
    if (a->positions && (a->num_axes < 1 || misaligned(a->positions, 4) || (a->num_axes > 1 && a->positions_stride < a->num_rows))) return SV_EINVAL;
    if (a->positions && a->num_axes > SV_MAX_AXES) return SV_ECAPACITY;
    if (a->axes && !a->positions) return SV_EINVAL;
    AppendParams P;
    memset(P.axes, 0, sizeof(P.axes));
    for (int m = 0; a->axes && m < a->rotary_dim / 2; ++m) {
        if (a->axes[m] >= a->num_axes) return SV_EINVAL;
        P.axes[m / 16] |= static_cast<uint32_t>(a->axes[m]) << (m % 16 * 2);
    }
    const int D = a->head_dim;
    const View q = rows_of(a->q, a->num_rows, a->num_q_heads, a->q_row_stride, a->q_head_stride, D);
    const View out = rows_of(a->q_out, a->num_rows, a->num_q_heads, a->q_out_row_stride, a->q_out_head_stride, D);
    const View k = rows_of(a->k, a->num_rows, a->num_kv_heads, a->k_row_stride, a->k_head_stride, D);
    const View v = rows_of(a->v, a->num_rows, a->num_kv_heads, a->v_row_stride, a->v_head_stride, D);
    if (!q.sound() || !out.sound() || (a->num_q_heads > 0 && !out.distinct()) || !k.sound() || !v.sound()) return SV_EINVAL;
    if (a->num_rows == 0 || a->num_reqs == 0) return SV_OK;
    if (!a->k || !a->v || (a->num_q_heads > 0 && (!a->q || !a->q_out))) return SV_EINVAL;
    for (const void *p : {a->q, a->k, a->v, static_cast<const void *>(a->q_out)})
        if (misaligned(p, 16)) return SV_EINVAL;
    // in place means every element in its own place
    if (a->q == a->q_out && ((a->num_rows > 1 && a->q_row_stride != a->q_out_row_stride) || (a->num_q_heads > 1 && a->q_head_stride != a->q_out_head_stride)))
        return SV_EINVAL;
    const int rd = cache_device(a->device);
    if (rd != SV_OK) return rd;
    const DeviceGuard guard(a->device);
    if (!guard.ok) return SV_EDEVICE;
    P.s = step_of(*a);
    P.q = static_cast<const unsigned char *>(a->q);
    P.k = static_cast<const unsigned char *>(a->k);
    P.v = static_cast<const unsigned char *>(a->v);
    P.q_out = static_cast<unsigned char *>(a->q_out);
    P.q_row = stride_of(a->num_rows, a->q_row_stride, 2);
    P.q_head = stride_of(a->num_q_heads, a->q_head_stride, 2);
    P.k_row = stride_of(a->num_rows, a->k_row_stride, 2);
    P.k_head = stride_of(a->num_kv_heads, a->k_head_stride, 2);
    P.v_row = stride_of(a->num_rows, a->v_row_stride, 2);
    P.v_head = stride_of(a->num_kv_heads, a->v_head_stride, 2);
    P.out_row = stride_of(a->num_rows, a->q_out_row_stride, 2);
    P.out_head = stride_of(a->num_q_heads, a->q_out_head_stride, 2);
    P.kc = cache_of(kc);
    P.vc = cache_of(vc);
    P.inv_freq = a->inv_freq;
    P.k_scale = a->k_scale;
    P.v_scale = a->v_scale;
    P.positions = a->positions;
    P.positions_stride = a->num_axes > 1 ? a->positions_stride : 0;
    P.hq = a->num_q_heads;
    P.hk = a->num_kv_heads;
    P.dim = D;
    P.half = a->rotary_dim / 2;
    P.interleaved = a->interleaved;
    const auto stream = static_cast<cudaStream_t>(cuda_stream);
#ifdef SV_DEBUG_BOUNDS
    SpanList s;
    s.add(a->k_cache, false, true, kc.bytes());
    s.add(a->v_cache, false, true, vc.bytes());
    if (a->num_q_heads) {
        s.add(a->q, true, false, q.bytes());
        s.add(a->q_out, false, true, out.bytes());
    }
    s.add(a->k, true, false, k.bytes());
    s.add(a->v, true, false, v.bytes());
    s.add(a->inv_freq, true, false, a->rotary_dim * 2ll);
    s.add(a->positions, true, false, ((a->num_axes - 1) * P.positions_stride + a->num_rows) * 4);
    add_step(s, *a);
    if (s.push(stream) != SV_OK) return SV_ECUDA;
#endif
    // Parts of a row where there are fewer rows than the device holds warps (32 an SM): no more than one a warp, of 32 items
    // at least.
    const int items = (P.hq + 2 * P.hk) * (D / 16), most = (items + 31) / 32;
    P.parts = std::max(1, std::min(most, 152 * 32 / a->num_rows));
    P.items = (items + P.parts - 1) / P.parts;
    P.by_parts = Divider(static_cast<uint32_t>(P.parts));
    P.by_items_a_head = Divider(static_cast<uint32_t>(D / 16));
    const i64 blocks = (static_cast<i64>(a->num_rows) * P.parts + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    const void *kernel = a->dtype == SV_BF16
                             ? a->cache_dtype == SV_E4M3 ? reinterpret_cast<const void *>(sv_cache_append_kernel<__nv_bfloat16, true>)
                                                         : reinterpret_cast<const void *>(sv_cache_append_kernel<__nv_bfloat16, false>)
                         : a->cache_dtype == SV_E4M3 ? reinterpret_cast<const void *>(sv_cache_append_kernel<__half, true>)
                                                     : reinterpret_cast<const void *>(sv_cache_append_kernel<__half, false>);
    void *params[] = {&P};
    return launch_after(kernel, static_cast<unsigned>(std::min<i64>(blocks, kAppendBlocks)), kAppendThreads, 0, stream, params);
}

extern "C" int spec_verify_cache_attention_workspace(const spec_verify_cache_attention_args *a, int64_t *bytes)
{
    if (!a || !bytes) return SV_EINVAL;
    spec_verify_cache_attention_args sizes = *a;  // (the sizes alone: no address is looked at)
    sizes.num_rows = 0;
    View k, v;
    const int rc = a->num_rows < 0 ? SV_EINVAL : check_attention(sizes, k, v);
    *bytes = rc == SV_OK && a->num_rows > 0 && a->num_reqs > 0 ? workspace_of(*a, kernel_for(*a)) : 0;
    return rc;
}

extern "C" int spec_verify_cache_attention(const spec_verify_cache_attention_args *a, void *cuda_stream)
{
    const NvtxRange nvtx("spec_verify_cache_attention");
    if (!a) return SV_EINVAL;
    View kc, vc;
    const int rc = check_attention(*a, kc, vc);
    if (rc != SV_OK) return rc;
    const View q = rows_of(a->q, a->num_rows, a->num_q_heads, a->q_row_stride, a->q_head_stride, a->head_dim);
    const View out = rows_of(a->out, a->num_rows, a->num_q_heads, a->out_row_stride, a->out_head_stride, a->head_dim);
    if (!q.sound() || !out.sound() || !out.distinct() || !walkable(q) || !walkable(kc) || !walkable(vc)) return SV_EINVAL;
    if (a->num_rows == 0 || a->num_reqs == 0) return SV_OK;
    if (!a->q || !a->out || a->q == a->out || misaligned(a->q, 16) || misaligned(a->out, 16) || misaligned(a->lse, 4)) return SV_EINVAL;
    const Kernel kernel = kernel_for(*a);
    if (static_cast<wide>(most_groups(*a, kernel)) * most_tiles(*a, kernel) >= (1ll << 31)) return SV_ECAPACITY;
    const int64_t workspace = workspace_of(*a, kernel);
    if (a->workspace_bytes < workspace || (workspace > 0 && !a->workspace) || misaligned(a->workspace, 16)) return SV_EINVAL;
    const int rd = cache_device(a->device);
    if (rd != SV_OK) return rd;
    const DeviceGuard guard(a->device);
    if (!guard.ok) return SV_EDEVICE;
    AttentionParams P;
    P.s = step_of(*a);
    P.q = static_cast<const unsigned char *>(a->q);
    P.out = static_cast<unsigned char *>(a->out);
    P.q_row = stride_of(a->num_rows, a->q_row_stride, 2);
    P.q_head = stride_of(a->num_q_heads, a->q_head_stride, 2);
    P.out_row = stride_of(a->num_rows, a->out_row_stride, 2);
    P.out_head = stride_of(a->num_q_heads, a->out_head_stride, 2);
    P.kc = cache_of(kc);
    P.vc = cache_of(vc);
    P.k_scale = a->k_scale;
    P.v_scale = a->v_scale;
    P.lse = a->lse;
    P.scale = a->scale * kLog2e;
    P.window = a->window;
    P.hq = a->num_q_heads;
    P.hk = a->num_kv_heads;
    P.group = a->num_q_heads / a->num_kv_heads;
    P.bf16 = a->dtype == SV_BF16;
    P.cut = cut_of(*a, kernel);
    P.by_group = Divider(static_cast<uint32_t>(P.group));
    P.by_span = Divider(static_cast<uint32_t>(P.cut.span));
    P.by_parts = Divider(static_cast<uint32_t>(P.cut.parts));
    const i64 ctas = ctas_for(*a, kernel);
    P.sums = static_cast<float *>(workspace ? a->workspace : nullptr);
    P.stats = workspace ? reinterpret_cast<float2 *>(P.sums + ctas * 2 * kernel.rows * kernel.dim) : nullptr;
    P.parts = workspace ? reinterpret_cast<Part *>(P.stats + ctas * 2 * kernel.rows) : nullptr;
    const auto stream = static_cast<cudaStream_t>(cuda_stream);
#ifdef SV_DEBUG_BOUNDS
    SpanList s;
    s.add(a->k_cache, true, false, kc.bytes());
    s.add(a->v_cache, true, false, vc.bytes());
    s.add(a->q, true, false, q.bytes());
    s.add(a->out, false, true, out.bytes());
    s.add(a->lse, false, true, static_cast<int64_t>(a->num_rows) * a->num_q_heads * 4);
    s.add(a->workspace, true, true, a->workspace_bytes);
    add_step(s, *a);
    if (s.push(stream) != SV_OK) return SV_ECUDA;
    // SV_DEBUG_PATIENCE: looks of a wait before it is given up
    P.patience = kPatience;
    if (const char *e = getenv("SV_DEBUG_PATIENCE")) P.patience = std::max(1, std::min(kPatience, atoi(e)));
#endif
    TensorMaps maps;
    memset(&maps, 0, sizeof(maps));
    const bool bf16 = a->cache_dtype == SV_BF16;
    if (a->cache_dtype != SV_E4M3) {
        const View queries{a->q, {a->num_q_heads, a->num_rows, 1}, {a->q_head_stride, a->q_row_stride, 0}, a->head_dim, 2};
        if (map_of(maps.q, bf16, queries, P.cut.q_box) != SV_OK) return SV_ECUDA;
    }
    if (P.cut.box) {
        // (sizes of the map: slots, heads, pages. Without a page only zeros come of it, whatever it names)
        auto turned = [&](const View &c) {
            View v{a->num_pages ? c.at : a->q, {c.size[1], c.size[2], c.size[0]}, {c.stride[1], c.stride[2], c.stride[0]}, c.inner, c.elem};
            if (!a->num_pages) v.size[0] = v.size[1] = v.size[2] = 1;
            return v;
        };
        if (map_of(maps.k, bf16, turned(kc), P.cut.box) != SV_OK || map_of(maps.v, bf16, turned(vc), P.cut.box) != SV_OK) return SV_ECUDA;
    }
    // Each kernel may start while the one before it ends; it waits for that on the device before it looks at memory.
    void *params[] = {&P, &maps};
    int rc_launch = launch_after(kernel.run, static_cast<unsigned>(ctas), static_cast<unsigned>(kernel.threads), kernel.bytes, stream, params);
    if (rc_launch != SV_OK || !workspace) return rc_launch;
    int rows = kernel.rows;
    float offset = kernel.offset;
    void *join[] = {&P, &rows, &offset};
    return launch_after(kernel.join, static_cast<unsigned>(ctas), kJoinThreads, 0, stream, join);
}

extern "C" int spec_verify_cache_last_error(uint32_t *err_word)
{
    if (!err_word) return SV_EINVAL;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return SV_EDEVICE;
    }
    const int rc = cache_device(dev);
    if (rc != SV_OK) return rc;
    const unsigned zero = 0;
    unsigned w = 0;
    if (cudaDeviceSynchronize() != cudaSuccess || cudaMemcpyFromSymbol(&w, g_cache_error, sizeof(w)) != cudaSuccess ||
        (w && cudaMemcpyToSymbol(g_cache_error, &zero, sizeof(zero)) != cudaSuccess))
        return SV_ECUDA;
    *err_word = w;
    return SV_OK;
}

#ifdef SV_DEBUG_BOUNDS
// Of the checked build only: SV_ERR_BOUNDS in *word if a kernel of a cache operator that has ended tried an
// access outside its call's arrays (the current device's; read and cleared).
extern "C" int spec_verify_cache_outside(uint32_t *word)
{
    const unsigned zero = 0;
    if (!word) return SV_EINVAL;
    return cudaMemcpyFromSymbol(word, g_outside, sizeof(*word)) == cudaSuccess &&
                   cudaMemcpyToSymbol(g_outside, &zero, sizeof(zero)) == cudaSuccess
               ? SV_OK
               : SV_ECUDA;
}
#endif
