// What the cache operators share: the rows of a step and the places of the paged cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "spec_verify.h"

namespace sv_cache {

using i64 = long long;
using u64 = unsigned long long;

constexpr float kInf = __builtin_huge_valf();

// Division of whole numbers below 2^31 by one of 1 to 2^31 - 1: with 2^l the power of two from the divisor on,
// by = ceil(2^(31 + l) / divisor) is off by less than 1 in 2^l steps, so x by / 2^(31 + l) is off by less than x / 2^31 < 1.
struct Divider {
    uint32_t by;
    int shift;
    explicit Divider(uint32_t divisor = 1)
    {
        int l = 0;
        while ((uint64_t{1} << l) < divisor) ++l;
        shift = 31 + l;
        by = static_cast<uint32_t>(((uint64_t{1} << shift) + divisor - 1) / divisor);
    }
    __device__ __forceinline__ int operator()(int x) const { return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(x)) * by) >> shift); }
};

// The requests of a step and where their keys are.
struct Step {
    const int32_t *table, *lengths, *cu;  // cu NULL: one row a request
    i64 table_stride;
    int n, rows, pages, page, width;      // requests, rows, pages of the pool, slots of a page, pages of a request at most
    Divider by_page;
};

// One cache: address and strides in bytes.
struct Cache {
    unsigned char *at;
    i64 page, slot, head;
};

// ---------------------------------------------------------------------------------------
// global memory
// ---------------------------------------------------------------------------------------
// Every global load and store of the cache operators goes through these. Built with -DSV_DEBUG_BOUNDS
// each is checked against the extents of the call's arrays (loads against its inputs and its
// workspace, stores against its outputs and its workspace), which the host registers before the
// launch: one that is outside is skipped (a load gives 0) and leaves a mark that
// spec_verify_cache_outside() reads. In a normal build they are plain accesses.
#ifdef SV_DEBUG_BOUNDS
struct Span {
    u64 at, bytes;
    int in, out;
};
constexpr int kSpans = 16;
struct Spans {
    Span s[kSpans];
    int n;
};
static __device__ Spans g_spans;
static __device__ unsigned g_outside;

static __device__ __noinline__ bool inside(const void *p, unsigned bytes, bool out)
{
    const u64 a = reinterpret_cast<u64>(p);
    for (int k = 0; k < g_spans.n; ++k) {
        const Span &s = g_spans.s[k];
        if ((out ? s.out : s.in) && a >= s.at && a - s.at + bytes <= s.bytes) return true;
    }
    atomicOr(&g_outside, SV_ERR_BOUNDS);
    return false;
}
#define SV_CACHE_INSIDE(p, bytes, out) inside((p), (bytes), (out))
#else
#define SV_CACHE_INSIDE(p, bytes, out) true
#endif

// Not by the read-only path: it is for memory that nobody writes while the kernel lives, and these kernels live before the work that
// writes their inputs (lengths, prefix sums, the queries that an append has turned) has ended; and queries may be turned in place.
template <typename T>
__device__ __forceinline__ T ld(const T *p)
{
    if (!SV_CACHE_INSIDE(p, sizeof(T), false)) return T{};
    return *p;
}
template <typename T>
__device__ __forceinline__ void st(T *p, const T &v)
{
    if (SV_CACHE_INSIDE(p, sizeof(T), true)) *p = v;
}

// ---------------------------------------------------------------------------------------
// rows and places
// ---------------------------------------------------------------------------------------
// The rows of request i: the first, and how many; none where they are not all rows of the step.
__device__ __forceinline__ int request_rows(const Step &s, int i, int &first)
{
    if (!s.cu) {
        first = i;
        return i < s.rows;
    }
    const int a = ld(s.cu + i), b = ld(s.cu + i + 1);
    const i64 at = static_cast<i64>(a) + i, count = static_cast<i64>(b) - a + 1;
    first = static_cast<int>(at);
    return a >= 0 && count >= 1 && at + count <= s.rows ? static_cast<int>(count) : 0;
}

// The request of row r (found by the 32 lanes of a warp together, 33 parts a look), -1 where it has none.
__device__ __forceinline__ int request_of(const Step &s, int r)
{
    if (!s.cu) return r < s.n ? r : -1;
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = s.n;  // the last request whose first row is at most r is in [lo, hi), if there is one
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const bool at = i < hi && static_cast<i64>(ld(s.cu + i)) + i <= r;
        const int k = __popc(__ballot_sync(~0u, at));  // (with an inconsistent cu some request, checked below)
        if (k == 0) return -1;
        lo += (k - 1) * step;
        hi = min(hi, lo + step);
    }
    int first;
    const int count = request_rows(s, lo, first);
    return lo < s.n && count > 0 && r >= first && r - first < count ? lo : -1;  // (without rows `first` may be any number)
}

// Page and slot of place x of request i; false where it has none.
__device__ __forceinline__ bool place(const Step &s, int i, i64 x, i64 &page, int &slot)
{
    if (x < 0 || x >= static_cast<i64>(s.width) * s.page) return false;
    const i64 c = x < (1ll << 31) ? s.by_page(static_cast<int>(x)) : x / s.page;
    slot = static_cast<int>(x - c * s.page);
    page = ld(s.table + i * s.table_stride + c);
    return page >= 0 && page < s.pages;
}

// ---------------------------------------------------------------------------------------
// elements
// ---------------------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float2 pair_of(uint32_t w);
template <>
__device__ __forceinline__ float2 pair_of<__nv_bfloat16>(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 pair_of<__half>(uint32_t w)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// Two e4m3 as binary16 (exact, NaN stays NaN).
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t w)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
    return r;
}
// (a, b) as e4m3, a in the lower byte; beyond 448 becomes 448.
__device__ __forceinline__ uint32_t e4m3_of(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

}  // namespace sv_cache
