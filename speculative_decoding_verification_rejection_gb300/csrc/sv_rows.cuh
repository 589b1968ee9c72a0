// Arithmetic of the row operators: clusters, logits and weights. See sv_rows.cu for the mathematics.
#pragma once

#include <cfloat>
#include <climits>
#include <cstdint>
#include <cstring>

#include "spec_verify.h"
#include "sv_device.cuh"

namespace sv_rows {

using u64 = unsigned long long;

constexpr int kMaxCluster = 8;
constexpr int kAhead = 8;         // vectors a lane reads before it uses the first
constexpr int kList = 1024;       // entries of the leader's candidate list
constexpr int kHits = 2048;       // groups a CTA looks through for candidates
constexpr int kPairs = 256;       // most entries that are compared each with each, and the threads that do it
constexpr int kFewPairs = 128;    // most that are so before the k largest are picked out
constexpr int kTopP = 64;         // lane maxima that the cut for top-p alone is to reach, of a CTA of two at most
constexpr int kWideList = 2048;   // the same of a bracket's tokens
constexpr int kBeside = 64;       // tokens on each side of a guess
constexpr int kBins = 4096;       // bins of the value histogram
constexpr float kSpan = 28.5f;    // the d they cover: below -28.43 a weight is 0
constexpr float kInf = __builtin_huge_valf();
constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kRise = 4.0f;     // doublings that a log-probability's logits pass their reference by before it moves
static_assert(kPairs <= 256, "a sum of weights below 2^48, and a number above it, in 64 bits");
static_assert(kWideList < 4096, "sums of the weights' upper 20 bits in 32");

// What a launch is told.
struct Split {
    int per_cta, per_warp;  // vectors
};
struct SampleParams {
    long long stride, probs_stride;
    const float *temperature, *top_p, *min_p, *uniforms;
    const int32_t *top_k;
    int32_t *tokens;
    float *logprob, *probs;
    int V, cluster, ordered;  // ordered: the rows, where those that may take long come first, else 0
    Split split;
};
struct LogprobParams {
    long long stride;
    const float *temperature;
    const int32_t *tokens, *cu;
    int token_stride, num_reqs, num_top, V, cluster;
    float *logprob, *top_logprob;
    int32_t *rank, *top_ids;
    Split split;
};

// ---------------------------------------------------------------------------------------
// global memory
// ---------------------------------------------------------------------------------------
// Every global load and store of the row operators goes through these. Built with -DSV_DEBUG_BOUNDS
// each is checked against the rows of the call's arrays (loads against its inputs, stores against its
// outputs; what lies between the rows of a strided array is outside), which the host registers before
// the launch: one that is outside is skipped (a load gives 0) and leaves a mark that
// spec_verify_rows_outside() reads. In a normal build they are plain accesses.
#ifdef SV_DEBUG_BOUNDS
struct Span {
    u64 at, stride, bytes, rows;  // rows of `bytes` bytes, `stride` apart
    bool out;
};
constexpr int kSpans = 12;
struct Spans {
    Span s[kSpans];
    int n;
};
__device__ Spans g_spans;
__device__ unsigned g_outside;

__device__ __noinline__ bool inside(const void *p, unsigned bytes, bool out)
{
    const u64 a = reinterpret_cast<u64>(p);
    for (int k = 0; k < g_spans.n; ++k) {
        const Span &s = g_spans.s[k];
        if (a < s.at || s.out != out) continue;
        const u64 off = a - s.at, row = s.rows > 1 ? off / s.stride : 0;
        if (row < s.rows && off - row * s.stride + bytes <= s.bytes) return true;
    }
    atomicOr(&g_outside, SV_ERR_BOUNDS);
    return false;
}
#define SV_INSIDE(p, bytes, out) inside((p), (bytes), (out))
#else
#define SV_INSIDE(p, bytes, out) true
#endif

template <typename T>
__device__ __forceinline__ T ld(const T *p)
{
    if (!SV_INSIDE(p, sizeof(T), false)) return T{};
    return __ldg(p);
}
// A vector of a row of logits, read once a pass: not kept in L1.
__device__ __forceinline__ uint4 ld_row(const uint4 *p)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (SV_INSIDE(p, 16, false))
        asm("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
template <typename T, typename U>
__device__ __forceinline__ void st(T *p, const U &v)
{
    if (SV_INSIDE(p, sizeof(T), true)) *p = v;
}
// Four floats that leave the L2 cache first.
__device__ __forceinline__ void st_leaving(float4 *p, const float4 &v)
{
    if (SV_INSIDE(p, sizeof(float4), true)) __stcs(p, v);
}

// ---------------------------------------------------------------------------------------
// thread-block clusters
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ unsigned smem_addr(const void *p) { return static_cast<unsigned>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ unsigned cluster_rank()
{
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA of the cluster; what was written before (shared memory of any CTA of
// the cluster, global memory) is visible after.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_announce() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}
// Address of p, of this CTA's shared memory, in that of CTA `rank`.
__device__ __forceinline__ unsigned remote(const void *p, unsigned rank)
{
    unsigned a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void put(unsigned a, unsigned v) { asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ void put(unsigned a, u64 v) { asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(v) : "memory"); }

__device__ __forceinline__ uint4 get16(unsigned a)
{
    uint4 v;
    asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// ---------------------------------------------------------------------------------------
// logits and weights
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ float as_float(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ float as_float(float f) { return f; }
template <typename T> struct Low;  // -inf in the logits' type
template <> struct Low<uint16_t> {
    static constexpr unsigned word = 0xFF80FF80u;
    static __device__ __forceinline__ uint16_t value() { return 0xFF80u; }
};
template <> struct Low<float> {
    static constexpr unsigned word = 0xFF800000u;
    static __device__ __forceinline__ float value() { return -kInf; }
};

// The logits of a 16-byte vector as binary32.
template <typename T> struct Vec;
template <> struct Vec<uint16_t> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void get(const uint4 &v, float (&f)[8])
    {
        const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <> struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void get(const uint4 &v, float (&f)[4])
    {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
};

// The largest of the logits added and -inf; a NaN loses.
template <typename T> struct Largest;
template <> struct Largest<uint16_t> {
    unsigned a = 0xFF80FF80u, b = 0xFF80FF80u;  // (two chains)
    static __device__ __forceinline__ unsigned pick(unsigned x, unsigned y)
    {
        unsigned r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        return r;
    }
    __device__ __forceinline__ void add(const uint4 &v)
    {
        a = pick(pick(a, v.x), v.y);
        b = pick(pick(b, v.z), v.w);
    }
    __device__ __forceinline__ float get() const
    {
        const unsigned m = pick(a, b);
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
};
template <> struct Largest<float> {
    float a = -kInf, b = -kInf;
    __device__ __forceinline__ void add(const uint4 &v)
    {
        a = fmaxf(fmaxf(a, __uint_as_float(v.x)), __uint_as_float(v.y));
        b = fmaxf(fmaxf(b, __uint_as_float(v.z)), __uint_as_float(v.w));
    }
    __device__ __forceinline__ float get() const { return fmaxf(a, b); }
};

// How many of the logits added are above a bound. The bf16 form counts in bf16, which is exact up to
// 256 in each half: flush() at the latest after 64 vectors.
template <typename T> struct Above;
template <> struct Above<uint16_t> {
    unsigned bound, part = 0, count = 0;
    explicit __device__ __forceinline__ Above(float l) { bound = __float_as_uint(l) >> 16; bound |= bound << 16; }
    __device__ __forceinline__ void add(const uint4 &v)
    {
        const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            unsigned one;
            asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(one) : "r"(w[i]), "r"(bound));
            asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(part) : "r"(one));
        }
    }
    __device__ __forceinline__ void flush()
    {
        count += static_cast<unsigned>(__uint_as_float(part << 16) + __uint_as_float(part & 0xFFFF0000u));
        part = 0;
    }
    __device__ __forceinline__ unsigned get() const { return count; }
};
template <> struct Above<float> {
    float bound;
    unsigned count = 0;
    explicit __device__ __forceinline__ Above(float l) : bound(l) {}
    __device__ __forceinline__ void add(const uint4 &v)
    {
        count += __uint_as_float(v.x) > bound;
        count += __uint_as_float(v.y) > bound;
        count += __uint_as_float(v.z) > bound;
        count += __uint_as_float(v.w) > bound;
    }
    __device__ __forceinline__ void flush() {}
    __device__ __forceinline__ unsigned get() const { return count; }
};

// Two binary32 values and the packed operations on them (each rounded as the single one).
struct Two {
    u64 v;
};
__device__ __forceinline__ Two two(float a, float b)
{
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ Two two(float a) { return two(a, a); }
__device__ __forceinline__ void parts(Two t, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(t.v)); }
__device__ __forceinline__ Two operator+(Two a, Two b)
{
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two operator*(Two a, Two b)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two fma(Two a, Two b, Two c)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// A vector of a row whose largest logit is +inf: 0 for the tokens at +inf, which share the row, and
// -inf for the others.
template <typename T>
__device__ __forceinline__ uint4 only_inf(uint4 v)
{
    T e[Vec<T>::n];
    memcpy(e, &v, 16);
#pragma unroll
    for (int i = 0; i < Vec<T>::n; ++i) e[i] = as_float(e[i]) == kInf ? T(0) : Low<T>::value();
    memcpy(&v, e, 16);
    return v;
}

// Logits as order-preserving unsigned integers, 0 for what is never kept (NaN and -inf); -0 as +0.
__device__ __forceinline__ unsigned key_of(float l)
{
    if (!(l > -kInf)) return 0u;
    const unsigned b = __float_as_uint(__fadd_rn(l, 0.0f));
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_key(unsigned k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k); }

// 1 / T as a normal number: an infinite T then gives a difference that overflowed a d of -inf, not
// of 0 times infinity, and a tiny T a finite factor for the differences that are 0.
__device__ __forceinline__ float inverse(float T) { return fminf(fmaxf(__frcp_rn(T), FLT_MIN), FLT_MAX); }

// d of a logit, L finite (a row with L = +inf is rewritten first); NaN for a NaN.
__device__ __forceinline__ float delta(float l, float L, float inv) { return __fmul_rn(__fsub_rn(l, L), inv); }

// sv::exp_f32 for d <= 0 where only the weight is wanted: below -32 a weight is 0 anyway, and so
// is that of a NaN or -inf, which the maximum takes to -32. The same operations otherwise; the
// factor 2^k goes into the exponent, which stays that of a normal number.
__device__ __forceinline__ float exp_weight(float d)
{
    d = fmaxf(d, -32.0f);
    const float shifter = 0x1.8p+23f;
    const float ks = __fmaf_rn(d, 0x1.715476p+0f, shifter);
    const float kf = __fsub_rn(ks, shifter);
    float r = __fmaf_rn(-kf, 0x1.62e430p-1f, d);
    r = __fmaf_rn(-kf, -0x1.05c610p-29f, r);
    float p = 0x1.a01a02p-13f;
    p = __fmaf_rn(p, r, 0x1.6c16c2p-10f);
    p = __fmaf_rn(p, r, 0x1.111112p-7f);
    p = __fmaf_rn(p, r, 0x1.555556p-5f);
    p = __fmaf_rn(p, r, 0x1.555556p-3f);
    p = __fmaf_rn(p, r, 0.5f);
    p = __fmaf_rn(p, r, 1.0f);
    p = __fmaf_rn(p, r, 1.0f);
    return __uint_as_float(__float_as_uint(p) + (__float_as_uint(ks) << 23));
}

__device__ __forceinline__ Two exp_weight(Two d)
{
    float a, b;
    parts(d, a, b);
    d = two(fmaxf(a, -32.0f), fmaxf(b, -32.0f));
    const Two ks = fma(d, two(0x1.715476p+0f), two(0x1.8p+23f));
    const Two kf = ks + two(-0x1.8p+23f);
    Two r = fma(kf, two(-0x1.62e430p-1f), d);
    r = fma(kf, two(0x1.05c610p-29f), r);
    Two p = fma(two(0x1.a01a02p-13f), r, two(0x1.6c16c2p-10f));
    p = fma(p, r, two(0x1.111112p-7f));
    p = fma(p, r, two(0x1.555556p-5f));
    p = fma(p, r, two(0x1.555556p-3f));
    p = fma(p, r, two(0.5f));
    p = fma(p, r, two(1.0f));
    p = fma(p, r, two(1.0f));
    float pa, pb, ka, kb;
    parts(p, pa, pb);
    parts(ks, ka, kb);
    return two(__uint_as_float(__float_as_uint(pa) + (__float_as_uint(ka) << 23)),
               __uint_as_float(__float_as_uint(pb) + (__float_as_uint(kb) << 23)));
}

// sv::exp_f32 of two d <= 0.
__device__ __forceinline__ Two exp_two(Two d)
{
    float da, db, a, b;
    parts(d, da, db);
    const Two x = two(fmaxf(da, -87.0f), fmaxf(db, -87.0f));
    const Two ks = fma(x, two(0x1.715476p+0f), two(0x1.8p+23f));
    const Two kf = ks + two(-0x1.8p+23f);
    Two r = fma(kf, two(-0x1.62e430p-1f), x);
    r = fma(kf, two(0x1.05c610p-29f), r);
    Two p = fma(two(0x1.a01a02p-13f), r, two(0x1.6c16c2p-10f));
    p = fma(p, r, two(0x1.111112p-7f));
    p = fma(p, r, two(0x1.555556p-5f));
    p = fma(p, r, two(0x1.555556p-3f));
    p = fma(p, r, two(0.5f));
    p = fma(p, r, two(1.0f));
    p = fma(p, r, two(1.0f));
    parts(ks, a, b);
    p = p * two(__uint_as_float((__float_as_uint(a) + 127u) << 23), __uint_as_float((__float_as_uint(b) + 127u) << 23));
    parts(p, a, b);
    return two(da >= -87.0f ? a : 0.0f, db >= -87.0f ? b : 0.0f);
}

// An exact sum of weights in two 32-bit words. Adding 12 to t in [0, 1] rounds it to a multiple of
// 2^-20, whose count the low mantissa bits then hold; what that left, at most 2^-21, is rounded to
// a multiple of 2^-40 by adding 1.5 2^-17 in the same way. Together they are rint(t 2^40), ties as
// rint's. The words add the bit patterns; the constant parts come off at the end. Good for up to
// kMostWeights weights. (Nothing here is done in binary64, nor by conversions to 64-bit integers: this
// part runs those at a sixtieth of the binary32 rate.)
constexpr int kMostWeights = 4095;  // (each adds up to 2^20 to the first word)
struct WeightSum {
    unsigned a = 0, b = 0;
    __device__ __forceinline__ void add(float t)
    {
        const float x = __fadd_rn(t, 12.0f);
        const float lo = __fsub_rn(t, __fsub_rn(x, 12.0f));
        a += __float_as_uint(x);
        b += __float_as_uint(__fadd_rn(lo, 0x1.8p-17f));
    }
    __device__ __forceinline__ void add(Two t)
    {
        const Two x = t + two(12.0f);
        const Two y = fma(x + two(-12.0f), two(-1.0f), t) + two(0x1.8p-17f);
        float p, q;
        parts(x, p, q);
        a += __float_as_uint(p) + __float_as_uint(q);
        parts(y, p, q);
        b += __float_as_uint(p) + __float_as_uint(q);
    }
    __device__ __forceinline__ u64 total(int n) const  // n: how many were added
    {
        const unsigned hi = a - static_cast<unsigned>(n) * __float_as_uint(12.0f);
        const int lo = static_cast<int>(b - static_cast<unsigned>(n) * __float_as_uint(0x1.8p-17f));
        return (static_cast<u64>(hi) << 20) + static_cast<u64>(static_cast<long long>(lo));
    }
};

// Two such sums at once: of all weights added, and of those that are marked.
struct WeightSums {
    unsigned a = 0, b = 0, ma = 0, mb = 0;
    __device__ __forceinline__ void add(Two t, bool first, bool second)
    {
        const Two x = t + two(12.0f);
        const Two y = fma(x + two(-12.0f), two(-1.0f), t) + two(0x1.8p-17f);
        float p, q;
        parts(x, p, q);
        a += __float_as_uint(p) + __float_as_uint(q);
        ma += (first ? __float_as_uint(p) : __float_as_uint(12.0f)) + (second ? __float_as_uint(q) : __float_as_uint(12.0f));
        parts(y, p, q);
        b += __float_as_uint(p) + __float_as_uint(q);
        mb += (first ? __float_as_uint(p) : __float_as_uint(0x1.8p-17f)) + (second ? __float_as_uint(q) : __float_as_uint(0x1.8p-17f));
    }
    __device__ __forceinline__ u64 total(int n) const { return WeightSum{a, b}.total(n); }
    __device__ __forceinline__ u64 total_marked(int n) const { return WeightSum{ma, mb}.total(n); }
};

__device__ __forceinline__ u64 weight(float t)
{
    WeightSum s;
    s.add(t);
    return s.total(1);
}

// floor(f Z), for a binary32 f in [0, 1), exactly; *whole: whether f Z is a whole number.
__device__ __forceinline__ u64 part_of(float f, u64 Z, bool *whole)
{
    const unsigned bits = __float_as_uint(f), exponent = bits >> 23;
    const unsigned m = (bits & 0x7FFFFFu) | (exponent ? 0x800000u : 0u);
    const int shift = 150 - static_cast<int>(exponent ? exponent : 1u);  // f = m 2^-shift, shift >= 24
    const u64 lo = m * Z, hi = __umul64hi(m, Z);
    if (shift < 64) {
        *whole = (lo << (64 - shift)) == 0;
        return (hi << (64 - shift)) | (lo >> shift);
    }
    if (shift == 64 || shift >= 128) {
        *whole = lo == 0 && (shift == 64 || hi == 0);
        return shift == 64 ? hi : 0;
    }
    *whole = lo == 0 && (hi << (128 - shift)) == 0;
    return hi >> (shift - 64);
}

// The least weight a top-p set has to reach: ceil(P Z).
__device__ __forceinline__ u64 share_of(float p, u64 Z)
{
    bool whole;
    const u64 f = part_of(fmaxf(p, 1e-6f), Z, &whole);
    return f + (whole ? 0 : 1);
}

// Z 2^-40 as binary32, rounded once (what the shift drops stays behind as a sticky bit).
__device__ __forceinline__ float as_sum(u64 Z)
{
    const int s = max(32 - __clzll(static_cast<long long>(Z)), 0);  // drop so many bits
    const unsigned top = static_cast<unsigned>(Z >> s) | ((Z & ((1ull << s) - 1)) != 0 ? 1u : 0u);
    return __fmul_rn(__uint2float_rn(top), __uint_as_float(static_cast<unsigned>(127 + s - 40) << 23));
}

// 2^40 / Z as binary32, to half a unit: a reciprocal and one correction by what it leaves of Z.
__device__ __forceinline__ float inverse_sum(u64 Z)
{
    const float z = as_sum(Z);
    const float rest = __ll2float_rn(static_cast<long long>(Z - __float2ull_rn(z * 0x1p+40f))) * 0x1p-40f;
    const float r = __frcp_rn(z);
    return __fmaf_rn(r, __fmaf_rn(-r, rest, __fmaf_rn(-r, z, 1.0f)), r);
}

// d - ln(Z 2^-40): Z 2^-40 = 2^k f, f in [sqrt(1/2), sqrt(2)); k ln 2 in two parts, the first with
// so few bits that its product with k is exact.
__device__ __forceinline__ float log_prob(float d, u64 Z)
{
    float f = as_sum(Z);
    int k = static_cast<int>(__float_as_uint(f) >> 23) - 127;
    f = __uint_as_float(__float_as_uint(f) - (static_cast<unsigned>(k) << 23));
    if (f > 0x1.6a09e6p+0f) {
        f *= 0.5f;
        k += 1;
    }
    const float kf = static_cast<float>(k);
    const float hi = kf * 0x1.62ep-1f, lo = __fmaf_rn(kf, 0x1.0bfbe8p-15f, sv::log_f32(f));
    const float a = __fsub_rn(d, hi), b = __fsub_rn(a, d);           // a + e = d - hi
    const float e = __fsub_rn(__fsub_rn(d, __fsub_rn(a, b)), __fadd_rn(hi, b));
    return __fadd_rn(a, __fsub_rn(e, lo));
}

}  // namespace sv_rows
