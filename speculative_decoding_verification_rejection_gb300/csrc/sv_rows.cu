// Row operators of the sampler (spec_verify_sample, spec_verify_logprobs of
// include/spec_verify.h): one token drawn from each row of logits by a given uniform number under
// temperature, top-k, top-p and min-p, with its log-probability and, on request, the distribution
// it was drawn from; and log-probabilities, ranks and best tokens of rows.
//
// Mathematics. With L = max l_v, d_v = (l_v - L) / T and t_v = exp(d_v) (the library's fixed
// binary32 exp), every token gets the whole-number weight W_v = rint(t_v 2^40). Sums of weights
// are 64-bit whole numbers, so they do not depend on the order in which threads add, and every
// decision that hangs on a sum (where the top-p set ends, which token a uniform number falls on)
// is the same bit for bit however a row is split. 2^-40 is a hundred thousand times finer than
// the 2^-24 steps of a binary32 uniform number; a token below half of it, relative to the row's
// most likely one, has weight 0 and is not drawn.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cfloat>
#include <climits>
#include <cstdint>
#include <mutex>

#include "spec_verify.h"
#include "sv_device.cuh"

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr float kInf = __builtin_huge_valf();
constexpr unsigned long long kOne = 1ull << 40;  // the weight of a row's largest logit

using u64 = unsigned long long;

__device__ __forceinline__ float elem(const float *p, long long k) { return __ldg(p + k); }
__device__ __forceinline__ float elem(const uint16_t *p, long long k)
{
    return __uint_as_float(static_cast<uint32_t>(__ldg(p + k)) << 16);
}

// Logits as order-preserving unsigned integers, 0 for what is never kept (NaN and -inf); -0 as +0.
__device__ __forceinline__ unsigned key_of(float l)
{
    if (!(l > -kInf)) return 0u;
    const unsigned b = __float_as_uint(__fadd_rn(l, 0.0f));
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// 1 / T as a normal number: an infinite T then gives a difference that overflowed a d of -inf, not
// of 0 times infinity, and a tiny T a finite factor for the differences that are 0.
__device__ __forceinline__ float inverse(float T) { return fminf(fmaxf(__frcp_rn(T), FLT_MIN), FLT_MAX); }

// d of a logit that is not NaN or -inf: 0 at the maximum (also where that is infinite).
__device__ __forceinline__ float delta(float l, float L, float inv)
{
    return l == L ? 0.0f : __fmul_rn(__fsub_rn(l, L), inv);
}

__device__ __forceinline__ u64 weight(float t) { return static_cast<u64>(__float2ll_rn(t * 0x1p+40f)); }

// ---------------------------------------------------------------------------------------
// block reductions (every thread calls them; `box` is shared memory for one value per warp + 1)
// ---------------------------------------------------------------------------------------
template <typename V, typename F>
__device__ V block_reduce(V v, V *box, F join)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int s = 16; s; s >>= 1) v = join(v, __shfl_xor_sync(0xFFFFFFFFu, v, s));
    __syncthreads();
    if (lane == 0) box[warp] = v;
    __syncthreads();
    v = box[0];
    for (int w = 1; w < kWarps; ++w) v = join(v, box[w]);
    return v;
}

template <typename V>
__device__ V block_sum(V v, V *box)
{
    return block_reduce(v, box, [](V a, V b) { return a + b; });
}

// Exclusive prefix sum over the block's threads; *all: the total.
__device__ u64 block_scan(u64 v, u64 *box, u64 *all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 s = v;
    for (int k = 1; k < 32; k <<= 1) {
        const u64 o = __shfl_up_sync(0xFFFFFFFFu, s, k);
        if (lane >= k) s += o;
    }
    __syncthreads();
    if (lane == 31) box[warp] = s;
    __syncthreads();
    u64 before = 0, total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += box[w];
        total += box[w];
    }
    *all = total;
    return before + s - v;
}

struct SampleParams {
    long long stride, probs_stride;
    const float *temperature, *top_p, *min_p, *uniforms;
    const int32_t *top_k;
    int32_t *tokens;
    float *logprob, *probs;
    int V;
};

struct Shared {
    u64 box[kWarps + 1];
    u64 bin[256];
    unsigned cnt[256];
    int token;
    unsigned digit;
    u64 rest;
    float d;
};

// The largest key such that the keys at least as large hold `need` tokens (kMass false) or the
// weight `need` (compared in binary64), among keys >= floor: four passes of eight bits.
template <typename T, bool kMass>
__device__ unsigned select_key(const T *row, int V, float L, float inv, unsigned floor, double need, Shared &sh)
{
    const int tid = threadIdx.x;
    unsigned prefix = 0;
    u64 above = 0;  // held by the keys above the current prefix's interval
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        if (tid < 256) sh.bin[tid] = 0;
        __syncthreads();
        for (int v = tid; v < V; v += kThreads) {
            const float l = elem(row, v);
            const unsigned key = key_of(l);
            if (key == 0 || key < floor || (shift < 24 && (key >> (shift + 8)) != prefix)) continue;
            const u64 w = kMass ? weight(sv::exp_f32(delta(l, L, inv))) : 1ull;
            if (w) atomicAdd(&sh.bin[(key >> shift) & 255u], w);
        }
        __syncthreads();
        if (tid == 0) {
            u64 s = above;
            int b = 255;
            for (; b > 0; --b) {
                if (static_cast<double>(s + sh.bin[b]) >= need) break;
                s += sh.bin[b];
            }
            sh.digit = static_cast<unsigned>(b);
            sh.rest = s;
        }
        __syncthreads();
        prefix = (prefix << 8) | sh.digit;
        above = sh.rest;
    }
    return prefix;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sv_sample_kernel(const T *logits, SampleParams P)
{
    __shared__ Shared sh;
    const int tid = threadIdx.x, V = P.V;
    const long long r = blockIdx.x;
    const T *row = logits + r * P.stride;
    float *probs = P.probs ? P.probs + r * P.probs_stride : nullptr;
    const float temp = P.temperature ? __ldg(P.temperature + r) : 1.0f;
    const int k = P.top_k ? __ldg(P.top_k + r) : 0;
    const float p = P.top_p ? __ldg(P.top_p + r) : 1.0f;
    const float m = P.min_p ? __ldg(P.min_p + r) : 0.0f;
    const bool greedy = !(temp > 0.0f) || k == 1;
    const float inv = greedy ? 1.0f : inverse(temp);

    // the largest logit and where it first stands
    float L = -kInf;
    for (int v = tid; v < V; v += kThreads) L = fmaxf(L, elem(row, v));
    L = block_reduce(L, reinterpret_cast<float *>(sh.box), [](float a, float b) { return fmaxf(a, b); });
    if (!(L > -kInf)) {  // nothing to keep
        if (tid == 0) {
            P.tokens[r] = -1;
            if (P.logprob) P.logprob[r] = -kInf;
        }
        if (probs)
            for (int v = tid; v < V; v += kThreads) probs[v] = 0.0f;
        return;
    }
    if (greedy) {
        int best = INT_MAX;
        for (int v = tid; v < V; v += kThreads)
            if (elem(row, v) == L) best = min(best, v);
        best = block_reduce(best, reinterpret_cast<int *>(sh.box), [](int a, int b) { return min(a, b); });
        if (tid == 0) {
            P.tokens[r] = best;
            if (P.logprob) P.logprob[r] = 0.0f;
        }
        if (probs)
            for (int v = tid; v < V; v += kThreads) probs[v] = v == best ? 1.0f : 0.0f;
        return;
    }
    unsigned floor = 1;
    if (k >= 1 && k < V) {
        int valid = 0;
        for (int v = tid; v < V; v += kThreads) valid += key_of(elem(row, v)) != 0;
        valid = block_sum(valid, reinterpret_cast<int *>(sh.box));
        if (k < valid) floor = select_key<T, false>(row, V, L, inv, 1, k, sh);
    }
    if (p < 1.0f) {
        u64 z = 0;
        for (int v = tid; v < V; v += kThreads) {
            const float l = elem(row, v);
            if (key_of(l) >= floor) z += weight(sv::exp_f32(delta(l, L, inv)));
        }
        z = block_sum(z, sh.box);
        const double need = static_cast<double>(fmaxf(p, 1e-6f)) * static_cast<double>(z);
        floor = max(floor, select_key<T, true>(row, V, L, inv, floor, need, sh));
    }
    const float low = m > 0.0f ? __double2float_rn(log(static_cast<double>(fminf(m, 1.0f)))) : -kInf;

    auto kept = [&](int v, float &d) -> float {
        const float l = elem(row, v);
        if (key_of(l) < floor) return 0.0f;
        d = delta(l, L, inv);
        return d >= low ? sv::exp_f32(d) : 0.0f;
    };
    float d = 0.0f;
    u64 Z = 0;
    for (int v = tid; v < V; v += kThreads) Z += weight(kept(v, d));
    Z = block_sum(Z, sh.box);
    const float u = __ldg(P.uniforms + r);
    const double target = static_cast<double>(u > 0.0f ? u : 0.0f) * static_cast<double>(Z);
    if (tid == 0) sh.token = -1;
    u64 base = 0;
    for (int v0 = 0; v0 < V; v0 += kThreads) {
        const int v = v0 + tid;
        float dv = 0.0f;
        const u64 w = v < V ? weight(kept(v, dv)) : 0;
        u64 all;
        const u64 upto = base + block_scan(w, sh.box, &all) + w;
        const bool hit = w && (static_cast<double>(upto) > target || upto == Z) &&
                         !(static_cast<double>(upto - w) > target);
        if (hit) {
            sh.token = v;
            sh.d = dv;
        }
        base += all;
        __syncthreads();
        if (sh.token >= 0) break;
    }
    if (tid == 0) {
        P.tokens[r] = sh.token;
        if (P.logprob)
            P.logprob[r] = static_cast<float>(static_cast<double>(sh.d) - log(static_cast<double>(Z) * 0x1p-40));
    }
    if (probs) {
        const float z = static_cast<float>(static_cast<double>(Z) * 0x1p-40);
        for (int v = tid; v < V; v += kThreads) probs[v] = __fdiv_rn(kept(v, d), z);
    }
}

struct LogprobParams {
    long long stride;
    const float *temperature;
    const int32_t *tokens, *cu;
    int token_stride, num_reqs, num_top, V;
    float *logprob, *top_logprob;
    int32_t *rank, *top_ids;
};

// The token wanted of row r: tokens[r], or with prefix sums of the draft lengths the entry of the
// verification output [num_reqs, token_stride] that row r is the logits of (row cu[i] + i + j is
// position j of request i). The search stays in [0, num_reqs) whatever cu holds.
__device__ int row_token(const LogprobParams &P, long long r)
{
    if (!P.cu) return __ldg(P.tokens + r);
    int lo = 0, hi = P.num_reqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<long long>(__ldg(P.cu + mid)) + mid <= r) lo = mid;
        else hi = mid;
    }
    const long long j = r - __ldg(P.cu + lo) - lo;
    return j >= 0 && j < P.token_stride ? __ldg(P.tokens + static_cast<long long>(lo) * P.token_stride + j) : -1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sv_logprobs_kernel(const T *logits, LogprobParams P)
{
    __shared__ Shared sh;
    const int tid = threadIdx.x, V = P.V, n = P.num_top;
    const long long r = blockIdx.x;
    const T *row = logits + r * P.stride;
    const int token = P.tokens ? row_token(P, r) : 0;
    int32_t *ids = n ? P.top_ids + r * n : nullptr;
    float *best = n ? P.top_logprob + r * n : nullptr;
    float L = -kInf;
    const bool wanted = token >= 0 && token < V;
    if (wanted)
        for (int v = tid; v < V; v += kThreads) L = fmaxf(L, elem(row, v));
    L = block_reduce(L, reinterpret_cast<float *>(sh.box), [](float a, float b) { return fmaxf(a, b); });
    if (!(L > -kInf)) {
        if (tid == 0 && P.logprob) P.logprob[r] = -kInf;
        if (tid == 0 && P.rank) P.rank[r] = wanted ? 1 : 0;
        for (int i = tid; i < n; i += kThreads) {
            ids[i] = -1;
            best[i] = -kInf;
        }
        return;
    }
    const float temp = P.temperature ? __ldg(P.temperature + r) : 1.0f;
    const float inv = temp > 0.0f ? inverse(temp) : 1.0f;
    const float lt = fmaxf(elem(row, token), -kInf);  // (NaN as -inf)
    double s = 0.0;
    int rank = 0;
    for (int v = tid; v < V; v += kThreads) {
        const float l = elem(row, v);
        if (l > -kInf) s += sv::exp_f32(delta(l, L, inv));
        rank += l > lt;
    }
    s = block_sum(s, reinterpret_cast<double *>(sh.box));
    rank = block_sum(rank, reinterpret_cast<int *>(sh.box));
    const double norm = log(s);
    if (tid == 0) {
        if (P.logprob)
            P.logprob[r] = lt > -kInf ? static_cast<float>(static_cast<double>(delta(lt, L, inv)) - norm) : -kInf;
        if (P.rank) P.rank[r] = rank + 1;
    }
    u64 last = ~0ull;  // (key, ~index) of the previous best
    for (int i = 0; i < n; ++i) {
        u64 b = 0;
        for (int v = tid; v < V; v += kThreads) {
            const unsigned key = key_of(elem(row, v));
            const u64 c = (static_cast<u64>(key) << 32) | static_cast<unsigned>(~v);
            if (key && c < last && c > b) b = c;
        }
        b = block_reduce(b, sh.box, [](u64 x, u64 y) { return x > y ? x : y; });
        last = b;
        if (tid == 0) {
            const int v = static_cast<int>(~static_cast<unsigned>(b));
            ids[i] = b ? v : -1;
            best[i] = b ? static_cast<float>(static_cast<double>(delta(elem(row, v), L, inv)) - norm) : -kInf;
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

constexpr int kMaxDevices = 64;
std::mutex g_rows_mutex;
bool g_rows_ready[kMaxDevices];

// Whether `dev` is a device the kernels run on; looked up once per device.
int rows_device(int dev)
{
    if (dev < 0 || dev >= kMaxDevices) return SV_EDEVICE;
    std::lock_guard<std::mutex> lock(g_rows_mutex);
    if (g_rows_ready[dev]) return SV_OK;
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
        cudaGetLastError();
        return SV_EDEVICE;
    }
    if (major != 10 || minor != 3) return SV_EDEVICE;  // built for sm_103a only
    g_rows_ready[dev] = true;
    return SV_OK;
}

bool misaligned(const void *p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// What both entry points ask of the rows themselves.
int check_rows(const void *logits, int64_t stride, int dtype, int num_rows, int vocab)
{
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_EDTYPE;
    if (num_rows < 0 || vocab <= 0) return SV_EINVAL;
    if (vocab > SV_ROWS_MAX_VOCAB) return SV_ECAPACITY;
    if (num_rows > 0 && (!logits || misaligned(logits, dtype == SV_BF16 ? 2 : 4) || stride < vocab)) return SV_EINVAL;
    return SV_OK;
}

}  // namespace

extern "C" int spec_verify_sample(const spec_verify_sample_args *a, void *cuda_stream)
{
    const NvtxRange nvtx("spec_verify_sample");
    if (!a) return SV_EINVAL;
    const int rc = check_rows(a->logits, a->logits_stride, a->logits_dtype, a->num_rows, a->vocab_size);
    if (rc != SV_OK || a->num_rows == 0) return rc;
    if (!a->uniforms || !a->tokens || (a->probs && a->probs_stride < a->vocab_size)) return SV_EINVAL;
    for (const void *p : {static_cast<const void *>(a->temperature), static_cast<const void *>(a->top_k),
                          static_cast<const void *>(a->top_p), static_cast<const void *>(a->min_p),
                          static_cast<const void *>(a->uniforms), static_cast<const void *>(a->tokens),
                          static_cast<const void *>(a->token_logprob), static_cast<const void *>(a->probs)})
        if (misaligned(p, 4)) return SV_EINVAL;
    const int rd = rows_device(a->device);
    if (rd != SV_OK) return rd;
    const DeviceGuard guard(a->device);
    if (!guard.ok) return SV_EDEVICE;
    SampleParams P;
    P.stride = a->logits_stride;
    P.probs_stride = a->probs_stride;
    P.temperature = a->temperature;
    P.top_k = a->top_k;
    P.top_p = a->top_p;
    P.min_p = a->min_p;
    P.uniforms = a->uniforms;
    P.tokens = a->tokens;
    P.logprob = a->token_logprob;
    P.probs = a->probs;
    P.V = a->vocab_size;
    const auto stream = static_cast<cudaStream_t>(cuda_stream);
    const auto grid = static_cast<unsigned>(a->num_rows);
    if (a->logits_dtype == SV_BF16)
        sv_sample_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(static_cast<const uint16_t *>(a->logits), P);
    else
        sv_sample_kernel<float><<<grid, kThreads, 0, stream>>>(static_cast<const float *>(a->logits), P);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ECUDA;
}

extern "C" int spec_verify_logprobs(const spec_verify_logprobs_args *a, void *cuda_stream)
{
    const NvtxRange nvtx("spec_verify_logprobs");
    if (!a) return SV_EINVAL;
    const int rc = check_rows(a->logits, a->logits_stride, a->logits_dtype, a->num_rows, a->vocab_size);
    if (rc != SV_OK || a->num_rows == 0) return rc;
    if (a->num_top < 0 || (a->num_top > 0 && (!a->top_ids || !a->top_logprobs))) return SV_EINVAL;
    if (a->num_top > SV_MAX_TOP) return SV_ECAPACITY;
    if (!a->tokens && (a->token_logprob || a->token_rank || a->cu_num_draft || a->num_top == 0)) return SV_EINVAL;
    if (a->cu_num_draft && (a->num_reqs < 1 || a->token_stride < 1)) return SV_EINVAL;
    for (const void *p : {static_cast<const void *>(a->temperature), static_cast<const void *>(a->tokens),
                          static_cast<const void *>(a->cu_num_draft), static_cast<const void *>(a->token_logprob),
                          static_cast<const void *>(a->token_rank), static_cast<const void *>(a->top_ids),
                          static_cast<const void *>(a->top_logprobs)})
        if (misaligned(p, 4)) return SV_EINVAL;
    const int rd = rows_device(a->device);
    if (rd != SV_OK) return rd;
    const DeviceGuard guard(a->device);
    if (!guard.ok) return SV_EDEVICE;
    LogprobParams P;
    P.stride = a->logits_stride;
    P.temperature = a->temperature;
    P.tokens = a->tokens;
    P.cu = a->cu_num_draft;
    P.token_stride = a->token_stride;
    P.num_reqs = a->num_reqs;
    P.num_top = a->num_top;
    P.V = a->vocab_size;
    P.logprob = a->token_logprob;
    P.rank = a->token_rank;
    P.top_ids = a->top_ids;
    P.top_logprob = a->top_logprobs;
    const auto stream = static_cast<cudaStream_t>(cuda_stream);
    const auto grid = static_cast<unsigned>(a->num_rows);
    if (a->logits_dtype == SV_BF16)
        sv_logprobs_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(static_cast<const uint16_t *>(a->logits), P);
    else
        sv_logprobs_kernel<float><<<grid, kThreads, 0, stream>>>(static_cast<const float *>(a->logits), P);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ECUDA;
}
