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

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <mutex>
#include <type_traits>

#include "spec_verify.h"
#include "sv_rows.cuh"

namespace {

using namespace sv_rows;

// The kernels, for two block sizes.
namespace b256 {
#define SV_ROWS_THREADS 256
#include "sv_rows_block.cuh"
#undef SV_ROWS_THREADS
}  // namespace b256
namespace b512 {
#define SV_ROWS_THREADS 512
#include "sv_rows_block.cuh"
#undef SV_ROWS_THREADS
}  // namespace b512

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

// How a launch splits its rows: CTAs per row, vectors of 16 bytes per CTA and per warp. As many CTAs
// for a row as the device holds at once (1024 threads on each of its 152 SMs) over the rows, in powers of
// two, and at least a vector for each of their threads. Where one CTA is a row's share and top-p may
// keep more than the list (`wide`), yet two: one wide row then decides how long the call takes
// (256 rows of 151936 bf16 logits, one in seven wide, 74 against 127 us; none wide 38 against 24).
struct Shape {
    int cluster;
    Split split;
};

Shape shape_of(int rows, int V, int elem_bytes, int threads, bool wide)
{
    const int vectors = V / (16 / elem_bytes) + 2;  // (a row may start and end within one)
    int c = 1;
    while (c < kMaxCluster && 2ll * rows * c <= 152 * (1024 / threads) && vectors >= 2 * c * threads) c *= 2;
    if (wide && c == 1 && rows <= 2 * 152 && vectors >= 4 * threads) c = 2;
    Shape s;
    s.cluster = c;
    const int warps = threads / 32;
    s.split.per_warp = ((vectors + c - 1) / c + warps - 1) / warps;
    s.split.per_cta = s.split.per_warp * warps;
    return s;
}

// Sampling by blocks of 512 threads, two on an SM, or, with more rows than four blocks on every SM,
// of 256: four rows in work on an SM hide one another's waits better than two (1024 rows of 151936
// bf16 logits with top-k and top-p 80 against 93 us, of 32000 35 against 45), while up to that a row's
// own time counts, which is shorter with more threads (256 rows 25 against 30 us; where a top-p set is
// wide, 512 rows of 129280 float32 logits, 170 against 254).
// The smaller number of rows, where the device does not hold them at once, starts with those that may
// take long if it may be of both kinds, which top-k and top-p given together say: the look at all rows'
// limits costs a CTA 1.5 us (256 mixed rows of 151936 bf16 logits 74 against 89 us, all with top-k and
// top-p 38.5 against 37).
constexpr int kManyRows = 4 * 152;

#ifdef SV_DEBUG_BOUNDS
// The arrays of one call, registered in g_spans (in stream order) before its launch. The environment
// variable SV_DEBUG_SHRINK leaves that many bytes of the end of every row of the first (the logits) out, so
// that tests can check that the check fires on memory that is there.
struct SpanList {
    Spans l{};
    void add(const void *p, bool out, size_t bytes, size_t rows = 1, size_t stride = 1)
    {
        if (p && bytes && rows && l.n < kSpans) l.s[l.n++] = Span{reinterpret_cast<u64>(p), stride, bytes, rows, out};
    }
    int push(cudaStream_t stream)
    {
        if (const char *e = getenv("SV_DEBUG_SHRINK")) l.s[0].bytes -= std::min<u64>(strtoull(e, nullptr, 10), l.s[0].bytes);
        return cudaMemcpyToSymbolAsync(g_spans, &l, sizeof(l), 0, cudaMemcpyHostToDevice, stream) == cudaSuccess ? SV_OK : SV_ECUDA;
    }
};

int push_spans(const spec_verify_sample_args &a, cudaStream_t stream)
{
    const size_t R = static_cast<size_t>(a.num_rows), V = static_cast<size_t>(a.vocab_size), e = a.logits_dtype == SV_BF16 ? 2 : 4;
    SpanList s;
    s.add(a.logits, false, V * e, R, static_cast<size_t>(a.logits_stride) * e);
    for (const void *p : {static_cast<const void *>(a.temperature), static_cast<const void *>(a.top_k), static_cast<const void *>(a.top_p),
                          static_cast<const void *>(a.min_p), static_cast<const void *>(a.uniforms)})
        s.add(p, false, R * 4);
    s.add(a.tokens, true, R * 4);
    s.add(a.token_logprob, true, R * 4);
    s.add(a.probs, true, V * 4, R, static_cast<size_t>(a.probs_stride) * 4);
    return s.push(stream);
}

int push_spans(const spec_verify_logprobs_args &a, cudaStream_t stream)
{
    const size_t R = static_cast<size_t>(a.num_rows), V = static_cast<size_t>(a.vocab_size), e = a.logits_dtype == SV_BF16 ? 2 : 4;
    const size_t n = static_cast<size_t>(a.num_reqs), top = static_cast<size_t>(a.num_top);
    SpanList s;
    s.add(a.logits, false, V * e, R, static_cast<size_t>(a.logits_stride) * e);
    s.add(a.temperature, false, R * 4);
    s.add(a.tokens, false, a.cu_num_draft ? n * static_cast<size_t>(a.token_stride) * 4 : R * 4);
    s.add(a.cu_num_draft, false, (n + 1) * 4);
    s.add(a.token_logprob, true, R * 4);
    s.add(a.token_rank, true, R * 4);
    s.add(a.top_ids, true, R * top * 4);
    s.add(a.top_logprobs, true, R * top * 4);
    return s.push(stream);
}
#endif

template <typename T, typename Params>
int launch(void (*kernel)(const T *, Params), const void *logits, Params P, int rows, int threads, bool wide, size_t room,
           cudaStream_t stream)
{
    const Shape s = shape_of(rows, P.V, sizeof(T), threads, wide);
    P.cluster = s.cluster;
    P.split = s.split;
    if constexpr (std::is_same_v<Params, SampleParams>)
        P.ordered = P.top_p && P.top_k && threads == 512 && rows <= 2 * threads && rows * s.cluster > 152 * (1024 / threads) ? rows : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows) * static_cast<unsigned>(s.cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = room;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(s.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<const T *>(logits), P) == cudaSuccess) return SV_OK;
    cudaGetLastError();
    return SV_ECUDA;
}

template <typename T>
int launch_sample(const void *logits, const SampleParams &P, int rows, cudaStream_t stream)
{
    return rows > kManyRows ? launch(b256::sv_sample_kernel<T>, logits, P, rows, 256, false, b256::Room::bytes, stream)
                            : launch(b512::sv_sample_kernel<T>, logits, P, rows, 512, P.top_p != nullptr, b512::Room::bytes, stream);
}

template <typename T>
int launch_logprobs(const void *logits, const LogprobParams &P, int rows, cudaStream_t stream)
{
    return P.num_top > 0
               ? launch(b256::sv_logprobs_kernel<T, true>, logits, P, rows, 256, false, b256::Room::bytes, stream)
               : launch(b256::sv_logprobs_kernel<T, false>, logits, P, rows, 256, false, 0, stream);
}

bool misaligned(const void *p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// Whether the memory from the first row's start to the last one's end is shared by two matrices of
// `rows` rows of V elements (of a and b bytes; strides in elements).
bool spans_meet(const void *p, int64_t p_stride, unsigned a, const void *q, int64_t q_stride, unsigned b, int rows, int V)
{
    using wide = unsigned __int128;
    const wide p0 = reinterpret_cast<uintptr_t>(p), q0 = reinterpret_cast<uintptr_t>(q);
    const wide p1 = p0 + (static_cast<wide>(rows - 1) * static_cast<wide>(p_stride) + static_cast<wide>(V)) * a;
    const wide q1 = q0 + (static_cast<wide>(rows - 1) * static_cast<wide>(q_stride) + static_cast<wide>(V)) * b;
    return p0 < q1 && q0 < p1;
}

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
    // (the distributions are set to 0 before the logits are read a second time)
    if (a->probs && spans_meet(a->logits, a->logits_stride, a->logits_dtype == SV_BF16 ? 2 : 4, a->probs, a->probs_stride, 4,
                               a->num_rows, a->vocab_size))
        return SV_EINVAL;
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
#ifdef SV_DEBUG_BOUNDS
    if (push_spans(*a, stream) != SV_OK) return SV_ECUDA;
#endif
    return a->logits_dtype == SV_BF16 ? launch_sample<uint16_t>(a->logits, P, a->num_rows, stream)
                                      : launch_sample<float>(a->logits, P, a->num_rows, stream);
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
#ifdef SV_DEBUG_BOUNDS
    if (push_spans(*a, stream) != SV_OK) return SV_ECUDA;
#endif
    return a->logits_dtype == SV_BF16 ? launch_logprobs<uint16_t>(a->logits, P, a->num_rows, stream)
                                      : launch_logprobs<float>(a->logits, P, a->num_rows, stream);
}

#ifdef SV_DEBUG_BOUNDS
// Of the checked build only: SV_ERR_BOUNDS in *word if a kernel of a row operator that has ended tried an
// access outside its call's arrays (the current device's; read and cleared).
extern "C" int spec_verify_rows_outside(uint32_t *word)
{
    const unsigned zero = 0;
    if (!word) return SV_EINVAL;
    return cudaMemcpyFromSymbol(word, g_outside, sizeof(*word)) == cudaSuccess &&
                   cudaMemcpyToSymbol(g_outside, &zero, sizeof(zero)) == cudaSuccess
               ? SV_OK
               : SV_ECUDA;
}
#endif
