// Kernels of the row operators for blocks of SV_ROWS_THREADS threads; included once for each size,
// in a namespace of its own (so without a guard). See sv_rows.cu for the mathematics.
constexpr int kThreads = SV_ROWS_THREADS;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = kBins / kThreads;  // groups of a lane's vectors whose maxima are kept
constexpr int kCtas = 1024 / kThreads;     // CTAs on an SM: 64 registers for each thread
constexpr bool kOrdered = kThreads == 512;  // whether rows may be put in order (the smaller blocks take too many)

// ---------------------------------------------------------------------------------------
// warp and block reductions (block-wide ones by every thread)
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ u64 warp_sum(u64 v)
{
#pragma unroll
    for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
    return v;
}
__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int s = 16; s; s >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, s));
    return v;
}

// Exclusive prefix sum over the block's threads; *all: the total.
__device__ u64 block_scan(u64 v, u64 *box, u64 *all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 s = v;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const u64 o = __shfl_up_sync(0xFFFFFFFFu, s, k);
        if (lane >= k) s += o;
    }
    __syncthreads();
    if (lane == 31) box[warp] = s;
    __syncthreads();
    u64 before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += box[w];
        total += box[w];
    }
    *all = total;
    return before + s - v;
}

// The same for a float and a whole number, totals in *all and *count (`box` takes both).
__device__ __forceinline__ void block_scan(float &v, unsigned &c, u64 *box, float *all, unsigned *count)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float s = v;
    unsigned t = c;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const float o = __shfl_up_sync(0xFFFFFFFFu, s, k);
        const unsigned p = __shfl_up_sync(0xFFFFFFFFu, t, k);
        if (lane >= k) {
            s += o;
            t += p;
        }
    }
    __syncthreads();
    if (lane == 31) box[warp] = (static_cast<u64>(t) << 32) | __float_as_uint(s);
    __syncthreads();
    float before = 0.0f, total = 0.0f;
    unsigned fewer = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const u64 x = box[w];
        if (w < warp) {
            before += __uint_as_float(static_cast<unsigned>(x));
            fewer += static_cast<unsigned>(x >> 32);
        }
        total += __uint_as_float(static_cast<unsigned>(x));
        sum += static_cast<unsigned>(x >> 32);
    }
    *all = total;
    *count = sum;
    v = before + s - v;
    c = fewer + t - c;
}

// ---------------------------------------------------------------------------------------
// a row over a cluster
// ---------------------------------------------------------------------------------------
// The 16-byte vectors that hold the row are split evenly over the cluster's CTAs and then over
// their warps, both in contiguous runs, so that the warps in order hold the row in index order; a
// lane has the vectors lane, lane + 32, ... of its warp's run. Every pass reads them from global
// memory: the first one from HBM, those after it from the L2 cache as far as that holds the rows in
// work (of 256 rows of 151936 bf16 logits, 78 MB, about a third of the reads hit it).
// (Rows copied to shared memory once were as fast where few are in work and slower where many
// are, since then the 227 KB of an SM bounds how many: 64 rows of 151936 bf16 logits 18 against 20 us,
// 1024 rows with top-k 157 against 108.) What of the first and last vector lies outside the row is
// -inf.
struct Shared {
    u64 box[kWarps];
    u64 seg[2][kMaxCluster * kWarps];  // a value of every warp of the cluster (two, used in turn)
    u64 runs[kMaxCluster * kWarps];    // kept weight of every warp's run
    u64 listed[kMaxCluster];           // the weight of every CTA's candidates
    unsigned count[kMaxCluster];       // their number
    float cut[kMaxCluster], peak[kMaxCluster];
    int small[kWarps];
    unsigned mine, hits, fits;
    float upper, lower, from, width;
    unsigned again;
    u64 below;
    u64 kept;
    int run;
    unsigned tau;
    int first, found;
    float d;
    uint4 edge[2];  // the row's first and last vector, if they are not wholly in it
};

// The parts of a CTA's dynamic shared memory.
struct Room {
    u64 *list;                // [kList] candidates; with `work` behind it, [kWideList]
    u64 *work;                // [kList] weights or sums
    float *peaks;             // [kGroups][kThreads] maxima of the lanes' groups; the histogram
    unsigned *hits;           // [kHits]
    static constexpr size_t bytes = 2 * kList * 8 + kGroups * kThreads * 4 + kHits * 4;
    explicit __device__ __forceinline__ Room(void *p)
        : list(static_cast<u64 *>(p)), work(list + kList), peaks(reinterpret_cast<float *>(work + kList)),
          hits(reinterpret_cast<unsigned *>(peaks + kGroups * kThreads)) {}
};
static_assert(kWideList == 2 * kList, "`work` lies behind `list`");

template <typename T>
struct Row {
    static constexpr int n = Vec<T>::n;
    using Elem = T;
    const uint4 *vec;     // this CTA's vectors
    const uint4 *edge;    // in place of the vectors `front` and `back`
    const T *row;
    int base;             // index in the row of its first vector's first element (may be negative)
    int lo, hi;           // this warp's vectors
    int front, back;      // -1 where there is none
    int mine, per_warp;   // vectors of this CTA, and of its warps but the last
    int V;
    int lane, warp;
    bool inf;             // read through only_inf()
    bool plain;           // this warp's run has neither of these vectors, and not inf

    __device__ __forceinline__ uint4 get(int j) const
    {
        uint4 v;
        if (j == front) v = edge[0];
        else if (j == back) v = edge[1];
        else v = ld_row(vec + j);
        return inf ? only_inf<T>(v) : v;
    }
    // Vectors j, j + 32, ... of this lane, k of them, those past the run's end all -inf. Returns how
    // many are not past the end for some lane of the warp.
    template <int k>
    __device__ __forceinline__ int load(int j, uint4 (&v)[k]) const
    {
#pragma unroll
        for (int i = 0; i < k; ++i) {  // the reads first, then the rare vectors that are something else
            const int a = j + 32 * i;
            v[i] = make_uint4(Low<T>::word, Low<T>::word, Low<T>::word, Low<T>::word);
            if (a < hi && a != front && a != back) v[i] = ld_row(vec + a);
        }
#pragma unroll
        for (int i = 0; i < k; ++i) {
            const int a = j + 32 * i;
            if (a < hi && (a == front || a == back)) v[i] = edge[a != front];
        }
        if (inf) {
#pragma unroll
            for (int i = 0; i < k; ++i) v[i] = only_inf<T>(v[i]);
        }
        return min((hi - (j - lane) + 31) / 32, k);
    }
    // Calls f(v, m, c) for this lane's vectors, k at a time: v[0, m) of the c-th time. With kTwice f is
    // there twice, once for the times when there is nothing to look at: for passes that compute more
    // than they wait for memory (a pass of exact sums 31 against 34 us with two rows of 151936 bf16
    // logits on an SM; in the first pass the registers it takes cost more, 68 against 76 us).
    template <int k, bool kTwice = false, typename F>
    __device__ __forceinline__ void each(F f) const
    {
        int c = 0, j = lo + lane;
        if (kTwice && plain)
            for (; j - lane + 32 * k <= hi; j += 32 * k, ++c) {
                uint4 v[k];
#pragma unroll
                for (int i = 0; i < k; ++i) v[i] = ld_row(vec + j + 32 * i);
                f(v, k, c);
            }
        for (; j - lane < hi; j += 32 * k, ++c) {
            uint4 v[k];
            const int m = load<k>(j, v);
            f(v, m, c);
        }
    }
    __device__ __forceinline__ float at(int i) const  // element i of the row; -inf outside
    {
        const float l = i >= 0 && i < V ? as_float(ld(row + i)) : -kInf;
        return !inf ? l : l == kInf ? 0.0f : -kInf;
    }
    __device__ __forceinline__ int first() const { return max(base, 0); }
    __device__ __forceinline__ int last() const { return min(base + mine * n, V); }
};

// This CTA's part of the row at `row`.
template <typename T>
__device__ __forceinline__ Row<T> start_row(const T *row, int V, const Split &sp, unsigned rank, Shared &sh)
{
    constexpr int n = Vec<T>::n;
    Row<T> R;
    R.lane = threadIdx.x & 31;
    R.warp = threadIdx.x >> 5;
    R.V = V;
    R.row = row;
    R.inf = false;
    const auto address = reinterpret_cast<uintptr_t>(row);
    const int off = static_cast<int>((address & 15u) / sizeof(T));
    const int vectors = (off + V + n - 1) / n;
    const int v0 = static_cast<int>(rank) * sp.per_cta;
    R.mine = max(min(sp.per_cta, vectors - v0), 0);
    R.per_warp = sp.per_warp;
    R.base = v0 * n - off;
    R.lo = min(R.warp * sp.per_warp, R.mine);
    R.hi = min(R.lo + sp.per_warp, R.mine);
    R.vec = reinterpret_cast<const uint4 *>(address & ~static_cast<uintptr_t>(15)) + v0;
    R.edge = sh.edge;
    R.front = off != 0 && rank == 0 ? 0 : -1;
    R.back = (off + V) % n != 0 && vectors - 1 - v0 < R.mine ? vectors - 1 - v0 : -1;
    R.plain = !(R.front >= R.lo && R.front < R.hi) && !(R.back >= R.lo && R.back < R.hi);
    if (off == 0 && (off + V) % n == 0) return R;
    if (threadIdx.x < 2 * n) {
        const int k = threadIdx.x / n, e = threadIdx.x % n, i = (k == 0 ? 0 : vectors - 1) * n - off + e;
        reinterpret_cast<T *>(&sh.edge[k])[e] = i >= 0 && i < V ? ld(row + i) : Low<T>::value();
    }
    __syncthreads();
    return R;
}

// Sum of 2^((l - ref) scale) over v[0, m), in binary32, no logit more than kRise / scale above ref; a NaN
// and -inf add nothing, and where ref is +inf each logit of +inf adds 1.
template <typename T, int k>
__device__ __forceinline__ float fast_sum(const uint4 (&v)[k], int m, float ref, float scale)
{
    constexpr int n = Vec<T>::n;
    Two sum = two(0.0f);
#pragma unroll
    for (int i = 0; i < k; ++i) {
        if (i >= m) continue;
        float f[n];
        Vec<T>::get(v[i], f);
#pragma unroll
        for (int e = 0; e < n; e += 2) {
            const Two x = (two(f[e], f[e + 1]) + two(-ref)) * two(scale);
            float a, b;
            parts(x, a, b);
            sum = sum + two(sv::ex2_approx(a), sv::ex2_approx(b));
        }
    }
    float a, b;
    parts(sum, a, b);
    a += b;
    if (a != a) {  // a NaN, or infinities on both sides of a difference
        a = 0.0f;
#pragma unroll
        for (int i = 0; i < k; ++i) {
            float f[n];
            Vec<T>::get(v[i], f);
            for (int e = 0; e < n; ++e)
                if (f[e] > -kInf) a += f[e] == ref ? 1.0f : sv::ex2_approx((f[e] - ref) * scale);
        }
    }
    return a;
}

// The largest of this lane's logits, and of each group of them (times c of kAhead vectors with the
// same c mod kGroups) into `peaks`; with kSum also *sum, the sum of 2^((l - largest) scale) over them.
template <bool kSum, typename T>
__device__ __forceinline__ float lane_max(const Row<T> &R, float *peaks, float scale, float *sum)
{
    float all = -kInf, s = 0.0f;
    R.template each<kAhead>([&](uint4 (&v)[kAhead], int n, int c) {
        Largest<T> m;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) m.add(v[i]);
        float *at = peaks + (c % kGroups) * kThreads + threadIdx.x;
        const float own = m.get(), ref = fmaxf(all, own);
        *at = c < kGroups ? own : fmaxf(*at, own);
        if (kSum) {
            if (ref > all && all > -kInf) s *= sv::ex2_approx((all - ref) * scale);
            s += fast_sum<T>(v, n, ref, scale);
        }
        all = ref;
    });
    if (kSum) *sum = s;
    return all;
}

// The largest of a value over the block.
__device__ __forceinline__ float block_max(float v, Shared &sh)
{
    v = warp_max(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) reinterpret_cast<float *>(sh.small)[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_max(reinterpret_cast<float *>(sh.small)[threadIdx.x & (kWarps - 1)]);
}

// A cut that at least `want` of this CTA's lane maxima reach and at most `most`, or what twenty halvings of the span of keys from the least to the largest of them give; the lowest
// finite number where there are not so many. The CTA's tokens at or above it hold its `want` largest, and are few more than that.
template <typename T>
__device__ float cut_for(float peak, float largest, int want, int most, Shared &sh)
{
    constexpr int drop = sizeof(T) == 2 ? 16 : 0;  // (of bf16 logits the upper half of the key says all)
    const unsigned key = key_of(peak) >> drop;
    int reach = __syncthreads_count(key != 0);
    if (reach < want) return -FLT_MAX;
    unsigned lo = key_of(-block_max(key ? -peak : -kInf, sh)) >> drop, hi = key_of(largest) >> drop;
    for (int i = 0; i < 20 && lo < hi && reach > most; ++i) {
        const unsigned mid = lo + (hi - lo) / 2 + 1;
        const int c = __syncthreads_count(key >= mid);
        if (c >= want) {
            lo = mid;
            reach = c;
        } else {
            hi = mid - 1;
        }
    }
    return of_key(lo << drop);
}

// ---------------------------------------------------------------------------------------
// sampling
// ---------------------------------------------------------------------------------------
// A lane's most vectors of a row: the largest vocabulary, by one CTA.
template <typename T>
constexpr int most_vectors()
{
    const int per_warp = (SV_ROWS_MAX_VOCAB / Vec<T>::n + 2 + kWarps - 1) / kWarps;
    return (per_warp + 31) / 32;
}
template <typename T>
constexpr int most_batches = (most_vectors<T>() + kAhead - 1) / kAhead;
static_assert(most_vectors<uint16_t>() * Vec<uint16_t>::n <= kMostWeights && most_vectors<float>() * Vec<float>::n <= kMostWeights,
              "a lane's weights go into one sum");
static_assert(SV_ROWS_MAX_VOCAB < 1 << 23, "a row's weights, 2^40 each at most, go into 64 bits");

// The row's weight by the lanes' sums is off by less than one part in kSure. In units of 2^-24, a rounding:
//   arguments  a term that is not 0 has a d of at most 29.2 (42 doublings). Its argument is a difference
//              times fl(fl(log2 e) / T): log2 e off by 0.25, two products and the difference, each
//              relative to the difference, also where the sum goes from one largest logit to another
//              (the differences then add up to that d); and the d that the weight is made from has two
//              roundings of its own: 29.2 * 5.25 < 154
//   moves      a lane's sum goes from one largest logit to another at most once a batch after the first,
//              and then to the row's: a 2^x of 4 and a product, 5 a batch
//   additions  at most 32 pairs in a batch, its halves, and one a batch
//   the rest   a term's 2^x 4, the weight's exp 2, its rounding to 2^-40 and the terms that are 0 there, over
//              a sum of at least 1, V 2^-41 each: 4 and 4, and the sum as a whole number 1: below 16
// (kRise is not in this: here the reference is the largest logit so far.)
constexpr u64 kSure = 1 << 14;
constexpr int kSumError = 154 + (5 + 1) * (most_batches<float> > most_batches<uint16_t> ? most_batches<float> : most_batches<uint16_t>) + 33 + 16;
static_assert(static_cast<u64>(kSumError) * kSure <= 1 << 24, "the row's weight is known to a part in kSure");

// What is kept, besides key_of(l) != 0: l >= tau and d >= low.
struct Kept {
    float L, inv, tau, low;
};

// The CTA's tokens at or above the cut, as (key, ~index), into its part of the list: the groups whose
// maximum reaches the cut are put down, and their vectors then read by all threads side by side, so
// that the wait for the cache is one and not one for each group. The CTA sends its part to the
// leader's list and its number, its weight (kMass) and, if it is this CTA's own, the cut to every CTA.
// Entries past the part's end are only counted, and groups past kHits make the part count as full.
template <bool kMass, typename T>
__device__ __forceinline__ void collect(const Row<T> &R, float cut, const Room &room, int part, unsigned rank, int cluster,
                                        const Kept &keep, bool tell_cut, Shared &sh)
{
    constexpr int n = Row<T>::n;
    const int tid = threadIdx.x;
    u64 *mine = room.list + rank * part;
    if (tid == 0) sh.mine = sh.hits = 0;
    __syncthreads();
    const int times = (R.hi - R.lo + 32 * kAhead - 1) / (32 * kAhead);
    for (int g = 0; g < min(times, kGroups); ++g)
        if (room.peaks[g * kThreads + tid] >= cut) {
            const unsigned at = atomicAdd(&sh.hits, 1u);
            if (at < kHits) room.hits[at] = static_cast<unsigned>(g * kThreads + tid);
        }
    __syncthreads();
    const int rounds = (R.per_warp + 32 * kAhead * kGroups - 1) / (32 * kAhead * kGroups);
    const int slots = rounds * kAhead, total = min(static_cast<int>(sh.hits), kHits) * slots;
    for (int i = tid; i < total; i += kThreads) {
        const int slot = i % slots;
        const auto hit = static_cast<int>(room.hits[i / slots]);
        const int owner = hit % kThreads, time = hit / kThreads + slot / kAhead * kGroups;
        const int lo = min((owner >> 5) * R.per_warp, R.mine), hi = min(lo + R.per_warp, R.mine);
        const int j = lo + (owner & 31) + 32 * (time * kAhead + slot % kAhead);
        if (j >= hi) continue;
        const uint4 v = R.get(j);
        Largest<T> m;
        m.add(v);
        if (m.get() >= cut) {
            float f[n];
            Vec<T>::get(v, f);
#pragma unroll
            for (int e = 0; e < n; ++e)
                if (f[e] >= cut) {
                    const unsigned at = atomicAdd(&sh.mine, 1u);
                    const auto index = static_cast<unsigned>(R.base + j * n + e);
                    if (at < static_cast<unsigned>(part))
                        mine[at] = (static_cast<u64>(key_of(f[e])) << 32) | static_cast<u64>(~index);
                }
        }
    }
    __syncthreads();
    const int count = sh.hits > kHits ? part + 1 : static_cast<int>(sh.mine);
    u64 w = 0;
    for (int i = tid; i < min(count, part); i += kThreads) {
        const u64 e = mine[i];
        if (kMass) w += weight(exp_weight(delta(of_key(static_cast<unsigned>(e >> 32)), keep.L, keep.inv)));
        if (rank != 0) put(remote(mine + i, 0), e);
    }
    if (kMass) {
        u64 all;
        block_scan(w, sh.box, &all);
        if (tid < cluster) put(remote(&sh.listed[rank], tid), all);
    }
    if (tid < cluster) {
        put(remote(&sh.count[rank], tid), static_cast<unsigned>(count));
        if (tell_cut) put(remote(&sh.cut[rank], tid), __float_as_uint(cut));
    }
}

// Whether every CTA's candidates found place; *total: their number.
__device__ __forceinline__ bool all_listed(const Shared &sh, int cluster, int part, int *total)
{
    bool fits = true;
    int n = 0;
    for (int c = 0; c < cluster; ++c) {
        fits &= sh.count[c] <= static_cast<unsigned>(part);
        n += static_cast<int>(sh.count[c]);
    }
    *total = n;
    return fits;
}

// Entry i of the leader's list, whose parts are filled from their beginnings; 0 past the end.
__device__ __forceinline__ u64 listed_entry(const u64 *list, int part, int cluster, const Shared &sh, int i)
{
    for (int c = 0; c < cluster; ++c) {
        const int n = static_cast<int>(sh.count[c]);
        if (i < n) return list[c * part + i];
        i -= n;
    }
    return 0;
}

// Bitonic sort of `size` (a power of two) entries, the largest first.
__device__ void sort_down(u64 *list, int size)
{
    for (int run = 2; run <= size; run *= 2)
        for (int step = run / 2; step > 0; step /= 2) {
            for (int p = threadIdx.x; p < size / 2; p += kThreads) {
                const int i = 2 * p - (p & (step - 1));
                const u64 a = list[i], b = list[i + step];
                if ((a < b) == ((i & run) == 0)) {
                    list[i] = b;
                    list[i + step] = a;
                }
            }
            __syncthreads();
        }
}

// Whether a running sum of weights has passed the uniform number's place in the total.
struct Target {
    u64 least;  // the least sum that is above u Z, or Z
    __device__ __forceinline__ Target(float u, u64 Z)
    {
        bool whole;
        least = u >= 1.0f ? Z : 1 + (u > 0.0f ? part_of(u, Z, &whole) : 0);
    }
    __device__ __forceinline__ bool passed(u64 c) const { return c >= least; }
};

// The d of a listed key: of the row's largest logit 0, also where that is +inf.
__device__ __forceinline__ float listed_delta(unsigned key, const Kept &keep)
{
    const float l = of_key(key);
    return l == keep.L ? 0.0f : delta(l, keep.L, keep.inv);
}

// What the leader leaves of a drawn or kept entry.
struct Drawn {
    const SampleParams &P;
    long long r;
    const Kept &keep;
    __device__ __forceinline__ void token(u64 entry, u64 Z) const
    {
        st(&P.tokens[r], static_cast<int>(~static_cast<unsigned>(entry)));
        if (P.logprob) st(&P.logprob[r], log_prob(listed_delta(static_cast<unsigned>(entry >> 32), keep), Z));
    }
    __device__ __forceinline__ void prob(u64 entry, float scale) const
    {
        st(&P.probs[r * P.probs_stride + static_cast<int>(~static_cast<unsigned>(entry))],
           sv::exp_f32(listed_delta(static_cast<unsigned>(entry >> 32), keep)) * scale);
    }
};

// The key of the k-th largest of the block's entries (each thread's `mine`, 0 for none; at least k
// of them), by halving the span from lo, which all of them reach, to hi, the largest, until just k
// reach it or it is found. Of bf16 logits the upper half of the key says all.
template <typename T, int kMine>
__device__ unsigned kth_key(const u64 (&mine)[kMine], int used, int k, unsigned lo, unsigned hi)
{
    constexpr int drop = sizeof(T) == 2 ? 16 : 0;
    lo >>= drop;
    hi >>= drop;
    while (lo < hi) {
        const unsigned mid = lo + (hi - lo) / 2 + 1;
        int c = 0;
#pragma unroll
        for (int q = 0; q < kMine; ++q)
            if (q < used) c += __syncthreads_count(static_cast<unsigned>(mine[q] >> 32) >> drop >= mid);
        if (c == k) return mid << drop;
        if (c > k) lo = mid;
        else hi = mid - 1;
    }
    return lo << drop;
}

// The share of the weight that a top-p set has to reach: somewhere in [least, most], the same where
// the whole is known exactly. A token is in the set if what lies above it is below that; false comes
// back from a draw that cannot tell for some token.
struct Share {
    bool on;
    u64 least, most;
};

// Among the first kPairs threads of the block, by a barrier of their own.
__device__ __forceinline__ void pairs_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kPairs) : "memory"); }
__device__ __forceinline__ u64 pairs_sum(u64 v, u64 *box)
{
    v = warp_sum(v);
    pairs_sync();
    if ((threadIdx.x & 31) == 0) box[threadIdx.x >> 5] = v;
    pairs_sync();
    v = 0;
#pragma unroll
    for (int w = 0; w < kPairs / 32; ++w) v += box[w];
    return v;
}

// The draw from `count` entries of work[0, count) with their weights in wts, at most kPairs of them
// (with k > 0 from the k largest and their equals): what lies above each in value, and then before
// each in index, is counted and summed over all pairs, several threads to an entry. By half the
// block: more warps would wait on one another's instructions longer than they save.
__device__ bool draw_pairs(const Drawn &out, const u64 *work, u64 *wts, int count, int k, float p, Share share, u64 *part,
                           u64 *box, float u)
{
    const int tid = threadIdx.x;
    if (tid >= kPairs) return true;
    int each = 64;  // threads side by side, one for each entry
    while (each < count) each *= 2;
    const int ways = kPairs / each, i = tid & (each - 1), way = tid / each;
    const int from = way * ((count + ways - 1) / ways), to = min(from + (count + ways - 1) / ways, count);
    const bool first = way == 0;
    const u64 entry = i < count ? work[i] : 0;
    const auto key = static_cast<unsigned>(entry >> 32);
    u64 w = i < count ? wts[i] : 0;
    bool keep = i < count && listed_delta(key, out.keep) >= out.keep.low;
    const bool within = k > 0 && p < 1.0f;  // the share is of what top-k keeps
    if (k > 0 || share.on) {
        u64 above = 0;
        unsigned larger = 0;
#pragma unroll 4
        for (int j = from; j < to; ++j)
            if (static_cast<unsigned>(work[j] >> 32) > key) {
                above += wts[j];
                ++larger;
            }
        if (ways > 1) {  // (the number goes above the weight: 2^40 times 2^8 entries)
            part[tid] = (static_cast<u64>(larger) << 48) + above;
            pairs_sync();
            above = 0;
            for (int v = 0; v < ways; ++v) above += part[v * each + i];
            larger = static_cast<unsigned>(above >> 48);
            above &= (1ull << 48) - 1;
        }
        const bool among = k == 0 || larger < static_cast<unsigned>(k);
        if (within) {
            share.on = true;
            share.least = share.most = share_of(p, pairs_sum(first && among ? w : 0, box));
        }
        keep = keep && among;
        if (share.on) {
            if (share.least != share.most) {
                const u64 doubt = pairs_sum(i < count && above >= share.least && above < share.most ? 1 : 0, box);
                if (doubt) return false;
            }
            keep = keep && above < share.least;
        }
    }
    w = keep ? w : 0;
    const u64 kept = pairs_sum(first ? w : 0, box);  // (its barriers also stand between the uses of wts)
    if (first && i < count) wts[i] = w;
    pairs_sync();
    const auto index = ~static_cast<unsigned>(entry);
    u64 upto = 0;
#pragma unroll 4
    for (int j = from; j < to; ++j)
        if (~static_cast<unsigned>(work[j]) <= index) upto += wts[j];
    if (ways > 1) {
        part[tid] = upto;
        pairs_sync();
        upto = 0;
        if (first)
            for (int v = 0; v < ways; ++v) upto += part[v * each + i];
    }
    if (first && keep) {
        const Target target(u, kept);
        if (target.passed(upto) && !target.passed(upto - w)) out.token(entry, kept);
        if (out.P.probs) out.prob(entry, inverse_sum(kept));
    }
    return true;
}

// The same for more entries, `size` (a power of two, the rest filled with zeros) of them: sorted by
// value and summed up, cut off, sorted by index and summed up again.
__device__ bool draw_sorted(const Drawn &out, u64 *list, u64 *sums, int size, bool within, float p, Share share, float u,
                            Shared &sh)
{
    const int tid = threadIdx.x;
    sort_down(list, size);
    const int q = (size + kThreads - 1) / kThreads;  // contiguous entries of a thread
    u64 own = 0, all;
    auto weight_of = [&](u64 entry) {
        return entry ? weight(exp_weight(listed_delta(static_cast<unsigned>(entry >> 32), out.keep))) : 0ull;
    };
    for (int i = tid * q; i < min(tid * q + q, size); ++i) own += weight_of(list[i]);
    u64 run = block_scan(own, sh.box, &all);
    if (within) {  // the share is of what is listed
        share.on = true;
        share.least = share.most = share_of(p, all);
    }
    for (int i = tid * q; i < min(tid * q + q, size); ++i) {
        run += weight_of(list[i]);
        sums[i] = run;  // up to and with entry i
    }
    if (tid == 0) sh.found = size;
    __syncthreads();
    bool unsure = false;
    for (int i = tid; i < size; i += kThreads) {
        const u64 e = list[i];
        bool out_of = e == 0 || listed_delta(static_cast<unsigned>(e >> 32), out.keep) < out.keep.low;
        if (share.on && i > 0 && static_cast<unsigned>(e >> 32) != static_cast<unsigned>(list[i - 1] >> 32)) {
            out_of |= sums[i - 1] >= share.least;
            unsure |= sums[i - 1] >= share.least && sums[i - 1] < share.most;
        }
        if (out_of) atomicMin(&sh.found, i);
    }
    if (__syncthreads_or(unsure)) return false;
    const int kept = sh.found;
    const u64 Zk = sums[kept - 1];
    if (out.P.probs)
        for (int i = tid; i < kept; i += kThreads) out.prob(list[i], inverse_sum(Zk));
    // index order: (~index, key), the largest first; the weight follows from the key again
    for (int i = tid; i < size; i += kThreads)
        list[i] = i < kept ? (list[i] << 32) | (list[i] >> 32) : 0;
    __syncthreads();
    sort_down(list, size);
    auto turned = [&](int i) { return (list[i] << 32) | (list[i] >> 32); };
    own = 0;
    for (int i = tid * q; i < min(tid * q + q, kept); ++i) own += weight_of(turned(i));
    run = block_scan(own, sh.box, &all);
    const Target target(u, Zk);
    for (int i = tid * q; i < min(tid * q + q, kept); ++i) {
        const u64 next = run + weight_of(turned(i));
        if (target.passed(next) && !target.passed(run)) out.token(turned(i), Zk);
        run = next;
    }
    return true;
}

// The leader's work on its list of `total` candidates. With k > 0 they hold the row's k largest for
// sure where every CTA listed its own k largest, and otherwise where k of them reach the largest of
// the CTAs' cuts (false is returned if not); the row's largest logit is among them in any case.
// Without k, `share` is the top-p set's share of the whole row.
template <typename T>
__device__ bool finish_list(const SampleParams &P, long long r, u64 *list, u64 *sums, int part, int total, int k,
                            bool sure, float p, Share share, float u, Kept &keep, Shared &sh)
{
    constexpr int kMine = kList / kThreads;
    const int tid = threadIdx.x, cluster = P.cluster;
    u64 mine[kMine];
    unsigned top = 0;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        const int i = tid + q * kThreads;
        mine[q] = i < total ? listed_entry(list, part, cluster, sh, i) : 0;
        top = max(top, static_cast<unsigned>(mine[q] >> 32));
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((tid & 31) == 0) sh.small[tid >> 5] = static_cast<int>(top);
    if (tid == 0) sh.mine = 0;
    __syncthreads();
    top = __reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(sh.small[tid & (kWarps - 1)]));
    keep.L = of_key(top);
    if (k > 0) {
        float low = kInf, high = -kInf;
        for (int c = 0; c < cluster; ++c) {
            low = fminf(low, sh.cut[c]);
            high = fmaxf(high, sh.cut[c]);
        }
        if (!sure && high > -FLT_MAX) {
            int c = 0;
#pragma unroll
            for (int q = 0; q < kMine; ++q) c += __syncthreads_count(static_cast<unsigned>(mine[q] >> 32) >= key_of(high));
            if (c < k) return false;
        }
        if (k < total && total > kFewPairs) {
            const unsigned kth = kth_key<T>(mine, (total + kThreads - 1) / kThreads, k, key_of(low), top);
#pragma unroll
            for (int q = 0; q < kMine; ++q)
                if (static_cast<unsigned>(mine[q] >> 32) < kth) mine[q] = 0;
        }
    }
    const Drawn out{P, r, keep};
    if (total <= kFewPairs) {
        u64 *wts = sums, *part = sums + kPairs;
        if (tid < total) {
            list[tid] = mine[0];  // (all entries have been read)
            wts[tid] = weight(exp_weight(listed_delta(static_cast<unsigned>(mine[0] >> 32), keep)));
        }
        __syncthreads();
        return draw_pairs(out, list, wts, total, k, p, share, part, sh.box, u);
    }
    // the entries left, in any order, closed up
    u64 *wts = sums;
#pragma unroll
    for (int q = 0; q < kMine; ++q) {
        const unsigned some = __ballot_sync(0xFFFFFFFFu, mine[q] != 0);
        int at = 0;
        if ((tid & 31) == 0 && some) at = static_cast<int>(atomicAdd(&sh.mine, __popc(some)));
        at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(some & ((1u << (tid & 31)) - 1));
        if (mine[q]) {
            list[at] = mine[q];
            wts[at] = weight(exp_weight(listed_delta(static_cast<unsigned>(mine[q] >> 32), keep)));
        }
    }
    __syncthreads();
    const int count = static_cast<int>(sh.mine);
    if (count <= kPairs) return draw_pairs(out, list, wts, count, k, p, share, sums + kPairs, sh.box, u);
    int size = 1;
    while (size < count) size *= 2;
    for (int i = count + tid; i < size; i += kThreads) list[i] = 0;
    __syncthreads();
    return draw_sorted(out, list, sums, size, k > 0 && p < 1.0f, p, share, u, sh);
}

template <bool kAll>
__device__ __forceinline__ float kept_weight(float l, const Kept &keep)
{
    const float d = delta(l, keep.L, keep.inv);
    const float t = exp_weight(d);
    return kAll || (l >= keep.tau && d >= keep.low) ? t : 0.0f;
}
template <bool kAll>
__device__ __forceinline__ Two kept_weight(float l, float m, const Kept &keep)
{
    const Two d = (two(l, m) + two(-keep.L)) * two(keep.inv);
    const Two t = exp_weight(d);
    if (kAll) return t;
    float da, db, a, b;
    parts(d, da, db);
    parts(t, a, b);
    return two(l >= keep.tau && da >= keep.low ? a : 0.0f, m >= keep.tau && db >= keep.low ? b : 0.0f);
}

// This warp's sum of the kept tokens' weights.
template <bool kAll, typename RowT>
__device__ __forceinline__ u64 warp_weight(const RowT &R, const Kept &keep)
{
    constexpr int n = RowT::n, k = 4;
    WeightSum s;
    int count = 0;
    R.template each<k, true>([&](uint4 (&v)[k], int m, int) {
#pragma unroll
        for (int i = 0; i < k; ++i)
            if (i < m) {
                float f[n];
                Vec<typename RowT::Elem>::get(v[i], f);
#pragma unroll
                for (int e = 0; e < n; e += 2) s.add(kept_weight<kAll>(f[e], f[e + 1], keep));
            }
        count += n * m;
    });
    return warp_sum(s.total(count));
}

// A value of every warp to every CTA of the cluster (`turn` alternates between the two buffers:
// a CTA that writes one again has passed a barrier that the others reach only after reading it).
struct Exchange {
    Shared &sh;
    unsigned rank;
    int cluster, turn;
    __device__ __forceinline__ const u64 *all(u64 mine)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        u64 *to = sh.seg[turn & 1];
        ++turn;
        if (lane < cluster) put(remote(to + rank * kWarps + warp, lane), mine);
        cluster_sync();
        return to;
    }
    __device__ u64 sum(u64 mine)
    {
        const u64 *v = all(mine);
        u64 s = 0;
        for (int i = threadIdx.x & 31; i < cluster * kWarps; i += 32) s += v[i];
        return warp_sum(s);
    }
};

// How much the tokens from l >= bound on hold: tokens or, with kMass, weight; of those >= keep.tau.
template <bool kMass, typename RowT>
__device__ u64 held_from(const RowT &R, const Kept &keep, float bound, Exchange &ex)
{
    constexpr int n = RowT::n, k = 4;
    Kept from = keep;
    from.tau = fmaxf(bound, keep.tau);
    from.low = -kInf;
    if (kMass) return ex.sum(warp_weight<false>(R, from));
    int c = 0;
    R.template each<k>([&](uint4 (&v)[k], int, int) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
            float f[n];
            Vec<typename RowT::Elem>::get(v[i], f);
#pragma unroll
            for (int e = 0; e < n; ++e) c += f[e] >= from.tau;
        }
    });
    return ex.sum(warp_sum(static_cast<u64>(c)));
}

// The largest key in [lo, hi] such that the tokens with keys at least as large hold `need`, or 0
// where those from lo on do not: by halving, one pass over the row for each step.
template <bool kMass, typename RowT>
__device__ unsigned search_key(const RowT &R, const Kept &keep, u64 need, unsigned lo, unsigned hi, Exchange &ex)
{
    constexpr int drop = RowT::n == 8 ? 16 : 0;  // (of bf16 logits the upper half of the key says all)
    constexpr unsigned least = 0x00800000u;        // the key of the lowest finite number
    lo >>= drop;
    hi >>= drop;
    if (held_from<kMass>(R, keep, of_key(max(lo << drop, least)), ex) < need) return 0;
    while (lo < hi) {
        const unsigned mid = lo + (hi - lo) / 2 + 1;
        if (held_from<kMass>(R, keep, of_key(max(mid << drop, least)), ex) >= need) lo = mid;
        else hi = mid - 1;
    }
    return max(lo << drop, least);
}

// What is known of a row before its bracket is looked for: the weight `heavy` (2^40 to 1) of the
// tokens >= ceiling (+inf and 0: nothing is), the -d beyond which it does not lie, and about the weight
// of the whole (1 to 1; 0: nothing is).
struct Known {
    float ceiling, lowest, whole;
    u64 heavy;
};

// A bracket of the value at which the row's tokens from the largest on hold `count` of them or, with
// kMass, the part p of their weight; of the tokens >= keep.tau. From a histogram of the tokens by
// d, kBins bins: for counts the bin it is in; for weights, which the bins' middles stand for, that and
// the bins beside it until they hold kBeside tokens on each side (the error is that of a few tokens:
// the heaviest, those from known.ceiling on, are not in the histogram, and their weight is exact).
// Where the bracket holds more than the list, a second histogram of just that span narrows it down
// further. A guess that the caller checks: sh.lower and sh.upper of every CTA.
template <bool kMass, typename T>
__device__ void bracket(const Row<T> &R, const Kept &keep, unsigned count, float p, const Known &known, const Room &room,
                        Exchange &ex)
{
    constexpr int n = Row<T>::n, kv = 4;
    Shared &sh = ex.sh;
    const int tid = threadIdx.x, cluster = ex.cluster;
    auto *bins = reinterpret_cast<unsigned *>(room.peaks);
    // the bins' first edge and width, in -d
    float from = 0.0f;
    if (known.ceiling < kInf) {
        // (between the last value that is known and the next: of bf16 logits half-way, whose ceiling is a
        // key with zeros below; a token there in neither part, or in both, would be missed by the guess)
        const unsigned key = key_of(known.ceiling);
        from = (keep.L - (sizeof(T) == 4 ? known.ceiling : of_key(key & 0x80000000u ? key - 0x8000u : key + 0x7FFFu))) * keep.inv;
    }
    float width = fmaxf(fminf(known.lowest, kSpan) - from, 1e-3f) / kBins;
    float before = static_cast<float>(known.heavy >> 20) * 0x1p-20f, want = 0.0f;  // (the leader's)
    for (int level = 0; level < 2; ++level) {
        const float scale = keep.inv / width, shift = from / width;
        for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
        __syncthreads();
        R.template each<kv, true>([&](uint4 (&v)[kv], int m, int) {
#pragma unroll
            for (int i = 0; i < kv; ++i)
                if (i < m) {
                    float f[n];
                    Vec<T>::get(v[i], f);
#pragma unroll
                    for (int e = 0; e < n; ++e) {
                        const int b = __float2int_rd(__fmaf_rn(keep.L - f[e], scale, -shift));
                        if (static_cast<unsigned>(b) < kBins && f[e] >= keep.tau) atomicAdd(bins + b, 1u);
                    }
                }
        });
        cluster_sync();
        if (ex.rank == 0) {
            constexpr int q = kBins / kThreads;  // bins of a thread
            unsigned c[q] = {};
#pragma unroll 4
            for (int k = 0; k < cluster; ++k)
#pragma unroll
                for (int i = 0; i < q / 4; ++i) {
                    const uint4 v = get16(remote(bins + tid * q + 4 * i, k));
                    c[4 * i] += v.x;
                    c[4 * i + 1] += v.y;
                    c[4 * i + 2] += v.z;
                    c[4 * i + 3] += v.w;
                }
            float w[q], mass = 0.0f, total;
            unsigned tokens = 0, all;
#pragma unroll
            for (int i = 0; i < q; ++i) {
                float middle = from + (static_cast<float>(tid * q + i) + 0.5f) * width;
                if (kMass && sizeof(T) == 2) {
                    // (a bin that holds one bf16 value: that, or the bins of evenly spaced values would all
                    // be off to one side)
                    const unsigned near = __float_as_uint(keep.L - middle / keep.inv) + 0x8000u;
                    const float value = __uint_as_float(near & 0xFFFF0000u);
                    if (__float2int_rd(__fmaf_rn(keep.L - value, scale, -shift)) == tid * q + i) middle = (keep.L - value) * keep.inv;
                }
                w[i] = kMass ? static_cast<float>(c[i]) * sv::ex2_approx(-middle * kLog2e) : static_cast<float>(c[i]);
                mass += w[i];
                tokens += c[i];
            }
            float run = mass;
            unsigned passed = tokens;
            block_scan(run, passed, sh.box, &total, &all);
            if (level == 0) want = kMass ? p * (known.whole > 0.0f ? known.whole : before + total) : static_cast<float>(count);
            // the bin in which it lies, and the number of tokens before it
            if (tid == 0) {
                sh.first = before < want ? kBins : 0;
                sh.mine = before < want ? all : 0;
                sh.run = 0;
                sh.found = kBins - 1;
            }
            __syncthreads();
            run += before;
            if (run < want && run + mass >= want) {
                int i = 0;
                unsigned t = passed;
                float m = run;
#pragma unroll
                for (int j = 0; j < q - 1; ++j)
                    if (i == j && m + w[j] < want) {
                        m += w[j];
                        t += c[j];
                        ++i;
                    }
                if (atomicMin(&sh.first, tid * q + i) > tid * q + i) sh.mine = t;
            }
            __syncthreads();
            const int b = sh.first;
            const unsigned here = sh.mine, beside = kMass ? kBeside : 0;
            // the bracket's first bin: the last one below b before which `beside` fewer tokens lie; its
            // last: the first one above b up to which as many more lie
            if (kMass && b < kBins) {
                unsigned t = passed;
#pragma unroll
                for (int i = 0; i < q; ++i) {
                    const int at = tid * q + i;
                    if (at < b && t + beside <= here) atomicMax(&sh.run, at);
                    t += c[i];
                    if (at > b && t >= here + 2 * beside) atomicMin(&sh.found, at);
                }
            }
            __syncthreads();
            const int head = kMass && b < kBins ? sh.run : min(b, kBins - 1);
            const int tail = kMass && b < kBins ? max(sh.found, min(b + 1, kBins - 1)) : min(b, kBins - 1);
            // what the bracket holds in tokens, and what lies before it
            unsigned in = 0;
            float m = run, none = 0.0f, unused;
#pragma unroll
            for (int i = 0; i < q; ++i) {
                const int at = tid * q + i;
                if (at >= head && at <= tail) in += c[i];
                if (at == head) sh.d = m;
                m += w[i];
            }
            block_scan(none, in, sh.box, &unused, &all);
            before = sh.d;
            // (in the last bin or beyond it: everything below)
            const float slack = 4e-6f * fmaxf(fabsf(keep.L), kSpan / keep.inv);
            const float lo = from + static_cast<float>(head) * width, hi = from + static_cast<float>(tail + 1) * width;
            const float upper = head == 0 && level == 0 ? (known.ceiling < kInf ? known.ceiling : keep.L) : keep.L - lo / keep.inv + slack;
            const float lower = level == 0 && tail == kBins - 1 ? -FLT_MAX : keep.L - hi / keep.inv - slack;
            if (tid < cluster) {
                put(remote(&sh.upper, tid), __float_as_uint(upper));
                put(remote(&sh.lower, tid), __float_as_uint(fmaxf(lower, -FLT_MAX)));
                put(remote(&sh.from, tid), __float_as_uint(lo));
                put(remote(&sh.width, tid), __float_as_uint((hi - lo) / kBins));
                // (of bf16 logits with a distinct value or two there a second look tells nothing more)
                const bool again = level == 0 && b < kBins && all * (cluster > 1 ? 5 : 3) / 3 > kWideList &&
                                   (sizeof(T) == 4 || key_of(upper) >> 16 > (key_of(lower) >> 16) + 2);
                put(remote(&sh.again, tid), static_cast<unsigned>(again));
            }
        }
        cluster_sync();
        if (!sh.again) return;
        from = sh.from;
        width = sh.width;
    }
}

// One pass over the row for a bracket: the tokens within it go to the leader's list as (key, ~index);
// *above: this warp's tokens above it or, with kMass, their weight, and *all the weight of all tokens
// >= keep.tau (kAll: of all).
template <bool kMass, bool kAll, typename T>
__device__ __forceinline__ void gather(const Row<T> &R, const Kept &keep, float lower, float upper, const Room &room, int part,
                                       u64 *above, u64 *all, Exchange &ex)
{
    constexpr int n = Row<T>::n, kv = 4;
    Shared &sh = ex.sh;
    const int tid = threadIdx.x;
    if (tid == 0) sh.mine = 0;
    __syncthreads();
    u64 *mine = room.list + ex.rank * part;
    WeightSums sums;
    int count = 0;
    R.template each<kv, true>([&](uint4 (&v)[kv], int m, int c) {
#pragma unroll
        for (int i = 0; i < kv; ++i) {
            if (i >= m) continue;
            float f[n];
            Vec<T>::get(v[i], f);
            bool within = false;
#pragma unroll
            for (int e = 0; e < n; e += 2) {
                if (kMass) {
                    sums.add(kept_weight<kAll>(f[e], f[e + 1], keep), f[e] > upper, f[e + 1] > upper);
                } else {
                    count += f[e] > upper;
                    count += f[e + 1] > upper;
                }
                within |= (f[e] >= lower && f[e] <= upper) || (f[e + 1] >= lower && f[e + 1] <= upper);
            }
            if (within)
#pragma unroll
                for (int e = 0; e < n; ++e)
                    if (f[e] >= lower && f[e] <= upper) {
                        const unsigned at = atomicAdd(&sh.mine, 1u);
                        const auto index = static_cast<unsigned>(R.base + (R.lo + R.lane + 32 * (c * kv + i)) * n + e);
                        if (at < static_cast<unsigned>(part))
                            mine[at] = (static_cast<u64>(key_of(f[e])) << 32) | static_cast<u64>(~index);
                    }
        }
        if (kMass) count += n * m;
    });
    *above = warp_sum(kMass ? sums.total_marked(count) : static_cast<u64>(count));
    *all = kMass ? warp_sum(sums.total(count)) : 0;
    __syncthreads();
    const int listed = static_cast<int>(sh.mine);
    if (ex.rank != 0)
        for (int i = tid; i < min(listed, part); i += kThreads) put(remote(mine + i, 0), mine[i]);
    if (tid < ex.cluster) put(remote(&sh.count[ex.rank], tid), static_cast<unsigned>(listed));
}

// The leader's entries of the list, a thread's share of them, with their weights (kMass) or 1.
template <bool kMass>
struct Listed {
    static constexpr int per = kWideList / kThreads;
    u64 entry[per], w[per];
    __device__ __forceinline__ Listed(const u64 *list, int part, int cluster, int total, const Kept &keep, const Shared &sh)
    {
#pragma unroll
        for (int q = 0; q < per; ++q) {
            const int i = static_cast<int>(threadIdx.x) + q * kThreads;
            entry[q] = i < total ? listed_entry(list, part, cluster, sh, i) : 0;
            const auto key = static_cast<unsigned>(entry[q] >> 32);
            w[q] = key == 0 ? 0 : kMass ? weight(exp_weight(delta(of_key(key), keep.L, keep.inv))) : 1;
        }
    }
    // The largest key in [lo, hi] such that `over` and the entries with keys at least as large hold
    // `need`, or 0; *held: what they hold.
    template <typename T>
    __device__ __forceinline__ unsigned key(u64 over, u64 need, unsigned lo, unsigned hi, u64 *held, Shared &sh) const
    {
        constexpr int drop = sizeof(T) == 2 ? 16 : 0;
        // (in halves of 20 bits, which the warp's own addition takes, and one barrier a step)
        int turn = 0;
        auto from = [&](unsigned bound) {
            unsigned a = 0, b = 0;
#pragma unroll
            for (int q = 0; q < per; ++q)
                if (static_cast<unsigned>(entry[q] >> 32) >> drop >= bound) {
                    a += static_cast<unsigned>(w[q]) & 0xFFFFFu;
                    b += static_cast<unsigned>(w[q] >> 20);
                }
            a = __reduce_add_sync(0xFFFFFFFFu, a);
            b = __reduce_add_sync(0xFFFFFFFFu, b);
            u64 *box = sh.seg[turn ^= 1];
            const int lane = threadIdx.x & 31;
            if (lane == 0) box[threadIdx.x >> 5] = (static_cast<u64>(b) << 32) | a;
            __syncthreads();
            const u64 x = lane < kWarps ? box[lane] : 0;
            return over + __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(x)) +
                   (static_cast<u64>(__reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(x >> 32))) << 20);
        };
        lo >>= drop;
        hi >>= drop;
        __syncthreads();  // (what was in these boxes has been read)
        *held = from(lo);
        if (*held < need) return 0;
        while (lo < hi) {
            const unsigned mid = lo + (hi - lo) / 2 + 1;
            const u64 h = from(mid);
            if (h >= need) {
                lo = mid;
                *held = h;
            } else {
                hi = mid - 1;
            }
        }
        return max(lo << drop, 1u);
    }
};

// The largest key such that the tokens at least as large hold k of them, for a k beyond the list; 0
// where the row has fewer tokens. Where the bracket holds more than the list, or the guess was wrong,
// it is found by halving.
template <typename T>
__device__ __noinline__ unsigned find_kth(const Row<T> &R, const Kept &keep, u64 k, const Room &room, Exchange &ex)
{
    Shared &sh = ex.sh;
    const int part = kWideList / ex.cluster;
    bracket<false>(R, keep, static_cast<unsigned>(k), 0.0f, Known{kInf, kSpan, 0.0f, 0}, room, ex);
    const float upper = sh.upper, lower = sh.lower;
    u64 above, all;
    gather<false, true>(R, keep, lower, upper, room, part, &above, &all, ex);
    const u64 over = ex.sum(above);
    int total;
    unsigned found = 0;
    if (over < k) {
        if (all_listed(sh, ex.cluster, part, &total)) {
            if (ex.rank == 0) {
                const Listed<false> mine(room.list, part, ex.cluster, total, keep, sh);
                found = mine.template key<T>(over, k, key_of(lower), key_of(upper), &all, sh);
                if (threadIdx.x < ex.cluster) put(remote(&sh.fits, threadIdx.x), found);
            }
            cluster_sync();
            found = sh.fits;
        } else {
            found = search_key<false>(R, keep, k, key_of(lower), key_of(upper), ex);
        }
    }
    return found ? found : search_key<false>(R, keep, k, 0, key_of(keep.L), ex);
}

// Where in the runs of the cluster's warps, whose kept weights are in seg, the target falls: the run
// and the weight before it. By every warp that calls it.
__device__ __forceinline__ int find_run(const u64 *seg, int warps, float u, u64 *Z, u64 *below)
{
    constexpr int q = kMaxCluster * kWarps / 32;  // a lane's consecutive runs
    const int lane = threadIdx.x & 31;
    u64 own = 0;
#pragma unroll
    for (int i = 0; i < q; ++i)
        if (lane * q + i < warps) own += seg[lane * q + i];
    u64 upto = own;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const u64 o = __shfl_up_sync(0xFFFFFFFFu, upto, k);
        if (lane >= k) upto += o;
    }
    *Z = __shfl_sync(0xFFFFFFFFu, upto, 31);
    const Target target(u, *Z);
    const int at = __ffs(__ballot_sync(0xFFFFFFFFu, target.passed(upto))) - 1;
    int s = 0;
    u64 b = upto - own;
    if (lane == at) {
        s = lane * q;
        while (!target.passed(b + seg[s])) b += seg[s++];
    }
    *below = __shfl_sync(0xFFFFFFFFu, b, at);
    return __shfl_sync(0xFFFFFFFFu, s, at);
}

// The CTA's part of the distribution over kept tokens. Where not all are kept the row is 0 before,
// and only vectors with kept tokens are written. Four probabilities at a time where the rows of
// logits and probabilities lie alike to 16 bytes, else one by one, neighbours by neighbouring lanes.
template <bool kAll, typename T>
__device__ __forceinline__ void write_probs(const Row<T> &R, float *probs, const Kept &keep, u64 Z)
{
    constexpr int n = Row<T>::n, k = 2;
    const float scale = inverse_sum(Z);
    if ((reinterpret_cast<uintptr_t>(probs + R.base) & 15u) != 0) {
        for (int i = R.first() + static_cast<int>(threadIdx.x); i < R.last(); i += kThreads) {
            const float l = R.at(i), d = delta(l, keep.L, keep.inv);
            const bool in = l > -kInf && (kAll || (l >= keep.tau && d >= keep.low));
            if (kAll || in) st(&probs[i], in ? sv::exp_f32(d) * scale : 0.0f);
        }
        return;
    }
    R.template each<k, true>([&](uint4 (&v)[k], int m, int c) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
            const int j = R.lo + R.lane + 32 * (c * k + i);
            if (i >= m || j >= R.hi) continue;
            Largest<T> largest;
            largest.add(v[i]);
            if (!kAll && !(largest.get() >= keep.tau)) continue;
            float f[n];
            Vec<T>::get(v[i], f);
#pragma unroll
            for (int e = 0; e < n; e += 2) {
                const Two d = (two(f[e], f[e + 1]) + two(-keep.L)) * two(keep.inv);
                float da, db, a, b;
                parts(d, da, db);
                parts(exp_two(d) * two(scale), a, b);
                // (the comparison also keeps a NaN and -inf out)
                f[e] = f[e] > -kInf && (kAll || (f[e] >= keep.tau && da >= keep.low)) ? a : 0.0f;
                f[e + 1] = f[e + 1] > -kInf && (kAll || (f[e + 1] >= keep.tau && db >= keep.low)) ? b : 0.0f;
            }
            const int first = R.base + j * n;
            if (first >= 0 && first + n <= R.V) {
#pragma unroll
                for (int e = 0; e < n; e += 4)
                    st(reinterpret_cast<float4 *>(probs + first + e), make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]));
            } else {
#pragma unroll
                for (int e = 0; e < n; ++e)
                    if (first + e >= 0 && first + e < R.V) st(&probs[first + e], f[e]);
            }
        }
    });
}

// Zeros for the CTA's part of a distribution, marked to leave the L2 cache first: the logits are read
// again, these are not (256 mixed rows of 151936 bf16 logits 116 against 142 us).
template <typename T>
__device__ __forceinline__ void write_zeros(const Row<T> &R, float *probs)
{
    const int tid = threadIdx.x, first = R.first(), last = R.last();
    const int head = min(first + static_cast<int>((16u - (reinterpret_cast<uintptr_t>(probs + first) & 15u)) / 4u % 4u), last);
    const int body = head + max(last - head, 0) / 4 * 4;
    if (first + tid < head) st(&probs[first + tid], 0.0f);
    for (int i = head + 4 * tid; i < body; i += 4 * kThreads) st_leaving(reinterpret_cast<float4 *>(probs + i), make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    if (body + tid < last) st(&probs[body + tid], 0.0f);
}

// The draw where the run on which the uniform number falls is known: the CTA that holds it finds the
// token in it, and each writes its part of the distribution.
template <bool kAll, typename T>
__device__ void draw_run(const SampleParams &P, const Row<T> &R, long long r, float u, const Kept &keep, int s, u64 below, u64 Z,
                         unsigned rank, Shared &sh)
{
    constexpr int n = Row<T>::n;
    const int tid = threadIdx.x;
    if (s / kWarps == static_cast<int>(rank)) {
        const Target target(u, Z);
        const int lo = min((s % kWarps) * R.per_warp, R.mine), hi = min(lo + R.per_warp, R.mine);
        const int each = (hi - lo + kThreads - 1) / kThreads;
        const int from = min(lo + tid * each, hi), to = min(from + each, hi);
        u64 sum = 0, all;
        for (int j = from; j < to; ++j) {
            float f[n];
            Vec<T>::get(R.get(j), f);
#pragma unroll
            for (int e = 0; e < n; ++e) sum += weight(kept_weight<kAll>(f[e], keep));
        }
        u64 run = below + block_scan(sum, sh.box, &all);
        if (target.passed(run + sum) && !target.passed(run)) {
            const int last = R.base + to * n - 1;  // (it ends before this, unless the row changes meanwhile)
            int i = R.base + from * n;
            float l = R.at(i);
            while (!target.passed(run += weight(kept_weight<kAll>(l, keep))) && i < last) l = R.at(++i);
            st(&P.tokens[r], i);
            if (P.logprob) st(&P.logprob[r], log_prob(delta(l, keep.L, keep.inv), Z));
        }
    }
    if (P.probs) write_probs<kAll>(R, P.probs + r * P.probs_stride, keep, Z);
}

// The draw over the whole row by one pass of exact sums: every warp's goes to every CTA.
template <bool kAll, typename T>
__device__ void draw_row(const SampleParams &P, const Row<T> &R, long long r, float u, const Kept &keep, Exchange &ex)
{
    const u64 *seg = ex.all(warp_weight<kAll>(R, keep));
    u64 Z, below;
    const int s = find_run(seg, P.cluster * kWarps, u, &Z, &below);
    draw_run<kAll>(P, R, r, u, keep, s, below, Z, ex.rank, ex.sh);
}

// The draw from a top-p set larger than the list (of the tokens >= keep.tau): a bracket of the least
// logit in it by the histogram, one pass that sums up all, what lies above the bracket in every
// warp's run, and lists what lies in it; the leader finds the least logit, adds the listed tokens
// that are in the set to their runs, and finds the run to draw from.
template <typename T>
__device__ __noinline__ void draw_wide(const SampleParams &P, const Row<T> &R, long long r, float p, float u, Kept keep,
                                      const Known &known, const Room &room, Exchange &ex)
{
    constexpr int n = Row<T>::n;
    Shared &sh = ex.sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cluster = ex.cluster, part = kWideList / cluster;
    bracket<true>(R, keep, 0, p, known, room, ex);
    const float upper = sh.upper, lower = fmaxf(sh.lower, keep.tau);
    u64 above, all;
    Kept whole = keep;
    whole.low = -kInf;
    if (keep.tau == -FLT_MAX) gather<true, true>(R, whole, lower, upper, room, part, &above, &all, ex);
    else gather<true, false>(R, whole, lower, upper, room, part, &above, &all, ex);
    if (lane < cluster) put(remote(&sh.runs[ex.rank * kWarps + warp], lane), above);  // (as Exchange does)
    const u64 Z = ex.sum(all);
    u64 over = 0;
    for (int i = lane; i < cluster * kWarps; i += 32) over += sh.runs[i];
    over = warp_sum(over);
    const u64 need = share_of(p, Z);
    int total;
    bool done = false;
    unsigned key = 0;
    if (over < need && all_listed(sh, cluster, part, &total)) {
        if (ex.rank == 0) {
            const Listed<true> mine(room.list, part, cluster, total, keep, sh);
            u64 held;
            key = mine.template key<T>(over, need, key_of(lower), key_of(upper), &held, sh);
            const float tau = of_key(max(key, 0x00800000u));
            // (what min-p leaves out of the set is not in these sums)
            const bool plain = key && !(delta(tau, keep.L, keep.inv) < keep.low);
            if (plain) {
                const int off = static_cast<int>((reinterpret_cast<uintptr_t>(R.row) & 15u) / sizeof(T));
#pragma unroll
                for (int q = 0; q < mine.per; ++q)
                    if (static_cast<unsigned>(mine.entry[q] >> 32) >= key) {
                        const int j = (static_cast<int>(~static_cast<unsigned>(mine.entry[q])) + off) / n;
                        const int at = j / P.split.per_cta * kWarps + j % P.split.per_cta / P.split.per_warp;
                        atomicAdd(&sh.runs[at], mine.w[q]);
                    }
            }
            __syncthreads();
            if (plain && warp == 0) {
                u64 kept, below;
                const int s = find_run(sh.runs, cluster * kWarps, u, &kept, &below);
                if (lane < cluster) {
                    put(remote(&sh.kept, lane), kept);
                    put(remote(&sh.below, lane), below);
                    put(remote(&sh.run, lane), static_cast<unsigned>(s));
                }
            }
            if (tid < cluster) {
                put(remote(&sh.tau, tid), key);
                put(remote(&sh.fits, tid), static_cast<unsigned>(plain));
            }
        }
        cluster_sync();
        key = sh.tau;
        done = sh.fits != 0;
    } else if (over < need) {
        key = search_key<true>(R, keep, need, key_of(lower), key_of(upper), ex);
    }
    if (key == 0) key = search_key<true>(R, keep, need, 0, key_of(keep.L), ex);
    keep.tau = of_key(key);
    if (done) draw_run<false>(P, R, r, u, keep, sh.run, sh.below, sh.kept, ex.rank, sh);
    else draw_row<false>(P, R, r, u, keep, ex);
}

// The calls of the two functions that stay functions (in line, their registers would be taken from
// the common rows): with copies, so that what the caller keeps in registers stays there.
template <typename T>
__device__ __forceinline__ void call_wide(const SampleParams &P, const Row<T> &R, long long r, float p, float u, const Kept &keep,
                                          const Known &known, const Room &room, const Exchange &ex)
{
    const Row<T> row = R;
    const Known k = known;
    const Room m = room;
    Exchange e = ex;
    draw_wide(P, row, r, p, u, keep, k, m, e);
}
template <typename T>
__device__ __forceinline__ unsigned call_kth(const Row<T> &R, const Kept &keep, u64 k, const Room &room, Exchange &ex)
{
    const Row<T> row = R;
    const Kept kept = keep;
    const Room m = room;
    Exchange e = ex;
    const unsigned key = find_kth(row, kept, k, m, e);
    ex.turn = e.turn;
    return key;
}

// The row of the cluster at place `at`, where those whose top-p set or k may be beyond the list come
// first (each kind in order): they take three times as long as the others, and where the device does not
// hold all rows at once the last to start decides how long the call takes. For up to 2 kThreads rows
// (more than that go to the smaller blocks, without an order).
__device__ __forceinline__ int long_first(const SampleParams &P, int at, Shared &sh)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rows = P.ordered;
    bool is_long[2];
    unsigned same[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = tid + q * kThreads;
        is_long[q] = false;
        if (row < rows) {
            const int k = P.top_k ? ld(P.top_k + row) : 0;
            const bool limited = k >= 1 && k < P.V;
            is_long[q] = limited ? k > kList / 2 : P.top_p && ld(P.top_p + row) < 1.0f;
            is_long[q] = is_long[q] && (!P.temperature || ld(P.temperature + row) > 0.0f);
        }
        same[q] = __ballot_sync(0xFFFFFFFFu, is_long[q]);
    }
    if (tid == 0) sh.first = at;  // (a row in any case, also where the limits change meanwhile)
    if (lane == 0) sh.box[warp] = (static_cast<u64>(__popc(same[1])) << 32) | static_cast<u64>(__popc(same[0]));
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sh.box[w];
        all += sh.box[w];
    }
    const int first = static_cast<int>(all & 0xFFFFFFFFu), total = first + static_cast<int>(all >> 32);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = tid + q * kThreads;
        const int n = (q ? first + static_cast<int>(before >> 32) : static_cast<int>(before & 0xFFFFFFFFu)) +
                      __popc(same[q] & ((1u << lane) - 1));
        if (row < rows && (is_long[q] ? n : total + row - n) == at) sh.first = row;
    }
    __syncthreads();
    return sh.first;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtas) sv_sample_kernel(const T *logits, SampleParams P)
{
    extern __shared__ uint4 store[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, cluster = P.cluster;
    const unsigned rank = cluster_rank();
    const int place = static_cast<int>(blockIdx.x) / cluster;
    const Room room(store);
    cluster_announce();  // (waited for before the first write to another CTA: that it runs by then)
    const long long r = kOrdered && P.ordered ? long_first(P, place, sh) : place;
    Row<T> R = start_row(logits + r * P.stride, P.V, P.split, rank, sh);
    const int part = kList / cluster;
    const float temp = P.temperature ? ld(P.temperature + r) : 1.0f;
    const int k0 = P.top_k ? ld(P.top_k + r) : 0;
    const float p = P.top_p ? ld(P.top_p + r) : 1.0f;
    const float m = P.min_p ? ld(P.min_p + r) : 0.0f;
    const float u = ld(P.uniforms + r);
    const bool greedy = !(temp > 0.0f) || k0 == 1;
    const int k = k0 >= 1 && k0 < P.V ? k0 : 0;
    const bool open = !greedy && !k && !(p < 1.0f) && !(m > 0.0f);
    float *probs = P.probs ? P.probs + r * P.probs_stride : nullptr;
    if (probs && !open) write_zeros(R, probs);  // what is kept goes over them
    // (in binary64, by one thread, while the others read)
    if (m > 0.0f && tid == 0) sh.d = __double2float_rn(log(static_cast<double>(fminf(m, 1.0f))));
    const bool mass = p < 1.0f && k == 0 && !greedy;  // the top-p set's total is the whole row's
    const float scale = fminf(inverse(temp) * kLog2e, FLT_MAX);
    float sum = 0.0f;
    const float peak = mass ? lane_max<true>(R, room.peaks, scale, &sum) : lane_max<false>(R, room.peaks, scale, &sum);
    const float largest = block_max(peak, sh);
    cluster_wait();

    if (greedy) {  // each CTA's first largest, and the first largest of those
        if (tid == 0) sh.first = INT_MAX;
        __syncthreads();
        if (peak == largest && peak > -kInf) {
            int best = INT_MAX;
            for (int j = R.lo + R.lane; j < R.hi && best == INT_MAX; j += 32) {
                float f[R.n];
                Vec<T>::get(R.get(j), f);
                for (int e = R.n - 1; e >= 0; --e)
                    if (f[e] == largest) best = R.base + j * R.n + e;
            }
            atomicMin(&sh.first, best);
        }
        __syncthreads();
        if (tid == 0) {
            put(remote(&sh.count[rank], 0), static_cast<unsigned>(sh.first));
            put(remote(&sh.peak[rank], 0), __float_as_uint(largest));
        }
        cluster_sync();
        if (rank == 0 && tid == 0) {
            int best = -1;
            float L = -kInf;
            for (int c = 0; c < cluster; ++c)
                if (sh.peak[c] > L) {
                    L = sh.peak[c];
                    best = static_cast<int>(sh.count[c]);
                }
            st(&P.tokens[r], best);
            if (P.logprob) st(&P.logprob[r], best < 0 ? -kInf : 0.0f);
            if (probs && best >= 0) st(&probs[best], 1.0f);
        }
        return;
    }

    Kept keep{0.0f, inverse(temp), -FLT_MAX, m > 0.0f ? sh.d : -kInf};
    int total;
    if (k > 0) {
        // the k largest: of every CTA at least its own k largest, or as many as find place. (Of tokens in
        // any order 0.8 part are expected from a cut on that the lanes' share 1 - exp(-0.8 part / lanes)
        // reaches: at most so many may, or the list would often be too small, and then the histogram takes
        // over: with a top-k of 300, 700 rows of 151936 bf16 logits, 725 us against 147.)
        const int lanes = static_cast<int>(kThreads * (1.0f - sv::ex2_approx(-0.8f * kLog2e / kThreads * static_cast<float>(part))));
        const int most = min(part / 8 * 5, lanes / 16 * 15), want = min(k, most);
        const float cut = cut_for<T>(peak, largest, want, min(want + (want >> 2), lanes), sh);
        collect<false>(R, cut, room, part, rank, cluster, keep, true, sh);
        cluster_sync();
        if (all_listed(sh, cluster, part, &total)) {
            if (total == 0) {  // nothing to keep
                if (rank == 0 && tid == 0) {
                    st(&P.tokens[r], -1);
                    if (P.logprob) st(&P.logprob[r], -kInf);
                }
                return;
            }
            if (k <= most) {
                if (rank == 0) finish_list<T>(P, r, room.list, room.work, part, total, k, true, p, Share{}, u, keep, sh);
                return;
            }
            if (rank == 0) {
                const bool done = finish_list<T>(P, r, room.list, room.work, part, total, k, false, p, Share{}, u, keep, sh);
                if (tid < cluster) put(remote(&sh.fits, tid), static_cast<unsigned>(done));
            }
            cluster_sync();
            if (sh.fits) return;
        }
    }
    // the row's largest logit
    // (a list of all CTAs that is still compared each with each: a row of 151936 bf16 logits whose set is
    // small 13 us, where eight CTAs list 64 each 27)
    const int few = kTopP / max(cluster / 2, 1);
    const float own_cut = mass ? cut_for<T>(peak, largest, few, few + (few >> 2), sh) : 0.0f;
    if (tid < cluster) {
        put(remote(&sh.peak[rank], tid), __float_as_uint(largest));
        put(remote(&sh.cut[rank], tid), __float_as_uint(own_cut));
    }
    cluster_sync();
    float L = -kInf, cut = -FLT_MAX;
    for (int c = 0; c < cluster; ++c) {
        L = fmaxf(L, sh.peak[c]);
        cut = fmaxf(cut, sh.cut[c]);
    }
    if (!(L > -kInf)) {
        if (rank == 0 && tid == 0) {
            st(&P.tokens[r], -1);
            if (P.logprob) st(&P.logprob[r], -kInf);
        }
        if (probs && open) write_zeros(R, probs);
        return;
    }
    if (L == kInf) {  // the tokens at +inf share the row
        R.inf = true;
        R.plain = false;
        L = cut = 0.0f;
        __syncthreads();
        for (int g = 0; g < kGroups; ++g) {
            float *at = room.peaks + g * kThreads + tid;
            *at = *at == kInf ? 0.0f : -kInf;
        }
    }
    keep.L = L;
    Exchange ex{sh, rank, cluster, 0};
    if (open) {
        draw_row<true>(P, R, r, u, keep, ex);
        return;
    }
    if (mass) {
        // the row's weight, to a part in kSure, and the candidates' exactly: where these reach the share
        // for sure, the leader draws from the list, unless a border between its tokens lies so near to
        // the share that this precision does not tell
        collect<true>(R, cut, room, part, rank, cluster, keep, false, sh);
        // the lanes' sums against the row's largest (a lane of tokens at +inf holds their number)
        const float own = R.inf ? (peak == kInf ? sum : 0.0f) : peak > -kInf ? sum * sv::ex2_approx((peak - L) * scale) : 0.0f;
        const u64 near = ex.sum(warp_sum(__float2ull_rn(own * 0x1p+40f)));
        Share share{true, share_of(p, near - near / kSure), share_of(p, near + near / kSure + 1)};
        if (scale == FLT_MAX) {  // (log2 e / T beyond that: the sums are of other powers)
            share.least = 0;
            share.most = ~0ull;
        }
        u64 listed = 0;
        for (int c = 0; c < cluster; ++c) listed += sh.listed[c];
        if (cut == -FLT_MAX) share.least = share.most = share_of(p, listed);  // (the whole row is listed)
        const bool fits = all_listed(sh, cluster, part, &total);
        if (fits && listed >= share.most) {
            if (rank == 0) {
                const bool done = finish_list<T>(P, r, room.list, room.work, part, total, 0, true, p, share, u, keep, sh);
                if (tid < cluster) put(remote(&sh.fits, tid), static_cast<unsigned>(done));
            }
            cluster_sync();
            if (sh.fits) return;
            if (rank == 0 && tid < cluster) sh.count[tid] = tid == 0 ? static_cast<unsigned>(total) : 0;  // (it closed the list up)
        }
        if (fits && listed >= share.least) {  // too near to tell: exactly, then
            share.least = share.most = share_of(p, ex.sum(warp_weight<true>(R, keep)));
            if (listed >= share.least) {
                if (rank == 0) finish_list<T>(P, r, room.list, room.work, part, total, 0, true, p, share, u, keep, sh);
                return;
            }
        }
        // (what lies so low that V tokens there hold no more than the rest is not looked through)
        const float lowest = sv::log_f32(static_cast<float>(P.V) / ((1.0f - p) * as_sum(near))) + 0.1f;
        const Known known{fits ? cut : kInf, lowest, as_sum(near), fits ? listed : 0};
        call_wide(P, R, r, p, u, keep, known, room, ex);
        return;
    }
    if (k > 0) {
        const unsigned key = call_kth(R, keep, static_cast<u64>(k), room, ex);
        if (key) keep.tau = of_key(key);
        if (p < 1.0f) call_wide(P, R, r, p, u, keep, Known{kInf, kSpan, 0.0f, 0}, room, ex);
        else draw_row<false>(P, R, r, u, keep, ex);
        return;
    }
    // min-p alone
    const float span = keep.low / keep.inv;
    cut = fmaxf(L + span - 4e-6f * (fabsf(L) + fabsf(span)), -FLT_MAX);
    collect<false>(R, cut, room, part, rank, cluster, keep, false, sh);
    cluster_sync();
    if (!all_listed(sh, cluster, part, &total)) draw_row<false>(P, R, r, u, keep, ex);
    else if (rank == 0) finish_list<T>(P, r, room.list, room.work, part, total, 0, true, p, Share{}, u, keep, sh);
}

// ---------------------------------------------------------------------------------------
// log-probabilities
// ---------------------------------------------------------------------------------------
// The token wanted of row r: tokens[r], or with prefix sums of the draft lengths the entry of the
// verification output [num_reqs, token_stride] that row r is the logits of (row cu[i] + i + j is
// position j of request i). A search by every warp, 32 places at a time; it stays in [0, num_reqs)
// whatever cu holds.
__device__ __forceinline__ int row_token(const LogprobParams &P, long long r)
{
    if (!P.cu) return ld(P.tokens + r);
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = P.num_reqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
        const bool before = lane == 0 || (at < hi && static_cast<long long>(ld(P.cu + at)) + at <= r);
        lo += (31 - __clz(static_cast<int>(__ballot_sync(0xFFFFFFFFu, before)))) * step;
        hi = min(hi, lo + step);
    }
    const long long j = r - ld(P.cu + lo) - lo;
    return j >= 0 && j < P.token_stride ? ld(P.tokens + static_cast<long long>(lo) * P.token_stride + j) : -1;
}

__device__ __forceinline__ u64 pack(float a, float b)
{
    return (static_cast<u64>(__float_as_uint(a)) << 32) | __float_as_uint(b);
}

static_assert(SV_MAX_TOP <= kList / kMaxCluster / 8 * 5, "every CTA can list its own best tokens");

// Each lane sums 2^((l - m) / T log2 e) over its logits against a reference m and counts the logits above
// the token's; a warp joins its lanes' sums against its largest logit, the leader the warps'. The best
// tokens come from the list of those from the cut on that num_top lane maxima reach, each put by the
// leader in the place that the number of larger ones gives it.
// Without best tokens no row is read again, and a fifth block on an SM, with half the vectors read
// ahead, hides more than the second look at rows that no longer fit the L2 cache costs (640x40003
// float32 23 against 30 us; with 5 best of 1536x151936 bf16 78 against 69).
template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, kTop ? kCtas : kCtas + 1) sv_logprobs_kernel(const T *logits, LogprobParams P)
{
    constexpr int n = Vec<T>::n, ahead = kTop ? kAhead : kAhead / 2;
    extern __shared__ uint4 store[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, cluster = P.cluster, top = kTop ? P.num_top : 0;
    const unsigned rank = cluster_rank();
    const long long r = blockIdx.x / cluster;
    const T *row = logits + r * P.stride;
    const Room room(store);
    const int token = P.tokens ? row_token(P, r) : 0;
    const bool wanted = token >= 0 && token < P.V;
    if (!wanted) {
        if (rank != 0) return;
        if (tid == 0 && P.logprob) st(&P.logprob[r], -kInf);
        if (tid == 0 && P.rank) st(&P.rank[r], 0);
        for (int i = tid; i < top; i += kThreads) {
            st(&P.top_ids[r * top + i], -1);
            st(&P.top_logprob[r * top + i], -kInf);
        }
        return;
    }
    cluster_announce();  // (waited for before the first write to another CTA: that it runs by then)
    const Row<T> R = start_row(row, P.V, P.split, rank, sh);
    const float lt = fmaxf(as_float(ld(row + token)), -kInf);  // (NaN as -inf)
    const float temp = P.temperature ? ld(P.temperature + r) : 1.0f;
    const float inv = temp > 0.0f ? inverse(fmaxf(temp, FLT_MIN)) : 1.0f;
    const float scale = inv * kLog2e;
    // Some vectors at a time, against a reference that moves to the largest logit only once that is kRise
    // above it: each move rounds what was added before, and where logits rise a little all along the row
    // those errors would add up (moved each time, -13.1639 was off by 6.8e-6 after 128 moves). Batches
    // are added by Kahan's compensated summation: a batch far smaller than the sum would otherwise
    // round it the same way each time (-0.0257 off by 3.1e-6). Together they cost 2 to 4 %. The logit from
    // which the reference moves is held in a register where float32 rows are read once and found anew for
    // each batch elsewhere: 512x128256 float32 50 against 58 us, 640x151936 bf16 46 against 44.5, with 5
    // best tokens 65 against 57.
    constexpr bool held = !kTop && sizeof(T) == 4;
    float peak = -kInf, ref = -kInf, limit = -kInf, s = 0.0f, lost = 0.0f;
    const float up = held ? kRise / scale : 0.0f;
    Above<T> above(lt);
    R.template each<ahead>([&](uint4 (&v)[ahead], int m, int c) {
        Largest<T> largest;
#pragma unroll
        for (int i = 0; i < ahead; ++i) largest.add(v[i]);
        const float own = largest.get();
        if (kTop) {
            float *at = room.peaks + (c % kGroups) * kThreads + tid;
            *at = c < kGroups ? own : fmaxf(*at, own);
        }
        peak = fmaxf(peak, own);
        if (held ? own > limit : (own - ref) * scale > kRise) {
            const float f = sv::ex2_approx((ref - own) * scale);  // (of the first reference, -inf, 0)
            s *= f;
            lost *= f;
            ref = own;
            if (held) limit = own < kInf ? fminf(own + up, FLT_MAX) : kInf;  // (+inf moves it in any case, once)
        }
        const float batch = __fadd_rn(fast_sum<T>(v, m, ref, scale), lost);
#pragma unroll
        for (int i = 0; i < ahead; ++i)
            if (i < m) above.add(v[i]);
        above.flush();
        const float sum = __fadd_rn(s, batch);
        lost = __fsub_rn(batch, __fsub_rn(sum, s));
        s = sum;
    });
    s += lost;
    const float top_of_warp = warp_max(peak);
    if (ref < top_of_warp && s > 0.0f) s *= sv::ex2_approx((ref - top_of_warp) * scale);
#pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
    const unsigned larger = __reduce_add_sync(0xFFFFFFFFu, above.get());
    cluster_wait();
    if (R.lane == 0) {
        put(remote(&sh.seg[0][rank * kWarps + R.warp], 0), pack(top_of_warp, s));
        put(remote(&sh.seg[1][rank * kWarps + R.warp], 0), static_cast<u64>(larger));
    }
    const int part = kList / cluster;
    if (kTop) {
        const float largest = block_max(peak, sh);
        const float cut = largest > -kInf && largest < kInf ? cut_for<T>(peak, largest, top, top + (top >> 2), sh) : -FLT_MAX;
        collect<false>(R, cut, room, part, rank, cluster, Kept{}, true, sh);
    }
    cluster_sync();
    float L = -kInf;
    float norm = 0.0f;
    if (rank == 0) {
        u64 rank_sum = 0;
        for (int i = R.lane; i < cluster * kWarps; i += 32) {
            L = fmaxf(L, __uint_as_float(static_cast<unsigned>(sh.seg[0][i] >> 32)));
            rank_sum += sh.seg[1][i];
        }
        L = warp_max(L);
        rank_sum = warp_sum(rank_sum);
        float sum = 0.0f;
        for (int i = R.lane; i < cluster * kWarps; i += 32) {
            const float mw = __uint_as_float(static_cast<unsigned>(sh.seg[0][i] >> 32));
            const float sw = __uint_as_float(static_cast<unsigned>(sh.seg[0][i]));
            if (mw > -kInf) sum += mw == L ? sw : sw * sv::exp_f32((mw - L) * inv);
        }
#pragma unroll
        for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
        norm = sv::log_f32(sum);
        if (tid == 0) {
            const float d = lt == L ? 0.0f : (lt - L) * inv;
            if (P.logprob) st(&P.logprob[r], lt > -kInf ? d - norm : -kInf);
            if (P.rank) st(&P.rank[r], 1 + static_cast<int>(rank_sum));
        }
    }
    if (!kTop) return;
    auto write = [&](int i, u64 entry) {
        const auto index = static_cast<int>(~static_cast<unsigned>(entry));
        const float l = entry ? of_key(static_cast<unsigned>(entry >> 32)) : -kInf;
        const float d = l == L ? 0.0f : (l - L) * inv;
        st(&P.top_ids[r * top + i], entry ? index : -1);
        st(&P.top_logprob[r * top + i], entry ? d - norm : -kInf);
    };
    int total;
    if (all_listed(sh, cluster, part, &total)) {
        if (rank != 0) return;
        // an entry's place is the number of larger ones; past the row's tokens nothing is left
        for (int i = total + tid; i < top; i += kThreads) write(i, 0);
        u64 mine[kList / kThreads];
#pragma unroll
        for (int q = 0; q < kList / kThreads; ++q) {
            mine[q] = tid + q * kThreads < total ? listed_entry(room.list, part, cluster, sh, tid + q * kThreads) : 0;
            if (mine[q]) room.work[tid + q * kThreads] = mine[q];
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kList / kThreads; ++q)
            if (mine[q]) {
                int place = 0;
                for (int j = 0; j < total; ++j) place += room.work[j] > mine[q];
                if (place < top) write(place, mine[q]);
            }
        return;
    }
    // more ties than the list holds: one token after the other
    cluster_sync();  // (the leader has read what the warps sent)
    Exchange ex{sh, rank, cluster, 0};
    u64 last = ~0ull;
    for (int i = 0; i < top; ++i) {
        u64 best = 0;
        for (int j = R.lo + R.lane; j < R.hi; j += 32) {
            float f[n];
            Vec<T>::get(R.get(j), f);
#pragma unroll
            for (int e = 0; e < n; ++e) {
                const unsigned key = key_of(f[e]);
                const u64 c = (static_cast<u64>(key) << 32) | static_cast<unsigned>(~static_cast<unsigned>(R.base + j * n + e));
                if (key && c < last && c > best) best = c;
            }
        }
#pragma unroll
        for (int k = 16; k; k >>= 1) {
            const u64 o = __shfl_xor_sync(0xFFFFFFFFu, best, k);
            best = o > best ? o : best;
        }
        const u64 *v = ex.all(best);
        for (int c = 0; c < cluster * kWarps; ++c) best = v[c] > best ? v[c] : best;
        last = best;
        if (rank == 0 && tid == 0) write(i, best);
    }
}

