// sample.hip -- drawing a token a row from logits, with temperature, top-k, top-p and min-p,
// from given uniform numbers, for gfx950: the end of a draft step and of a verify step.
//
//     w_i = exp((logit_i - max) / T)
//     order the tokens by (logit descending, index ascending);
//     keep the first k;  of these the shortest prefix whose weights sum to at least
//     top_p times theirs (at least one token);  of these the ones with w_i >= min_p
//     token = the first index, in the order of the vocabulary, at which the running sum of
//     the kept weights passes u times their sum;  prob = w_token / that sum
//
// Which token a uniform number falls on is a comparison of long sums, so the weights are
// computed in binary64 and summed as integers, in units of 2^-44 of the largest weight: integer
// sums do not depend on the order of atomics, and the result is the same in every run.  2^19
// weights of at most 2^44 stay below 2^63.
//
// Nothing is sorted.  Both cuts keep a prefix of the order, so the kept tokens are those up to
// one (logit, index) pair.  Three passes over the logits, the second and third mostly from the
// caches:
//   1. the row's largest logit;
//   2. counts and weight sums by bins of 1/128 nat below the largest (rows with a cut only):
//      the bins in which the cuts fall;
//   3. weight sums of the tokens above those bins, and the few tokens inside them (pairs in a
//      list), whose exact ranks give the cut; then the token.
// Each row is split into chunks over workgroups; the last workgroup of a row to arrive does
// the row's serial part (at pass 2: scanning 4096 bins, at pass 3: the cut and the draw, which
// re-reads one chunk).
#include "internal.h"

using namespace w4host;
using namespace w4dev;

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 4096;            // the last one also takes all that lies further below
constexpr float kBinsPerNat = 128.0f;  // 32 nats: a weight below 2^-46 of the largest rounds to 0
constexpr int kList = 2048;            // tokens of the cuts' bins that a row's list holds
constexpr double kUnit = 17592186044416.0;  // 2^44
constexpr int64_t kMaxV = 1 << 19;
constexpr int kMaxChunks = 64;
constexpr int64_t kRows = 1024;        // rows of one set of launches (their scratch is 50 KB each)

// What pass 2 leaves for pass 3.
struct RowCut {
    int sure_end;        // bins below this are kept by top-k and top-p
    int lo, hi;          // bins in which the top-p cut may fall (lo > hi: none)
    int bin_k;           // bin of the top-k cut (-1: none)
    unsigned left_k;     // tokens that top-k keeps of bin_k
    unsigned long long sum_before_lo, sum_before_k, sum_all;
};

struct SampleParams {
    const void *logits;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int32_t *token;
    float *prob;
    int64_t stride;
    int V, chunks, chunk_len;
    // workspace
    unsigned *arrive;            // [2][B], zero between calls
    unsigned long long *top;     // [B][kMaxChunks] largest (logit, index) of each chunk
    unsigned long long *sums;    // [B][kMaxChunks] kept weight of each chunk, above the cuts' bins
    unsigned long long *hist_w;  // [B][kBins]
    unsigned *hist_n;            // [B][kBins]
    unsigned long long *list;    // [B][kList]
    unsigned *listed;            // [B]
    RowCut *cut;                 // [B]
};

// Device-coherent accesses: what a workgroup leaves for another one of the same launch.
template <typename T>
__device__ __forceinline__ void put(T *p, T v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T get(const T *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The order of the tokens as one integer, smaller first: logit descending, index ascending.
// (-0 and +0 are equal: -0 takes +0's place.)
__device__ __forceinline__ unsigned long long place_of(float l, int i)
{
    uint32_t b = __builtin_bit_cast(uint32_t, l == 0.f ? 0.f : l);
    b = (b & 0x80000000u) ? b : ~b & 0x7FFFFFFFu;
    return ((unsigned long long)b << 32) | (unsigned)i;
}
__device__ __forceinline__ float logit_of(unsigned long long place)
{
    uint32_t b = (uint32_t)(place >> 32);
    b = (b & 0x80000000u) ? b : ~b & 0x7FFFFFFFu;
    return __builtin_bit_cast(float, b);
}

template <bool F32>
__device__ __forceinline__ float logit_at(const void *row, int i)
{
    const float l = load_one<F32>(row, i);
    return l == l ? l : -__builtin_huge_valf();  // a NaN is never drawn
}

// Four logits from element e (a multiple of 4), -inf past the end.
template <bool F32, bool VEC>
__device__ __forceinline__ f32x4 logits4(const void *row, int e, int end)
{
    const float none = -__builtin_huge_valf();
    f32x4 v = {none, none, none, none};
    if (VEC && e + 4 <= end) {
        if (F32) {
            v = *(const f32x4 *)((const float *)row + e);
        } else {
            const u32x2 r = *(const u32x2 *)((const uint16_t *)row + e);
            v = f32x4{bf16_lo(r[0]), bf16_hi(r[0]), bf16_lo(r[1]), bf16_hi(r[1])};
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v[j] != v[j]) v[j] = none;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e + j < end) v[j] = logit_at<F32>(row, e + j);
    }
    return v;
}

struct Row {
    float top, bin_scale;
    double inv_t;
    float min_p;
};

// Bin of a logit: monotone in it, since each binary32 step is.
__device__ __forceinline__ int bin_of(float l, const Row &r)
{
    if (l == r.top) return 0;
    const float b = (r.top - l) * r.bin_scale;
    return b < (float)(kBins - 1) ? (int)b : kBins - 1;  // infinite or NaN (infinity * 0): the last
}

// exp((l - top) / T) of a logit outside the last bin, so the argument lies in (-33, 0].  The
// same weight is computed in several places and has to come out with the same bits, so every
// step is spelled out: x = n ln 2 + f with |f| <= ln 2 / 2, the exponential series of f to its
// 12th power (the first term left out is below 2e-16), and n added to the exponent.
__device__ __forceinline__ double weight_of(float l, const Row &r)
{
#pragma clang fp contract(off)
    if (l == r.top) return 1.0;
    const double x = ((double)l - (double)r.top) * r.inv_t;
    const double n = __builtin_rint(x * 1.4426950408889634);
    const double f = __builtin_fma(n, -1.9082149292705877e-10, __builtin_fma(n, -0.6931471803691238, x));
    double s = 1.0 / 479001600.0;
    s = __builtin_fma(s, f, 1.0 / 39916800.0);
    s = __builtin_fma(s, f, 1.0 / 3628800.0);
    s = __builtin_fma(s, f, 1.0 / 362880.0);
    s = __builtin_fma(s, f, 1.0 / 40320.0);
    s = __builtin_fma(s, f, 1.0 / 5040.0);
    s = __builtin_fma(s, f, 1.0 / 720.0);
    s = __builtin_fma(s, f, 1.0 / 120.0);
    s = __builtin_fma(s, f, 1.0 / 24.0);
    s = __builtin_fma(s, f, 1.0 / 6.0);
    s = __builtin_fma(s, f, 0.5);
    s = __builtin_fma(s, f, 1.0);
    s = __builtin_fma(s, f, 1.0);
    return __builtin_ldexp(s, (int)n);
}
// A weight in units of 2^-44 of the largest, and the same with min-p applied.
__device__ __forceinline__ unsigned long long fixed(double w)
{
    return (unsigned long long)__builtin_fma(w, kUnit, 0.5);
}
__device__ __forceinline__ unsigned long long drawn_weight(float l, const Row &r)
{
    const double w = weight_of(l, r);
    return w >= (double)r.min_p ? fixed(w) : 0ull;
}

__device__ __forceinline__ unsigned long long wave_sum(unsigned long long v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
__device__ __forceinline__ unsigned long long wave_scan(unsigned long long v, int lane)  // inclusive
{
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const unsigned long long o = __shfl_up(v, off, 64);
        if (lane >= off) v += o;
    }
    return v;
}

// Sum over the workgroup, in every thread.
__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, unsigned long long *s)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v += s[i];
    return v;
}
__device__ __forceinline__ unsigned long long block_min(unsigned long long v, unsigned long long *s)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const unsigned long long o = __shfl_xor(v, off, 64);
        v = o < v ? o : v;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) v = s[i] < v ? s[i] : v;
    return v;
}

// Whether this workgroup is the last of the row's `chunks` to arrive.  The workgroup's
// coherent stores and atomics are complete before its count, and the last one's loads come
// after all counts.
__device__ __forceinline__ bool last_to_arrive(unsigned *count, int chunks, unsigned *s_last)
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *s_last = before == (unsigned)(chunks - 1);
        if (*s_last) {
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
            put(count, 0u);  // ready for the next call
        }
    }
    __syncthreads();
    return *s_last != 0;
}

__device__ __forceinline__ unsigned long long row_top(const SampleParams &p, int b)
{
    unsigned long long best = ~0ull;
    for (int c = 0; c < p.chunks; ++c) {
        const unsigned long long v = p.top[(int64_t)b * kMaxChunks + c];
        best = v < best ? v : best;
    }
    return best;
}

__device__ __forceinline__ Row row_of(const SampleParams &p, int b, float top, float t)
{
    Row r;
    r.top = top;
    r.inv_t = 1.0 / (double)t;
    r.bin_scale = kBinsPerNat / t;
    const float m = p.min_p ? p.min_p[b] : 0.f;
    r.min_p = m > 0.f ? fminf(m, 1.f) : 0.f;
    return r;
}

__device__ __forceinline__ const void *row_ptr(const SampleParams &p, int b, bool f32)
{
    return (const char *)p.logits + (int64_t)b * p.stride * (f32 ? 4 : 2);
}

// ------------------------------------------------------------------------------------
// Pass 1: each chunk's largest (logit, lowest index); the row's bins cleared.

template <bool F32, bool VEC>
__global__ __launch_bounds__(kThreads) void sample_top_kernel(const SampleParams p, bool clear)
{
    __shared__ unsigned long long s[kWaves];
    const int c = blockIdx.x, b = blockIdx.y;
    const int begin = c * p.chunk_len, end = min(p.V, begin + p.chunk_len);
    const void *row = row_ptr(p, b, F32);
    unsigned long long best = ~0ull;
#pragma unroll 4
    for (int e = begin + threadIdx.x * 4; e < end; e += kThreads * 4) {
        const f32x4 l = logits4<F32, VEC>(row, e, end);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned long long v = place_of(l[j], e + j);
            best = v < best ? v : best;
        }
    }
    best = block_min(best, s);
    if (threadIdx.x == 0) p.top[(int64_t)b * kMaxChunks + c] = best;
    if (clear) {
        const int share = (kBins + p.chunks - 1) / p.chunks;
        for (int i = c * share + threadIdx.x; i < min(kBins, (c + 1) * share); i += kThreads) {
            p.hist_w[(int64_t)b * kBins + i] = 0ull;
            p.hist_n[(int64_t)b * kBins + i] = 0u;
        }
    }
    if (c == 0 && threadIdx.x == 0) p.listed[b] = 0u;
}

// ------------------------------------------------------------------------------------
// Pass 2: counts and weight sums by bins, and the bins of the cuts.

template <bool F32, bool VEC>
__global__ __launch_bounds__(kThreads) void sample_bins_kernel(const SampleParams p)
{
    __shared__ unsigned long long s_w[kBins];
    __shared__ unsigned s_n[kBins];
    __shared__ unsigned long long s_scan[kWaves];
    __shared__ unsigned s_scan_n[kWaves];
    __shared__ unsigned s_last;
    __shared__ int s_bin_k, s_lo, s_hi;
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const float t = p.temperature ? p.temperature[b] : 1.f;
    const int k = p.top_k ? p.top_k[b] : 0;
    const float top_p = p.top_p ? p.top_p[b] : 1.f;
    const bool cut_k = k > 0 && k < p.V, cut_p = top_p < 1.f;
    if (!(t > 0.f) || (!cut_k && !cut_p)) return;  // no cut in this row
    const float top = logit_of(row_top(p, b));
    if (top == -__builtin_huge_valf()) return;     // nothing to draw
    const Row r = row_of(p, b, top, t);
    for (int i = tid; i < kBins; i += kThreads) {
        s_w[i] = 0ull;
        s_n[i] = 0u;
    }
    __syncthreads();
    const int begin = c * p.chunk_len, end = min(p.V, begin + p.chunk_len);
    const void *row = row_ptr(p, b, F32);
    for (int e = begin + tid * 4; e < end; e += kThreads * 4) {
        const f32x4 l = logits4<F32, VEC>(row, e, end);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (e + j >= end) break;
            const int bin = bin_of(l[j], r);
            if (bin == kBins - 1) continue;  // weighs nothing; counted as the rest
            atomicAdd(&s_n[bin], 1u);
            if (cut_p) atomicAdd(&s_w[bin], fixed(weight_of(l[j], r)));
        }
    }
    __syncthreads();
    for (int i = tid; i < kBins; i += kThreads) {
        if (!s_n[i]) continue;
        __hip_atomic_fetch_add(p.hist_n + (int64_t)b * kBins + i, s_n[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (cut_p)
            __hip_atomic_fetch_add(p.hist_w + (int64_t)b * kBins + i, s_w[i], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!last_to_arrive(p.arrive + b, p.chunks, &s_last)) return;

    // four bins a thread: exclusive sums before them
    constexpr int kPer = kBins / kThreads;
    const int lane = tid & 63, wave = tid >> 6;
    unsigned n[kPer], n_before = 0;
    unsigned long long w[kPer], w_before = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        n[i] = get(p.hist_n + (int64_t)b * kBins + tid * kPer + i);
        w[i] = cut_p ? get(p.hist_w + (int64_t)b * kBins + tid * kPer + i) : 0ull;
        n_before += n[i];
        w_before += w[i];
    }
    const unsigned n_own = n_before;
    const unsigned long long w_own = w_before;
    w_before = wave_scan(w_before, lane);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const unsigned o = (unsigned)__shfl_up((int)n_before, off, 64);
        if (lane >= off) n_before += o;
    }
    if (lane == 63) {
        s_scan[wave] = w_before;
        s_scan_n[wave] = n_before;
    }
    if (tid == 0) s_bin_k = -1, s_lo = kBins, s_hi = kBins;
    __syncthreads();
    unsigned long long w_all = 0;
    for (int i = 0; i < kWaves; ++i) {
        if (i < wave) {
            w_before += s_scan[i];
            n_before += s_scan_n[i];
        }
        w_all += s_scan[i];
    }
    n_before -= n_own;
    w_before -= w_own;
    RowCut *cut = p.cut + b;
    if (tid == 0) cut->sum_all = w_all;
    // the bin in which the k-th token lies (none: it lies where nothing weighs anything)
    __shared__ unsigned long long s_w1[2];
    if (tid == 0) s_w1[0] = s_w1[1] = w_all;
    __syncthreads();
    if (cut_k) {
        unsigned nb = n_before;
        unsigned long long wb = w_before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (nb < (unsigned)k && nb + n[i] >= (unsigned)k) {
                s_bin_k = tid * kPer + i;
                cut->left_k = (unsigned)k - nb;
                cut->sum_before_k = wb;
                s_w1[0] = wb;
                s_w1[1] = wb + w[i];
            }
            nb += n[i];
            wb += w[i];
        }
    }
    __syncthreads();
    // the bins in which the top-p cut lies, for the least and the most that top-k may keep
    if (cut_p) {
        const double pp = (double)fmaxf(top_p, 0.f);
        const double want0 = pp * (double)s_w1[0], want1 = pp * (double)s_w1[1];
        unsigned long long wb = w_before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const double before = (double)wb, through = (double)(wb + w[i]);
            const int bin = tid * kPer + i;
            if ((before < want0 || bin == 0) && through >= want0) {
                s_lo = bin;
                cut->sum_before_lo = wb;
            }
            if ((before < want1 || bin == 0) && through >= want1) s_hi = bin;
            wb += w[i];
        }
    }
    __syncthreads();
    if (tid == 0) {
        cut->bin_k = s_bin_k;
        cut->lo = cut_p ? s_lo : kBins;
        cut->hi = cut_p ? s_hi : -1;
        cut->sure_end = cut_p ? (s_bin_k >= 0 ? min(s_lo, s_bin_k) : s_lo) : (s_bin_k >= 0 ? s_bin_k : kBins);
    }
}

// ------------------------------------------------------------------------------------
// Pass 3: the cut, and the draw.

template <bool F32, bool VEC>
__global__ __launch_bounds__(kThreads) void sample_draw_kernel(const SampleParams p)
{
    __shared__ unsigned long long s_place[kList];
    __shared__ unsigned long long s_wt[kList];
    __shared__ uint8_t s_in[kList];  // 1: in the bin of the top-k cut, 2: in those of the top-p cut
    __shared__ unsigned long long s[kWaves];
    __shared__ unsigned s_count, s_base, s_last;
    const int c = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const float none = -__builtin_huge_valf();
    const unsigned long long best = row_top(p, b);
    const float top = logit_of(best);
    const float t = p.temperature ? p.temperature[b] : 1.f;
    if (top == none || !(t > 0.f)) {  // nothing to draw, or the largest
        if (c == 0 && tid == 0) {
            p.token[b] = top == none ? -1 : (int32_t)(uint32_t)best;
            if (p.prob) p.prob[b] = top == none ? 0.f : 1.f;
        }
        return;
    }
    const int k = p.top_k ? p.top_k[b] : 0;
    const float top_p = p.top_p ? p.top_p[b] : 1.f;
    const bool cut_k = k > 0 && k < p.V, cut_p = top_p < 1.f;
    const Row r = row_of(p, b, top, t);
    RowCut cut;
    if (cut_k || cut_p)
        cut = p.cut[b];
    else
        cut.sure_end = kBins, cut.lo = kBins, cut.hi = -1, cut.bin_k = -1;
    auto inside = [&](int bin) { return (bin >= cut.lo && bin <= cut.hi) || bin == cut.bin_k; };
    const int begin = c * p.chunk_len, end = min(p.V, begin + p.chunk_len);
    const void *row = row_ptr(p, b, F32);
    if (tid == 0) s_count = 0u;
    __syncthreads();
    unsigned long long mine = 0;
    for (int e = begin + tid * 4; e < end; e += kThreads * 4) {
        const f32x4 l = logits4<F32, VEC>(row, e, end);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (e + j >= end) break;
            const int bin = bin_of(l[j], r);
            if (bin == kBins - 1) continue;
            if (bin < cut.sure_end) {
                mine += drawn_weight(l[j], r);
            } else if (inside(bin)) {
                const unsigned at = atomicAdd(&s_count, 1u);
                if (at < kList) s_place[at] = place_of(l[j], e + j);
            }
        }
    }
    mine = block_sum(mine, s);
    if (tid == 0) {
        put(p.sums + (int64_t)b * kMaxChunks + c, mine);
        s_base = s_count ? __hip_atomic_fetch_add(p.listed + b, s_count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0u;
    }
    __syncthreads();
    for (unsigned i = tid; i < min(s_count, (unsigned)kList); i += kThreads)
        if (s_base + i < kList) put(p.list + (int64_t)b * kList + s_base + i, s_place[i]);
    if (!last_to_arrive(p.arrive + gridDim.y + b, p.chunks, &s_last)) return;

    // The cut: the last place that is kept.  ~0: all of them, as without cuts.
    unsigned long long last_place = ~0ull;
    const unsigned listed = get(p.listed + b);
    const double pp = (double)fmaxf(top_p, 0.f);
    if (cut.bin_k >= 0 || cut.hi >= 0) {
        if (listed <= kList) {
            for (unsigned i = tid; i < listed; i += kThreads) {
                const unsigned long long at = get(p.list + (int64_t)b * kList + i);
                const int bin = bin_of(logit_of(at), r);
                s_place[i] = at;
                s_wt[i] = fixed(weight_of(logit_of(at), r));
                s_in[i] = (bin == cut.bin_k ? 1 : 0) | (bin >= cut.lo && bin <= cut.hi ? 2 : 0);
            }
            __syncthreads();
            constexpr int kPer = kList / kThreads;
            unsigned rank_k[kPer] = {};
            unsigned long long before_p[kPer] = {}, w1 = 0;
            bool in_k[kPer] = {}, in_p[kPer] = {};
            // ranks and sums before each listed token, by comparing it with every other one
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const unsigned me = tid + i * kThreads;
                if (me >= listed) continue;
                const unsigned long long at = s_place[me];
                in_k[i] = s_in[me] & 1;
                in_p[i] = s_in[me] & 2;
                for (unsigned o = 0; o < listed; ++o) {
                    const bool earlier = s_place[o] < at;
                    rank_k[i] += earlier && (s_in[o] & 1);
                    before_p[i] += earlier && (s_in[o] & 2) ? s_wt[o] : 0ull;
                }
                if (in_k[i] && rank_k[i] < cut.left_k) w1 += s_wt[me];
            }
            w1 = block_sum(w1, s);
            const double want = pp * (double)(cut.bin_k >= 0 ? cut.sum_before_k + w1 : cut.sum_all);
            unsigned long long kept = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const unsigned me = tid + i * kThreads;
                if (me >= listed) continue;
                bool keep = true;
                if (cut.bin_k >= 0 && in_k[i]) keep = rank_k[i] < cut.left_k;
                if (cut_p) {
                    const unsigned long long before = cut.sum_before_lo + before_p[i];
                    keep = keep && in_p[i] && ((double)before < want || s_place[me] == best);
                }
                if (keep && s_place[me] > kept) kept = s_place[me];
            }
            last_place = ~block_min(~kept, s);
        } else {
            // More tokens in the cuts' bins than the list holds (thousands of equal or nearly
            // equal logits): halve the range of places until the cut is found, each step one
            // pass over the row.
            auto count_and_sum = [&](unsigned long long upto, int from, int to, unsigned long long *n_out,
                                     unsigned long long *w_out) {
                unsigned long long n = 0, w = 0;
                for (int e = tid * 4; e < p.V; e += kThreads * 4) {
                    const f32x4 l = logits4<F32, VEC>(row, e, p.V);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (e + j >= p.V || place_of(l[j], e + j) > upto) continue;
                        const int bin = bin_of(l[j], r);
                        if (bin < from || bin > to || bin == kBins - 1) continue;
                        ++n;
                        w += fixed(weight_of(l[j], r));
                    }
                }
                *n_out = block_sum(n, s);
                *w_out = block_sum(w, s);
            };
            unsigned long long n, w, lo, hi, kept = ~0ull;
            double all = (double)cut.sum_all;
            if (cut.bin_k >= 0) {
                // the smallest place with at least left_k tokens of bin_k up to it
                lo = best, hi = ~0ull;
                while (lo < hi) {
                    const unsigned long long mid = lo + (hi - lo) / 2;
                    count_and_sum(mid, cut.bin_k, cut.bin_k, &n, &w);
                    if (n >= cut.left_k)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                kept = lo;
                count_and_sum(kept, cut.bin_k, cut.bin_k, &n, &w);
                all = (double)(cut.sum_before_k + w);
            }
            if (cut_p) {
                // the smallest place up to which the weights reach top_p
                const double want = pp * all;
                lo = best, hi = kept;
                while (lo < hi) {
                    const unsigned long long mid = lo + (hi - lo) / 2;
                    count_and_sum(mid, cut.lo, cut.hi, &n, &w);
                    if ((double)(cut.sum_before_lo + w) >= want)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                kept = lo;
            }
            last_place = kept;
        }
    }

    // Kept weights of the cuts' bins join their chunks' sums.
    __shared__ unsigned long long s_sum[kMaxChunks];
    __syncthreads();
    if (tid < p.chunks) s_sum[tid] = get(p.sums + (int64_t)b * kMaxChunks + tid);
    __syncthreads();
    const bool cuts = cut.bin_k >= 0 || cut.hi >= 0;
    if (cuts && listed <= kList) {
        for (unsigned i = tid; i < listed; i += kThreads)
            if (s_place[i] <= last_place)
                atomicAdd(&s_sum[(uint32_t)s_place[i] / (unsigned)p.chunk_len], drawn_weight(logit_of(s_place[i]), r));
    } else if (cuts) {
        for (int e = tid; e < p.V; e += kThreads) {
            const float l = logit_at<F32>(row, e);
            const int bin = bin_of(l, r);
            if (bin != kBins - 1 && bin >= cut.sure_end && place_of(l, e) <= last_place)
                atomicAdd(&s_sum[e / p.chunk_len], drawn_weight(l, r));
        }
    }
    __syncthreads();
    // The chunk in which the running sum passes the target, then the wave's segment of that
    // chunk, then the token.  A target that rounding or u >= 1 puts past the end takes the last
    // token that weighs anything.
    unsigned long long total = 0;
    for (int i = 0; i < p.chunks; ++i) total += s_sum[i];
    const double u = (double)p.u[b];
    const double real = u > 0.0 ? u * (double)total : 0.0;
    unsigned long long target = real < (double)total ? (unsigned long long)real : total;
    if (target >= total) target = total - 1;  // drawn where the running sum first exceeds target
    int pick = 0;
    while (pick < p.chunks - 1 && target >= s_sum[pick]) target -= s_sum[pick++];
    const int cb = pick * p.chunk_len, ce = min(p.V, cb + p.chunk_len);
    const int seg = ((ce - cb + kWaves - 1) / kWaves + 63) / 64 * 64;
    const int sb = min(ce, cb + wave * seg), se = min(ce, sb + seg);
    auto kept_weight = [&](int e) -> unsigned long long {
        if (e >= se) return 0ull;
        const float l = logit_at<F32>(row, e);
        const int bin = bin_of(l, r);
        if (bin == kBins - 1 || (bin >= cut.sure_end && place_of(l, e) > last_place)) return 0ull;
        return drawn_weight(l, r);
    };
    unsigned long long part = 0;
    for (int e = sb + lane; e < se; e += 64) part += kept_weight(e);
    part = wave_sum(part);
    __syncthreads();
    if (lane == 0) s[wave] = part;
    __syncthreads();
    unsigned long long before = 0;
    for (int i = 0; i < wave; ++i) before += s[i];
    if (target < before || target >= before + part) return;  // another wave's segment
    target -= before;
    for (int e = sb; e < se; e += 64) {
        const unsigned long long w = kept_weight(e + lane);
        const unsigned long long run = wave_scan(w, lane);
        const unsigned long long whole = __shfl(run, 63, 64);
        if (target >= whole) {
            target -= whole;
            continue;
        }
        if (run > target && run - w <= target) {
            p.token[b] = e + lane;
            if (p.prob) p.prob[b] = (float)(weight_of(logit_at<F32>(row, e + lane), r) * kUnit / (double)total);
        }
        return;
    }
}

template <bool F32, bool VEC>
void launch_sample(const SampleParams &p, int64_t B, bool cuts, hipStream_t stream)
{
    const dim3 grid((unsigned)p.chunks, (unsigned)B), block(kThreads);
    hipLaunchKernelGGL((sample_top_kernel<F32, VEC>), grid, block, 0, stream, p, cuts);
    if (cuts) hipLaunchKernelGGL((sample_bins_kernel<F32, VEC>), grid, block, 0, stream, p);
    hipLaunchKernelGGL((sample_draw_kernel<F32, VEC>), grid, block, 0, stream, p);
}

}  // namespace

extern "C" {

w4_status w4_sample(const void *logits, int logits_type, int64_t row_stride, const float *u, const float *temperature,
                    const int32_t *top_k, const float *top_p, const float *min_p, int32_t *token, float *prob,
                    int64_t B, int64_t V, void *stream)
{
    if (logits_type != W4_F32 && logits_type != W4_BF16) {
        set_error("w4_sample: logits_type is neither W4_F32 nor W4_BF16");
        return W4_ERR_SHAPE;
    }
    if (B < 0 || B > 65535 || V < 1 || V > kMaxV || row_stride < V || row_stride > ((int64_t)1 << 32)) {
        set_error("w4_sample: shape B=%lld V=%lld row_stride=%lld: need 0<=B<=65535, 1<=V<=%lld, row_stride>=V",
                  (long long)B, (long long)V, (long long)row_stride, (long long)kMaxV);
        return W4_ERR_SHAPE;
    }
    if (B == 0) return W4_OK;
    if (!logits || !u || !token) {
        set_error("w4_sample: a required pointer is NULL");
        return W4_ERR_NULL;
    }
    const int size = logits_type == W4_F32 ? 4 : 2;
    if (!aligned(logits, size) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(token, 4) || !aligned(prob, 4)) {
        set_error("w4_sample: logits must be aligned to their type and the other arrays to 4 bytes");
        return W4_ERR_ALIGN;
    }
    int dev = -1;
    w4_status st = check_device(&dev);
    if (st != W4_OK) return st;
    const int64_t rows = B < kRows ? B : kRows;
    // about two workgroups a CU, and chunks of 4096 logits or more
    int64_t chunks = 512 / rows;
    if (chunks > V / 4096) chunks = V / 4096;
    if (chunks < 1) chunks = 1;
    if (chunks > kMaxChunks) chunks = kMaxChunks;
    const size_t words = (size_t)2 * kMaxChunks + kBins + kList;  // 8-byte words a row
    unsigned *count = nullptr;
    float *part = nullptr;
    st = get_workspace(dev, (hipStream_t)stream, (size_t)2 * rows,
                       (size_t)rows * (words * 8 + sizeof(RowCut) + (kBins + 1) * 4), &count, &part);
    if (st != W4_OK) return st;
    SampleParams p;
    p.stride = row_stride, p.V = (int)V;
    p.chunk_len = (int)(((V + chunks - 1) / chunks + 3) / 4 * 4);
    p.chunks = (int)((V + p.chunk_len - 1) / p.chunk_len);
    p.arrive = count;
    p.top = (unsigned long long *)part;
    p.sums = p.top + rows * kMaxChunks;
    p.hist_w = p.sums + rows * kMaxChunks;
    p.list = p.hist_w + rows * kBins;
    p.cut = (RowCut *)(p.list + rows * kList);
    p.hist_n = (unsigned *)(p.cut + rows);
    p.listed = p.hist_n + rows * kBins;
    const bool vec = aligned(logits, 16) && row_stride * size % 16 == 0;
    const bool cuts = top_k || top_p;
    for (int64_t b = 0; b < B; b += kRows) {
        const int64_t n = B - b < kRows ? B - b : kRows;
        p.logits = (const char *)logits + b * row_stride * size;
        p.u = u + b, p.token = token + b, p.prob = prob ? prob + b : nullptr;
        p.temperature = temperature ? temperature + b : nullptr, p.top_k = top_k ? top_k + b : nullptr;
        p.top_p = top_p ? top_p + b : nullptr, p.min_p = min_p ? min_p + b : nullptr;
        if (logits_type == W4_F32)
            vec ? launch_sample<true, true>(p, n, cuts, (hipStream_t)stream)
                : launch_sample<true, false>(p, n, cuts, (hipStream_t)stream);
        else
            vec ? launch_sample<false, true>(p, n, cuts, (hipStream_t)stream)
                : launch_sample<false, false>(p, n, cuts, (hipStream_t)stream);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_fail("w4_sample launch", e);
    return W4_OK;
}

}  // extern "C"
