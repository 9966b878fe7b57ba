// The best (beam, token) pairs of each request:
//   score(i, v) = scores[i] + x[i][v] - ln sum_u exp(x[i][u]),
// ordered by score descending, then i * V + v ascending.
//
// Two launches. The first reads the logits once, a CTA per stretch of up to
// 8192 of one beam's logits, which it holds in registers: their maximum, the
// sum of exp(x - max), and the stretch's best entries. The second, a CTA per
// request, forms the beams' normalisers and picks among the entries.
//
// The order has to be that of the numbers themselves, so everything that
// decides between beams is held in 64 bits: with scores near -20 an error of one fp32 rounding
// (2e-6) would swap neighbours of different beams once in a few hundred kept pairs. exp is
//   exp(d) = 2^(k/32) * (1 + r + r^2/2 + r^3/6 + r^4/24),  d = (k + f) ln2/32, r = f ln2/32, |r| <= ln2/64
// in fp64 (relative error below 2e-12 of a term): nine fp64 operations and two
// shuffles (the 32 powers sit one per lane).
//
// Best entries of a stretch: its threads' maxima go into a histogram between
// their least and largest; the bin edge with `keep` of them at or above it bounds
// the stretch's keep-th logit from below, so only the few logits above it are
// written. Where equal logits make them too many, a bisection over
// (logit, index) finds the exact border.
#include "decode.cuh"

namespace st {

constexpr int kSelThreads = 256;
constexpr int kSelPerThread = 32;
constexpr int kSelStretch = kSelThreads * kSelPerThread;
constexpr int kMergeThreads = 1024;
constexpr int kMergeCap = 2048;   // pairs sorted at the end
constexpr int kMergeUnits = 4096; // stretches listed as holding such pairs
constexpr int kHistBins = 256;

// One stretch's result.
struct Stretch {
    double sum;   // of exp(x - max)
    float max;    // -inf: no candidate
    int32_t count;  // entries written
};

// 2^(i/32), by the exponential series.
struct Powers32 {
    double v[32];
    constexpr Powers32() : v()
    {
        for (int i = 0; i < 32; ++i) {
            const double z = 0.693147180559945309417232121458 * i / 32;
            double s = 1, term = 1;
            for (int n = 1; n < 30; ++n) {
                term = term * z / n;
                s += term;
            }
            v[i] = s;
        }
    }
};
__device__ const Powers32 kPowers32{};

// order-preserving unsigned form of a float (no NaN)
__device__ __forceinline__ uint32_t float_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u ^ (u & 0x80000000u ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t double_key(double x)
{
    const uint64_t u = uint64_t(__double_as_longlong(x));
    return u ^ (u >> 63 ? ~0ull : 1ull << 63);
}

__device__ __forceinline__ float warp_max(float m)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}
__device__ __forceinline__ float warp_min(float m)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fminf(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}

template <typename T>
struct Logit;
template <>
struct Logit<float> {
    static constexpr int kPer = 4;  // per 16 bytes
    __device__ static void unpack(const uint4& w, float* x)
    {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
    __device__ static float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
};
template <>
struct Logit<__nv_bfloat16> {
    static constexpr int kPer = 8;
    __device__ static void unpack(const uint4& w, float* x)
    {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(a[i] << 16);
            x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
    }
    __device__ static float one(const void* p, int64_t i) { return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]); }
};
template <>
struct Logit<__half> {
    static constexpr int kPer = 8;
    __device__ static void unpack(const uint4& w, float* x)
    {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    __device__ static float one(const void* p, int64_t i) { return __half2float(static_cast<const __half*>(p)[i]); }
};

// The highest bin b such that bins 0..b hold at least `want`, -1 if all hold
// fewer; by the first warp, read by all after a barrier.
template <int BINS>
__device__ __forceinline__ void find_bin(const uint32_t* hist, uint32_t want, int* out)
{
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        constexpr int PER = BINS / 32;
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) mine += hist[lane * PER + i];
        uint32_t incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += t;
        }
        const unsigned reach = __ballot_sync(0xffffffffu, incl >= want);
        int bin = -1;
        if (reach && lane == __ffs(reach) - 1) {
            uint32_t c = incl - mine;
            for (int i = 0; i < PER; ++i) {
                c += hist[lane * PER + i];
                if (c >= want) {
                    bin = lane * PER + i;
                    break;
                }
            }
            *out = bin;
        }
        if (!reach && lane == 0) *out = -1;
    }
}

// A value's place in the histogram is (best - value) * inv; values not at or above `edge` there are kept
// (written so that an infinite range, with inv = 0, keeps them).
__device__ __forceinline__ float bin_scale(float range) { return range > 0.f ? fminf((kHistBins - 1) / range, 3e38f) : 0.f; }

template <typename T>
__global__ void __launch_bounds__(kSelThreads)
beam_stretch_kernel(SelectArgs a, int stretches, int cap, Stretch* res, uint2* lists)
{
    constexpr int PER = Logit<T>::kPer, VECS = kSelPerThread / PER;
    __shared__ float s_max[kSelThreads / 32], s_min[kSelThreads / 32];
    __shared__ double s_sum[kSelThreads / 32];
    __shared__ uint32_t s_hist[kHistBins];
    __shared__ int s_bin;
    __shared__ uint32_t s_count, s_total;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.y;
    const int b = int(row / a.K), i = int(row - int64_t(b) * a.K);
    const int64_t unit = row * stretches + blockIdx.x;
    uint2* list = lists + unit * cap;

    const float base = a.scores[row];
    const bool finished = a.ex.finished && a.ex.finished[row];
    if (!(fabsf(base) < INFINITY) || finished) {  // no logit counts
        if (tid == 0) {
            Stretch s{0.0, -INFINITY, 0};
            if (finished && fabsf(base) < INFINITY && blockIdx.x == 0) {  // one candidate of logit 0 with normaliser 0
                s = Stretch{1.0, 0.f, 1};
                list[0] = make_uint2(__float_as_uint(0.f), uint32_t(a.ex.end_token));
            }
            res[unit] = s;
        }
        return;
    }

    // Vectors of 16 aligned bytes; the first may begin before the row, the last end behind it.
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    const int before = int((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const int64_t first = int64_t(blockIdx.x) * kSelStretch - before;  // the row's index of the stretch's first element
    const uint32_t* allow = a.ex.allow ? a.ex.allow + b * a.ex.allow_request_stride + i * a.ex.allow_beam_stride : nullptr;
    const int words = (a.V + 31) / 32;
    float v[kSelPerThread];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
        const int64_t e = first + int64_t(j * kSelThreads + tid) * PER;
        float* y = v + j * PER;
        if (e >= 0 && e + PER <= a.V) {
            Logit<T>::unpack(__ldcs(reinterpret_cast<const uint4*>(x + e)), y);
        } else {
#pragma unroll
            for (int u = 0; u < PER; ++u) y[u] = e + u >= 0 && e + u < a.V ? Logit<T>::one(x, e + u) : -INFINITY;
        }
    }
    if (allow) {
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t e = first + int64_t(j * kSelThreads + tid) * PER;
            if (e + PER <= 0 || e >= a.V) continue;
            const int64_t at = e < 0 ? 0 : e;  // bits of elements at .. at + PER
            const int w = int(at >> 5);
            const uint32_t lo = allow[w], hi = w + 1 < words ? allow[w + 1] : 0u;
            uint32_t bits = __funnelshift_r(lo, hi, uint32_t(at & 31));
            bits <<= uint32_t(at - e);
#pragma unroll
            for (int u = 0; u < PER; ++u)
                if (!(bits >> u & 1u)) v[j * PER + u] = -INFINITY;
        }
    }
    float tmax = -INFINITY;
#pragma unroll
    for (int k = 0; k < kSelPerThread; ++k) {
        v[k] = v[k] < INFINITY ? v[k] + 0.f : -INFINITY;  // NaN and +inf leave; -0 becomes 0
        tmax = fmaxf(tmax, v[k]);
    }
    const int live = int(min(int64_t(kSelStretch), int64_t(a.V) - first));  // elements from the stretch's first on
    {
        const float wm = warp_max(tmax), wl = warp_min(tmax > -INFINITY ? tmax : INFINITY);
        if (lane == 0) {
            s_max[warp] = wm;
            s_min[warp] = wl;
        }
    }
    s_hist[tid] = 0;
    if (tid == 0) s_count = s_total = 0;
    __syncthreads();
    float m = s_max[0], least = s_min[0];
#pragma unroll
    for (int w = 1; w < kSelThreads / 32; ++w) {
        m = fmaxf(m, s_max[w]);
        least = fminf(least, s_min[w]);
    }
    if (!(m > -INFINITY)) {  // nothing allowed here
        if (tid == 0) res[unit] = Stretch{0.0, -INFINITY, 0};
        return;
    }

    // sum of exp(x - m)
    const double power = kPowers32.v[lane];
    constexpr double kC = 46.166241308446828384;  // 32 / ln 2
    constexpr double kMagic = 6755399441055744.0; // 1.5 * 2^52: adding it leaves the nearest integer in the low bits
    const double mc = double(m) * -kC;
    const float floor_x = m - 700.f;              // exp(-700) is nothing next to 1
    double sum = 0.0;
    if (fabsf(m) > 0x1p20f) {                     // that floor is not a number near m: rare, so the plain way
#pragma unroll
        for (int k = 0; k < kSelPerThread; ++k) {
            const double d = double(v[k]) - double(m);
            if (d >= -700.0) sum += exp(d);
        }
    } else {
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        if (j * kSelThreads * PER >= live) break;
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const double y = fma(double(fmaxf(v[j * PER + u], floor_x)), kC, mc);
            const double t = y + kMagic;
            const double r = y - (t - kMagic);
            const int k = __double2loint(t);
            const int hi = __shfl_sync(0xffffffffu, __double2hiint(power), k & 31);
            const int lo = __shfl_sync(0xffffffffu, __double2loint(power), k & 31);
            const double scaled = __hiloint2double(hi + ((k >> 5) << 20), lo);
            constexpr double z = 0.0216608493924982908;  // ln 2 / 32
            const double p = fma(r, fma(r, fma(r, fma(r, z * z * z * z / 24, z * z * z / 6), z * z / 2), z), 1.0);
            sum = fma(scaled, p, sum);
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) s_sum[warp] = sum;

    // the edge below which at least `keep` maxima lie
    const uint32_t keep = uint32_t(a.keep);
    float inv = bin_scale(m - least);
    {
        const bool coarse = keep <= kSelThreads / 2;  // a maximum per thread is enough to choose from
        if (coarse) {
            if (tmax > -INFINITY) {
                atomicAdd(&s_hist[min(kHistBins - 1, int((m - tmax) * inv))], 1u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VECS; ++j) {
                float y = v[j * PER];
#pragma unroll
                for (int u = 1; u < PER; ++u) y = fmaxf(y, v[j * PER + u]);
                if (y >= least) atomicAdd(&s_hist[min(kHistBins - 1, int((m - y) * inv))], 1u);
            }
        }
    }
    __syncthreads();
    find_bin<kHistBins>(s_hist, keep, &s_bin);
    __syncthreads();
    float edge = s_bin >= 0 ? float(s_bin + 1) : INFINITY;
    if (s_bin == kHistBins - 1) edge = INFINITY;  // that bin also holds what lies below `least`
    // entries above the edge
#pragma unroll
    for (int k = 0; k < kSelPerThread; ++k) {
        const float x0 = v[k];
        if (x0 > -INFINITY && !((m - x0) * inv >= edge)) {
            const uint32_t at = atomicAdd(&s_count, 1u);
            if (at < uint32_t(cap)) {
                const int64_t e = first + int64_t((k / PER) * kSelThreads + tid) * PER + k % PER;
                list[at] = make_uint2(__float_as_uint(x0), uint32_t(e));
            }
        }
    }
    __syncthreads();
    uint32_t count = s_count;
    if (count > uint32_t(cap)) {
        // Too many: the exact border, the largest key with at least `keep` keys at or above it
        // (the logit's order first, then the lower index).
        uint64_t border = 0;
        for (int bit = 63; bit >= 0; --bit) {
            const uint64_t mid = border | 1ull << bit;
            uint32_t c = 0;
#pragma unroll
            for (int k = 0; k < kSelPerThread; ++k) {
                const int64_t e = first + int64_t((k / PER) * kSelThreads + tid) * PER + k % PER;
                const uint64_t key = uint64_t(float_key(v[k])) << 32 | (0xffffffffu - uint32_t(e));
                c += v[k] > -INFINITY && key >= mid;
            }
            c = __reduce_add_sync(0xffffffffu, c);
            if (lane == 0) atomicAdd(&s_total, c);
            __syncthreads();
            const uint32_t total = s_total;
            __syncthreads();
            if (tid == 0) s_total = 0;
            __syncthreads();
            if (total >= keep) border = mid;
        }
        if (tid == 0) s_count = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSelPerThread; ++k) {
            const int64_t e = first + int64_t((k / PER) * kSelThreads + tid) * PER + k % PER;
            const uint64_t key = uint64_t(float_key(v[k])) << 32 | (0xffffffffu - uint32_t(e));
            if (v[k] > -INFINITY && key >= border) {
                const uint32_t at = atomicAdd(&s_count, 1u);
                if (at < uint32_t(cap)) list[at] = make_uint2(__float_as_uint(v[k]), uint32_t(e));
            }
        }
        __syncthreads();
        count = min(s_count, uint32_t(cap));
    }
    if (tid == 0) {
        double total = 0.0;
#pragma unroll
        for (int w = 0; w < kSelThreads / 32; ++w) total += s_sum[w];
        res[unit] = Stretch{total, m, int32_t(count)};
    }
}

struct MergeShared {
    double base[ST_BEAM_MAX_BEAMS];  // score minus normaliser; NaN: no candidates
    uint64_t key[kMergeCap];
    uint32_t flat[kMergeCap];
    int32_t units[kMergeUnits];
    uint32_t hist[kHistBins];
    double red[kMergeThreads / 32], red2[kMergeThreads / 32];
    uint32_t n_units, n_pairs, n_tops;
    int bin;
};

__global__ void __launch_bounds__(kMergeThreads)
beam_merge_kernel(SelectArgs a, int stretches, int cap, const Stretch* res, const uint2* lists)
{
    extern __shared__ __align__(16) unsigned char raw[];
    MergeShared& sh = *reinterpret_cast<MergeShared*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x;
    const int64_t row0 = int64_t(b) * a.K;
    const int n_units = a.K * stretches;
    const double kNone = __longlong_as_double(0x7ff8000000000000ll);
    res += row0 * stretches;
    lists += row0 * stretches * cap;

    // the beams' normalisers, a warp per beam
    for (int i = warp; i < a.K; i += kMergeThreads / 32) {
        float m = -INFINITY;
        for (int c = lane; c < stretches; c += 32) m = fmaxf(m, res[int64_t(i) * stretches + c].max);
        m = warp_max(m);
        double s = 0.0;
        if (m > -INFINITY)
            for (int c = lane; c < stretches; c += 32) {
                const Stretch t = res[int64_t(i) * stretches + c];
                if (t.max > -INFINITY) s += t.sum * exp(double(t.max) - double(m));
            }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (lane == 0) sh.base[i] = m > -INFINITY ? double(a.scores[row0 + i]) - (double(m) + log(s)) : kNone;
    }
    for (int i = tid; i < kHistBins; i += kMergeThreads) sh.hist[i] = 0;
    if (tid == 0) sh.n_units = sh.n_pairs = sh.n_tops = 0;
    __syncthreads();

    // the stretches' best scores: their range, and how many there are
    double best = -INFINITY, least = INFINITY;
    uint32_t tops = 0;
    for (int u = tid; u < n_units; u += kMergeThreads) {
        const float m = res[u].max;
        const double s = sh.base[u / stretches] + double(m);
        if (m > -INFINITY && s == s) {
            best = fmax(best, s);
            least = fmin(least, s);
            ++tops;
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        best = fmax(best, __shfl_xor_sync(0xffffffffu, best, off));
        least = fmin(least, __shfl_xor_sync(0xffffffffu, least, off));
    }
    tops = __reduce_add_sync(0xffffffffu, tops);
    if (lane == 0) {
        sh.red[warp] = best;
        sh.red2[warp] = least;
        if (tops) atomicAdd(&sh.n_tops, tops);
    }
    __syncthreads();
    for (int w = 0; w < kMergeThreads / 32; ++w) {
        best = fmax(best, sh.red[w]);
        least = fmin(least, sh.red2[w]);
    }
    const uint32_t keep = uint32_t(a.keep);
    float edge = INFINITY, inv = 0.f;
    if (sh.n_tops >= keep) {  // the edge that `keep` of them reach: the keep-th score is not below it
        inv = bin_scale(float(best - least));
        for (int u = tid; u < n_units; u += kMergeThreads) {
            const float m = res[u].max;
            const double s = sh.base[u / stretches] + double(m);
            if (m > -INFINITY && s == s) atomicAdd(&sh.hist[min(kHistBins - 1, int(float(best - s) * inv))], 1u);
        }
        __syncthreads();
        find_bin<kHistBins>(sh.hist, keep, &sh.bin);
        __syncthreads();
        if (sh.bin >= 0 && sh.bin < kHistBins - 1) edge = float(sh.bin + 1);
    }
    // the stretches that reach it, then their entries
    for (int u = tid; u < n_units; u += kMergeThreads) {
        const float m = res[u].max;
        const double s = sh.base[u / stretches] + double(m);
        if (m > -INFINITY && s == s && !(float(best - s) * inv >= edge)) {
            const uint32_t at = atomicAdd(&sh.n_units, 1u);
            if (at < kMergeUnits) sh.units[at] = u;
        }
    }
    __syncthreads();
    bool fits = sh.n_units <= kMergeUnits;
    if (fits) {
        const int n = int(sh.n_units);
        for (int k = warp; k < n; k += kMergeThreads / 32) {
            const int u = sh.units[k], i = u / stretches;
            const int count = res[u].count;
            for (int e = lane; e < count; e += 32) {
                const uint2 w = lists[int64_t(u) * cap + e];
                const double s = sh.base[i] + double(__uint_as_float(w.x));
                if (!(float(best - s) * inv >= edge)) {
                    const uint32_t at = atomicAdd(&sh.n_pairs, 1u);
                    if (at < kMergeCap) {
                        sh.key[at] = double_key(s);
                        sh.flat[at] = uint32_t(i) * uint32_t(a.V) + w.y;
                    }
                }
            }
        }
        __syncthreads();
        fits = sh.n_pairs <= kMergeCap;
    }
    if (!fits) {
        // Exact: the keep-th largest score by its eight digits, then the
        // largest index still taken among those that equal it by its four.
        uint64_t prefix = 0;
        uint32_t want = keep;
        bool all = false;
        auto each = [&](auto&& f) {
            for (int u = warp; u < n_units; u += kMergeThreads / 32) {
                const int count = res[u].count, i = u / stretches;
                for (int e0 = 0; e0 < count; e0 += 32) {
                    const int e = e0 + lane;
                    const uint2 w = e < count ? lists[int64_t(u) * cap + e] : make_uint2(0, 0);
                    const uint64_t key = e < count ? double_key(sh.base[i] + double(__uint_as_float(w.x))) : 0ull;
                    f(e < count, key, uint32_t(i) * uint32_t(a.V) + w.y);
                }
            }
        };
        for (int d = 7; d >= 0 && !all; --d) {  // digits from the top; bins reversed: the largest first
            __syncthreads();
            for (int i = tid; i < kHistBins; i += kMergeThreads) sh.hist[i] = 0;
            __syncthreads();
            each([&](bool on, uint64_t key, uint32_t) {
                on = on && (d == 7 || key >> (8 * d + 8) == prefix >> (8 * d + 8));
                const unsigned members = __ballot_sync(0xffffffffu, on);
                if (on) count_bin(sh.hist, 255 - int(key >> (8 * d) & 255), members);
            });
            __syncthreads();
            find_bin<kHistBins>(sh.hist, want, &sh.bin);
            __syncthreads();
            if (sh.bin < 0) {
                all = true;  // fewer than `keep` entries in all
            } else {
                for (int i = 0; i < sh.bin; ++i) want -= sh.hist[i];
                prefix |= uint64_t(255 - sh.bin) << (8 * d);
            }
        }
        uint32_t last = 0;  // of the entries equal to the border, `want` are taken: the lowest indexes
        for (int d = 3; d >= 0 && !all; --d) {
            __syncthreads();
            for (int i = tid; i < kHistBins; i += kMergeThreads) sh.hist[i] = 0;
            __syncthreads();
            each([&](bool on, uint64_t key, uint32_t flat) {
                on = on && key == prefix && (d == 3 || flat >> (8 * d + 8) == last >> (8 * d + 8));
                const unsigned members = __ballot_sync(0xffffffffu, on);
                if (on) count_bin(sh.hist, int(flat >> (8 * d) & 255), members);
            });
            __syncthreads();
            find_bin<kHistBins>(sh.hist, want, &sh.bin);
            __syncthreads();
            const int bin = max(sh.bin, 0);
            for (int i = 0; i < bin; ++i) want -= sh.hist[i];
            last |= uint32_t(bin) << (8 * d);
        }
        __syncthreads();
        if (tid == 0) sh.n_pairs = 0;
        __syncthreads();
        each([&](bool on, uint64_t key, uint32_t flat) {
            if (on && (all || key > prefix || (key == prefix && flat <= last))) {
                const uint32_t at = atomicAdd(&sh.n_pairs, 1u);
                if (at < kMergeCap) {
                    sh.key[at] = key;
                    sh.flat[at] = flat;
                }
            }
        });
        __syncthreads();
    }

    // order the pairs (bitonic, padded with the least key), write the best
    const int n = int(min(sh.n_pairs, uint32_t(kMergeCap)));
    int size = 32;
    while (size < n) size <<= 1;
    for (int i = n + tid; i < size; i += kMergeThreads) {
        sh.key[i] = 0;
        sh.flat[i] = 0xffffffffu;
    }
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int t = tid; t < size / 2; t += kMergeThreads) {
                const int lo = 2 * t - (t & (j - 1)), hi = lo + j;
                const uint64_t ka = sh.key[lo], kb = sh.key[hi];
                const uint32_t fa = sh.flat[lo], fb = sh.flat[hi];
                const bool ordered = ka > kb || (ka == kb && fa < fb);
                if (ordered != ((lo & k) == 0)) {
                    sh.key[lo] = kb;
                    sh.key[hi] = ka;
                    sh.flat[lo] = fb;
                    sh.flat[hi] = fa;
                }
            }
            __syncthreads();
        }
    for (int r = tid; r < a.keep; r += kMergeThreads) {
        const int64_t o = int64_t(b) * a.keep + r;
        float s = -INFINITY;
        int parent = -1, token = -1;
        bool done = false;
        if (r < n) {
            const uint64_t key = sh.key[r];
            const uint64_t bits = key >> 63 ? key ^ 1ull << 63 : ~key;
            s = float(__longlong_as_double((long long)(bits)));
            parent = int(sh.flat[r] / uint32_t(a.V));
            token = int(sh.flat[r] - uint32_t(parent) * uint32_t(a.V));
            if (a.ex.finished) done = a.ex.finished[row0 + parent] || token == a.ex.end_token;
        }
        a.out_scores[o] = s;
        a.out_parents[o] = parent;
        a.out_tokens[o] = token;
        if (a.ex.out_finished) a.ex.out_finished[o] = done;
    }
}

// A stretch begins at a 16-byte boundary, up to 7 elements before the row.
static int select_stretches(int32_t V) { return (V + 7 + kSelStretch - 1) / kSelStretch; }
// Entries a stretch may write: room for the bin that holds the border.
static int select_cap(int32_t V, int32_t keep)
{
    const int most = V < kSelStretch ? V : kSelStretch;
    return keep + 64 < most ? keep + 64 : most;
}

int64_t beam_select_workspace(int32_t B, int32_t K, int32_t V, int32_t keep)
{
    const int64_t units = int64_t(B) * K * select_stretches(V);
    return units * int64_t(sizeof(Stretch)) + units * select_cap(V, keep) * 8;
}

cudaError_t launch_beam_select(const SelectArgs& a, cudaStream_t s)
{
    const int stretches = select_stretches(a.V), cap = select_cap(a.V, a.keep);
    const int64_t rows = int64_t(a.B) * a.K;
    Stretch* res = static_cast<Stretch*>(a.workspace);
    uint2* lists = reinterpret_cast<uint2*>(res + rows * stretches);
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(beam_merge_kernel), int(sizeof(MergeShared)));
    if (e != cudaSuccess) return e;
    // grid y is at most 65535 rows
    const int64_t step = 65535 / a.K * int64_t(a.K);
    for (int64_t r0 = 0; r0 < rows; r0 += step) {
        const dim3 grid(unsigned(stretches), unsigned(rows - r0 < step ? rows - r0 : step));
        SelectArgs p = a;
        const int64_t size = a.dtype == ST_F32 ? 4 : 2;
        p.logits = static_cast<const char*>(a.logits) + r0 * a.stride * size;
        p.scores += r0;
        if (p.ex.finished) p.ex.finished += r0;
        if (p.ex.allow) p.ex.allow += r0 / a.K * a.ex.allow_request_stride;
        Stretch* pr = res + r0 * stretches;
        uint2* pl = lists + r0 * stretches * cap;
        switch (a.dtype) {
            case ST_BF16: beam_stretch_kernel<__nv_bfloat16><<<grid, kSelThreads, 0, s>>>(p, stretches, cap, pr, pl); break;
            case ST_F16: beam_stretch_kernel<__half><<<grid, kSelThreads, 0, s>>>(p, stretches, cap, pr, pl); break;
            default: beam_stretch_kernel<float><<<grid, kSelThreads, 0, s>>>(p, stretches, cap, pr, pl); break;
        }
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    beam_merge_kernel<<<a.B, kMergeThreads, sizeof(MergeShared), s>>>(a, stretches, cap, res, lists);
    return cudaGetLastError();
}

}  // namespace st
