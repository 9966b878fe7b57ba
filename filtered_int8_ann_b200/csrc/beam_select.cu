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
#include <cfloat>

#include "decode.cuh"

namespace st {

constexpr int kSelThreads = 256;
constexpr int kSelPerThread = 32;
constexpr int kSelStretch = kSelThreads * kSelPerThread;
constexpr int kMergeThreads = 1024;
constexpr int kMergeCap = 2048;   // pairs sorted at the end
constexpr int kMergeRank = kMergeThreads / 4;  // up to this many are ordered by counting
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
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 becomes 0
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

// Logits as they are held: 16 bytes are PER of them in four words. A 32-bit word holds one (f32) or two.
template <typename T>
struct Logit;
template <>
struct Logit<float> {
    static constexpr int kPer = 4, kIn = 1;  // per 16 bytes, per word
    static constexpr uint32_t kNone = 0xff800000u;  // -inf
    __device__ static uint32_t max2(uint32_t a, uint32_t b) { return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b))); }
    __device__ static float get(uint32_t w, int) { return __uint_as_float(w); }
    __device__ static uint32_t both(float x) { return __float_as_uint(x); }
    // bits of the word's elements that are at least x
    __device__ static uint32_t reach(uint32_t w, uint32_t x) { return __uint_as_float(w) >= __uint_as_float(x) ? 1u : 0u; }
    __device__ static uint32_t keep(uint32_t w, uint32_t bits) { return bits & 1u ? w : kNone; }
    __device__ static float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
    __device__ static uint32_t bits(const void* p, int64_t i) { return static_cast<const uint32_t*>(p)[i]; }
};
template <typename H, typename H2>
struct LogitHalf {
    static constexpr int kPer = 8, kIn = 2;
    __device__ static H2 as(uint32_t w) { return *reinterpret_cast<const H2*>(&w); }
    __device__ static uint32_t max2(uint32_t a, uint32_t b)
    {
        const H2 m = __hmax2(as(a), as(b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    __device__ static uint32_t reach(uint32_t w, uint32_t x)
    {
        const unsigned r = __hge2_mask(as(w), as(x));
        return (r & 1u) | (r >> 30 & 2u);
    }
    static __device__ uint32_t keep2(uint32_t w, uint32_t bits, uint32_t none)
    {
        const uint32_t on = (bits & 1u ? 0xffffu : 0u) | (bits & 2u ? 0xffff0000u : 0u);
        return (w & on) | (none & ~on);
    }
    __device__ static uint32_t bits(const void* p, int64_t i) { return static_cast<const uint16_t*>(p)[i]; }
};
template <>
struct Logit<__nv_bfloat16> : LogitHalf<__nv_bfloat16, __nv_bfloat162> {
    static constexpr uint32_t kNone = 0xff80ff80u;
    __device__ static float get(uint32_t w, int i) { return __uint_as_float(i ? w & 0xffff0000u : w << 16); }
    __device__ static uint32_t both(float x) { const __nv_bfloat162 h = __float2bfloat162_rn(fmaxf(x, -3.3895313892515355e38f)); return *reinterpret_cast<const uint32_t*>(&h); }
    __device__ static uint32_t keep(uint32_t w, uint32_t bits) { return keep2(w, bits, kNone); }
    __device__ static float one(const void* p, int64_t i) { return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]); }
};
template <>
struct Logit<__half> : LogitHalf<__half, __half2> {
    static constexpr uint32_t kNone = 0xfc00fc00u;
    __device__ static float get(uint32_t w, int i) { const __half2 h = as(w); return i ? __high2float(h) : __low2float(h); }
    __device__ static uint32_t both(float x) { const __half2 h = __float2half2_rn(fmaxf(x, -65504.f)); return *reinterpret_cast<const uint32_t*>(&h); }
    __device__ static uint32_t keep(uint32_t w, uint32_t bits) { return keep2(w, bits, kNone); }
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
__device__ __forceinline__ float bin_scale(float range, int bins) { return range > 0.f ? fminf(float(bins - 1) / range, 3e38f) : 0.f; }

template <typename T>
__global__ void __launch_bounds__(kSelThreads, 3)
beam_stretch_kernel(SelectArgs a, int stretches, int cap, Stretch* res, uint2* lists)
{
    using L = Logit<T>;
    constexpr int PER = L::kPer, IN = L::kIn, VECS = kSelPerThread / PER, WORDS = VECS * 4;
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
    const int first = int(blockIdx.x) * kSelStretch - before;  // the row's index of the stretch's first element
    const int live = min(kSelStretch, a.V - first);  // elements from there on
    // the row's index of element u of this thread's word k
    auto index_of = [&](int k, int u) { return first + ((k / 4) * kSelThreads + tid) * PER + (k % 4) * IN + u; };
    uint32_t v[WORDS];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
        const int e = first + (j * kSelThreads + tid) * PER;
        if (e >= 0 && e + PER <= a.V) {
            const uint4 w = __ldcs(reinterpret_cast<const uint4*>(x + e));
            v[4 * j] = w.x;
            v[4 * j + 1] = w.y;
            v[4 * j + 2] = w.z;
            v[4 * j + 3] = w.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t w = L::kNone;
#pragma unroll
                for (int u = 0; u < IN; ++u) {
                    const int at = e + k * IN + u;
                    if (at >= 0 && at < a.V) {
                        if (IN == 1) w = L::bits(x, at);
                        else w = (w & (u ? 0xffffu : 0xffff0000u)) | L::bits(x, at) << (16 * u);
                    }
                }
                v[4 * j + k] = w;
            }
        }
    }
    if (a.ex.allow) {
        const uint32_t* allow = a.ex.allow + b * a.ex.allow_request_stride + i * a.ex.allow_beam_stride;
        const int words = (a.V + 31) / 32;
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int e = first + (j * kSelThreads + tid) * PER;
            if (e + PER <= 0 || e >= a.V) continue;
            const int at = e < 0 ? 0 : e;  // bits of elements at .. at + PER
            const int w = int(at >> 5);
            const uint32_t lo = allow[w], hi = w + 1 < words ? allow[w + 1] : 0u;
            const uint32_t bits = __funnelshift_r(lo, hi, uint32_t(at & 31)) << uint32_t(at - e);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * j + k] = L::keep(v[4 * j + k], bits >> (k * IN));
        }
    }
    // The maximum (NaN takes no part). Where it is +inf, those entries leave and it is taken again.
    s_hist[tid] = 0;
    if (tid == 0) s_count = s_total = 0;
    float tmax, m, least;
    for (int pass = 0;; ++pass) {
        uint32_t top = v[0];
#pragma unroll
        for (int k = 1; k < WORDS; ++k) top = L::max2(top, v[k]);
        tmax = IN == 1 ? L::get(top, 0) : fmaxf(L::get(top, 0), L::get(top, 1));
        const float wm = warp_max(tmax), wl = warp_min(tmax > -INFINITY ? tmax : INFINITY);
        if (lane == 0) {
            s_max[warp] = wm;
            s_min[warp] = wl;
        }
        __syncthreads();
        m = s_max[0];
        least = s_min[0];
#pragma unroll
        for (int w = 1; w < kSelThreads / 32; ++w) {
            m = fmaxf(m, s_max[w]);
            least = fminf(least, s_min[w]);
        }
        if (m < INFINITY || pass > 0) break;
#pragma unroll
        for (int k = 0; k < WORDS; ++k) {
            uint32_t on = 0;
#pragma unroll
            for (int u = 0; u < IN; ++u) on |= (L::get(v[k], u) < INFINITY ? 1u : 0u) << u;
            v[k] = L::keep(v[k], on);
        }
        __syncthreads();
    }
    if (!(m > -INFINITY)) {  // nothing allowed here
        if (tid == 0) res[unit] = Stretch{0.0, -INFINITY, 0};
        return;
    }

    // sum of exp(x - m)
    const double power = kPowers32.v[lane];
    const int power_hi = __double2hiint(power), power_lo = __double2loint(power);
    double sum = 0.0;
    if (fabsf(m) > 0x1p20f) {  // m - 700 is not a number near m: rare, so the plain way
#pragma unroll 1
        for (int e = tid; e < live; e += kSelThreads) {
            // (from memory again, so that the registers need no index; allowed ones among them)
            const int at = first + e;
            if (at < 0) continue;
            bool on = true;
            if (a.ex.allow) on = (a.ex.allow + b * a.ex.allow_request_stride + i * a.ex.allow_beam_stride)[at >> 5] >> (at & 31) & 1u;
            const float y = L::one(x, at);
            const double d = double(y) - double(m);
            if (on && y < INFINITY && d >= -700.0) sum += exp(d);
        }
    } else {
        constexpr double kC = 46.166241308446828384;  // 32 / ln 2
        constexpr double kMagic = 6755399441055744.0; // 1.5 * 2^52: adding it leaves the nearest integer in the low bits
        constexpr double z = 0.0216608493924982908;   // ln 2 / 32
        const double mc = double(m) * -kC;
        const uint32_t floor2 = L::both(m - 700.f);   // exp(-700) is nothing next to 1; takes the place of -inf and NaN
        double part[2] = {0.0, 0.0};
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            if (j * kSelThreads * PER >= live) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t w = L::max2(v[4 * j + k], floor2);
#pragma unroll
                for (int u = 0; u < IN; ++u) {
                    const double y = fma(double(L::get(w, u)), kC, mc);
                    const double t = y + kMagic;
                    const double r = y - (t - kMagic);
                    const int n = __double2loint(t);
                    const int hi = __shfl_sync(0xffffffffu, power_hi, n), lo = __shfl_sync(0xffffffffu, power_lo, n);
                    const double scaled = __hiloint2double(hi + ((n >> 5) << 20), lo);
                    const double p = fma(r, fma(r, fma(r, fma(r, z * z * z * z / 24, z * z * z / 6), z * z / 2), z), 1.0);
                    part[(k + u) & 1] = fma(scaled, p, part[(k + u) & 1]);
                }
            }
        }
        sum = part[0] + part[1];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) s_sum[warp] = sum;

    // the edge below which at least `keep` maxima lie
    const uint32_t keep = uint32_t(a.keep);
    const float inv = bin_scale(m - least, kHistBins);
    if (keep <= kSelThreads / 2) {  // a maximum per thread is enough to choose from
        if (tmax > -INFINITY) atomicAdd(&s_hist[min(kHistBins - 1, int((m - tmax) * inv))], 1u);
    } else {  // one per vector
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const uint32_t w = L::max2(L::max2(v[4 * j], v[4 * j + 1]), L::max2(v[4 * j + 2], v[4 * j + 3]));
            const float y = IN == 1 ? L::get(w, 0) : fmaxf(L::get(w, 0), L::get(w, 1));
            if (y >= least) atomicAdd(&s_hist[min(kHistBins - 1, int((m - y) * inv))], 1u);
        }
    }
    __syncthreads();
    find_bin<kHistBins>(s_hist, keep, &s_bin);
    __syncthreads();
    // Entries down to a value that is surely not above the edge. The last bin also holds what lies below `least`.
    float edge = -FLT_MAX;
    if (s_bin >= 0 && s_bin < kHistBins - 1 && inv > 0.f) edge = fmaxf(edge, m - float(s_bin + 1) / inv * 1.00001f - fabsf(m) * 0x1p-20f);
    if (edge <= tmax) {  // (false where this thread has none: NaN or -inf)
        const uint32_t e2 = L::both(edge);
        // a value rounded up to the type would lose entries: one step down then
        const uint32_t from = L::get(e2, 0) <= edge ? e2 : L::both(edge - fabsf(edge) * 0.01f - FLT_MIN);
        uint32_t found = 0;
#pragma unroll
        for (int k = 0; k < WORDS; ++k) found |= L::reach(v[k], from) << (k * IN);
        while (found) {
            const int k = __ffs(found) - 1;
            found &= found - 1;
            const int e = index_of(k / IN, k % IN);
            const uint32_t at = atomicAdd(&s_count, 1u);
            if (at < uint32_t(cap)) list[at] = make_uint2(__float_as_uint(L::one(x, e)), uint32_t(e));
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
            for (int k = 0; k < WORDS; ++k)
#pragma unroll
                for (int u = 0; u < IN; ++u) {
                    const float y = L::get(v[k], u);
                    const uint64_t key = uint64_t(float_key(y)) << 32 | (0xffffffffu - uint32_t(index_of(k, u)));
                    c += y > -INFINITY && key >= mid;
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
        for (int k = 0; k < WORDS; ++k)
#pragma unroll
            for (int u = 0; u < IN; ++u) {
                const float y = L::get(v[k], u);
                const int e = index_of(k, u);
                const uint64_t key = uint64_t(float_key(y)) << 32 | (0xffffffffu - uint32_t(e));
                if (y > -INFINITY && key >= border) {
                    const uint32_t at = atomicAdd(&s_count, 1u);
                    if (at < uint32_t(cap)) list[at] = make_uint2(__float_as_uint(y), uint32_t(e));
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

// The second launch keeps a request's pairs in shared memory.
constexpr int kMergePairs = 4096;  // pairs collected
constexpr int kMergeBins = 1024;

struct MergeShared {
    double base[ST_BEAM_MAX_BEAMS];  // score minus normaliser; NaN: no candidates
    uint64_t key[kMergePairs];       // score (order-preserving); then the sorted ones
    uint32_t flat[kMergePairs];      // i * V + v
    uint64_t out_key[kMergeCap];
    uint32_t out_flat[kMergeCap];
    int32_t units[kMergeUnits];
    uint32_t hist[kMergeBins];
    double best[kMergeThreads / 32], least[kMergeThreads / 32];
    uint32_t n_units, n_pairs, n_out, n_tops;
    int bin;
};

__device__ __forceinline__ double key_double(uint64_t key)
{
    return __longlong_as_double((long long)(key >> 63 ? key ^ 1ull << 63 : ~key));
}

__global__ void __launch_bounds__(kMergeThreads)
beam_merge_kernel(SelectArgs a, int stretches, int cap, const Stretch* res, const uint2* lists)
{
    dep_enter();
    extern __shared__ __align__(16) unsigned char raw[];
    MergeShared& sh = *reinterpret_cast<MergeShared*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x;
    const int64_t row0 = int64_t(b) * a.K;
    const int n_units = a.K * stretches;
    const uint32_t keep = uint32_t(a.keep);
    res += row0 * stretches;
    lists += row0 * stretches * cap;

    // the beams' normalisers, a warp per beam, and the range of the stretches' best scores
    if (tid == 0) sh.n_units = sh.n_pairs = sh.n_out = sh.n_tops = 0;
    for (int i = tid; i < kMergeBins; i += kMergeThreads) sh.hist[i] = 0;
    __syncthreads();
    double best = -INFINITY, least = INFINITY;
    uint32_t tops = 0;
    for (int i = warp; i < a.K; i += kMergeThreads / 32) {
        const Stretch* r = res + int64_t(i) * stretches;
        float m = -INFINITY, low = INFINITY;
        uint32_t n = 0;
        for (int c = lane; c < stretches; c += 32) {
            const float t = r[c].max;
            m = fmaxf(m, t);
            if (t > -INFINITY) {
                low = fminf(low, t);
                ++n;
            }
        }
        m = warp_max(m);
        low = warp_min(low);
        double s = 0.0, base = __longlong_as_double(0x7ff8000000000000ll);
        if (m > -INFINITY) {
            for (int c = lane; c < stretches; c += 32)
                if (r[c].max > -INFINITY) s += r[c].sum * exp(double(r[c].max) - double(m));
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            base = double(a.scores[row0 + i]) - (double(m) + log(s));
            best = fmax(best, base + double(m));
            least = fmin(least, base + double(low));
            tops += n;
        }
        if (lane == 0) sh.base[i] = base;
    }
    tops = __reduce_add_sync(0xffffffffu, tops);
    if (lane == 0) {
        sh.best[warp] = best;
        sh.least[warp] = least;
        if (tops) atomicAdd(&sh.n_tops, tops);
    }
    __syncthreads();
    best = sh.best[lane];
    least = sh.least[lane];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        best = fmax(best, __shfl_xor_sync(0xffffffffu, best, off));
        least = fmin(least, __shfl_xor_sync(0xffffffffu, least, off));
    }
    // a score's place below the best: bins of `inv` per unit; scores whose place is not at or above the edge are kept
    float edge = INFINITY, inv = 0.f;
    auto place = [&](double s) { return float(best - s) * inv; };
    auto score_of = [&](int u, float x) { return sh.base[u / stretches] + double(x); };
    if (sh.n_tops >= keep) {  // the edge that `keep` of the stretches' best reach: the keep-th score is not below it
        inv = bin_scale(float(best - least), kMergeBins);
        for (int u = tid; u < n_units; u += kMergeThreads) {
            const float m = res[u].max;
            if (m > -INFINITY) atomicAdd(&sh.hist[min(kMergeBins - 1, int(place(score_of(u, m))))], 1u);
        }
        __syncthreads();
        find_bin<kMergeBins>(sh.hist, keep, &sh.bin);
        __syncthreads();
        if (sh.bin >= 0 && sh.bin < kMergeBins - 1) edge = float(sh.bin + 1);
    }
    // the stretches that reach it
    for (int u = tid; u < n_units; u += kMergeThreads) {
        const float m = res[u].max;
        if (m > -INFINITY && !(place(score_of(u, m)) >= edge)) {
            const uint32_t at = atomicAdd(&sh.n_units, 1u);
            if (at < kMergeUnits) sh.units[at] = u;
        }
    }
    __syncthreads();
    const int listed = int(sh.n_units);
    bool fits = listed <= kMergeUnits;
    // their entries that reach it; where those are too many, a finer edge from a histogram of them all first
    auto each_listed = [&](auto&& f) {
        for (int k = warp; k < listed; k += kMergeThreads / 32) {
            const int u = sh.units[k], i = u / stretches, count = res[u].count;
            for (int e = lane; e < count; e += 32) {
                const uint2 w = lists[int64_t(u) * cap + e];
                const double s = sh.base[i] + double(__uint_as_float(w.x));
                if (!(place(s) >= edge)) f(s, uint32_t(i) * uint32_t(a.V) + w.y);
            }
        }
    };
    for (int pass = 0; fits && pass < 2; ++pass) {
        each_listed([&](double s, uint32_t flat) {
            const uint32_t at = atomicAdd(&sh.n_pairs, 1u);
            if (at < kMergePairs) {
                sh.key[at] = double_key(s);
                sh.flat[at] = flat;
            }
        });
        __syncthreads();
        const bool all = sh.n_pairs <= kMergePairs;
        __syncthreads();
        if (all) break;
        fits = pass == 0;
        if (!fits) break;
        const float span = edge == INFINITY ? float(best - least) : edge / inv;  // (least bounds no entries, so the last bin takes those below)
        const float fine = bin_scale(span, kMergeBins);
        for (int i = tid; i < kMergeBins; i += kMergeThreads) sh.hist[i] = 0;
        if (tid == 0) sh.n_pairs = 0;
        __syncthreads();
        each_listed([&](double s, uint32_t) { atomicAdd(&sh.hist[min(kMergeBins - 1, int(float(best - s) * fine))], 1u); });
        __syncthreads();
        find_bin<kMergeBins>(sh.hist, keep, &sh.bin);
        __syncthreads();
        if (sh.bin < 0 || sh.bin >= kMergeBins - 1) {
            fits = false;
        } else {
            inv = fine;
            edge = float(sh.bin + 1);
        }
    }
    if (fits) {
        // In shared memory now: the edge that `keep` of them reach, and those above it.
        const int n = int(sh.n_pairs);
        const float span = edge == INFINITY ? float(best - least) : edge / inv;
        const float fine = bin_scale(span, kMergeBins);
        for (int i = tid; i < kMergeBins; i += kMergeThreads) sh.hist[i] = 0;
        __syncthreads();
        for (int k = tid; k < n; k += kMergeThreads)
            atomicAdd(&sh.hist[min(kMergeBins - 1, int(float(best - key_double(sh.key[k])) * fine))], 1u);
        __syncthreads();
        find_bin<kMergeBins>(sh.hist, keep, &sh.bin);
        __syncthreads();
        const float last = sh.bin >= 0 && sh.bin < kMergeBins - 1 ? float(sh.bin + 1) : INFINITY;
        for (int k = tid; k < n; k += kMergeThreads) {
            const uint64_t key = sh.key[k];
            if (!(float(best - key_double(key)) * fine >= last)) {
                const uint32_t at = atomicAdd(&sh.n_out, 1u);
                if (at < kMergeCap) {
                    sh.out_key[at] = key;
                    sh.out_flat[at] = sh.flat[k];
                }
            }
        }
        __syncthreads();
        fits = sh.n_out <= kMergeCap;
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
            for (int i = tid; i < 256; i += kMergeThreads) sh.hist[i] = 0;
            __syncthreads();
            each([&](bool on, uint64_t key, uint32_t) {
                on = on && (d == 7 || key >> (8 * d + 8) == prefix >> (8 * d + 8));
                const unsigned members = __ballot_sync(0xffffffffu, on);
                if (on) count_bin(sh.hist, 255 - int(key >> (8 * d) & 255), members);
            });
            __syncthreads();
            find_bin<256>(sh.hist, want, &sh.bin);
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
            for (int i = tid; i < 256; i += kMergeThreads) sh.hist[i] = 0;
            __syncthreads();
            each([&](bool on, uint64_t key, uint32_t flat) {
                on = on && key == prefix && (d == 3 || flat >> (8 * d + 8) == last >> (8 * d + 8));
                const unsigned members = __ballot_sync(0xffffffffu, on);
                if (on) count_bin(sh.hist, int(flat >> (8 * d) & 255), members);
            });
            __syncthreads();
            find_bin<256>(sh.hist, want, &sh.bin);
            __syncthreads();
            const int bin = max(sh.bin, 0);
            for (int i = 0; i < bin; ++i) want -= sh.hist[i];
            last |= uint32_t(bin) << (8 * d);
        }
        __syncthreads();
        if (tid == 0) sh.n_out = 0;
        __syncthreads();
        each([&](bool on, uint64_t key, uint32_t flat) {
            if (on && (all || key > prefix || (key == prefix && flat <= last))) {
                const uint32_t at = atomicAdd(&sh.n_out, 1u);
                if (at < kMergeCap) {
                    sh.out_key[at] = key;
                    sh.out_flat[at] = flat;
                }
            }
        });
        __syncthreads();
    }

    // order the pairs: few by counting what precedes each, many by a bitonic sort
    const int n = int(min(sh.n_out, uint32_t(kMergeCap)));
    const uint64_t* keys = sh.out_key;
    const uint32_t* flats = sh.out_flat;
    if (n <= kMergeRank) {
        // 4 threads per pair
        const int k = tid / 4, part = tid & 3;
        int before = 0;
        uint64_t key = 0;
        uint32_t flat = 0;
        if (k < n) {
            key = sh.out_key[k];
            flat = sh.out_flat[k];
            for (int o = part; o < n; o += 4) {
                const uint64_t ko = sh.out_key[o];
                before += ko > key || (ko == key && sh.out_flat[o] < flat);
            }
        }
        before += __shfl_xor_sync(0xffffffffu, before, 1);
        before += __shfl_xor_sync(0xffffffffu, before, 2);
        if (k < n && part == 0) {  // the collected pairs are not needed any more
            sh.key[before] = key;
            sh.flat[before] = flat;
        }
        keys = sh.key;
        flats = sh.flat;
        __syncthreads();
    } else {
        int size = 32;
        while (size < n) size <<= 1;
        for (int i = n + tid; i < size; i += kMergeThreads) {
            sh.out_key[i] = 0;
            sh.out_flat[i] = 0xffffffffu;
        }
        __syncthreads();
        for (int k = 2; k <= size; k <<= 1)
            for (int j = k >> 1; j > 0; j >>= 1) {
                for (int t = tid; t < size / 2; t += kMergeThreads) {
                    const int lo = 2 * t - (t & (j - 1)), hi = lo + j;
                    const uint64_t ka = sh.out_key[lo], kb = sh.out_key[hi];
                    const uint32_t fa = sh.out_flat[lo], fb = sh.out_flat[hi];
                    const bool ordered = ka > kb || (ka == kb && fa < fb);
                    if (ordered != ((lo & k) == 0)) {
                        sh.out_key[lo] = kb;
                        sh.out_key[hi] = ka;
                        sh.out_flat[lo] = fb;
                        sh.out_flat[hi] = fa;
                    }
                }
                __syncthreads();
            }
    }
    for (int r = tid; r < a.keep; r += kMergeThreads) {
        const int64_t o = int64_t(b) * a.keep + r;
        float s = -INFINITY;
        int parent = -1, token = -1;
        bool done = false;
        if (r < n) {
            s = float(key_double(keys[r]));
            parent = int(flats[r] / uint32_t(a.V));
            token = int(flats[r] - uint32_t(parent) * uint32_t(a.V));
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
    return launch_dep(beam_merge_kernel, dim3(unsigned(a.B)), dim3(kMergeThreads), sizeof(MergeShared), s, a, stretches, cap,
                      static_cast<const Stretch*>(res), static_cast<const uint2*>(lists));
}

}  // namespace st
