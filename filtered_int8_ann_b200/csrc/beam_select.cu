// The best (beam, token) pairs of each request:
//   score(i, v) = scores[i] + x[i][v] - ln sum_u exp(x[i][u]),
// ordered by score descending, then i * V + v ascending.
//
// Two launches. The first reads the logits once, a CTA per stretch of one beam's logits, which pass
// through its registers in chunks of 16 KB: their maximum, the
// sum of exp(x - max), and the stretch's best entries. The second, a CTA per
// request, forms the beams' normalisers and picks among the entries.
//
// The order has to be that of the numbers themselves, up to a relative 2e-12 of the normalisers' sums, so everything that
// decides between beams is held in 64 bits: with scores near -20 an error of one fp32 rounding
// (2e-6) would swap neighbours of different beams once in a few hundred kept pairs. exp is
//   exp(x) = 2^(n/32) * (1 + r + r^2/2 + r^3/6 + r^4/24),  n = rint(32 x / ln2), r = x - n ln2/32, |r| <= ln2/64
// with r and all that follows in fp64 (relative error below 2e-12 of a term): six fp64 operations, two
// conversions and two shuffles (the 32 powers sit one per lane). n is taken in fp32, which may only make
// |r| a few percent larger.
//
// Best entries of a stretch: its threads' maxima go into a histogram between
// their least and largest; the bin edge with `keep` of them at or above it bounds
// the stretch's keep-th logit from below, so only the few logits above it are
// written. Where equal logits make them too many, a bisection over
// (logit, index) finds the exact border.
//
// 1024 beams of 100003 bf16 logits, a fifth of the beams finished (160 MB are read): 128 us for both launches, of which the
// second waits for the first to end (only its launch is hidden; profiled alone, with cold caches, they take 116 and 21); 24 us
// would be the bytes'. With none finished 160 us, as f16 162, as f32 206. Bound by instructions: 28 per logit (six of
// them in fp64), 60% of the issue slots busy; the exponentials are about half of the time. 128 beams of 1021
// logits: 14.5 us, each launch's chain of barriers.
#include <cfloat>
#include <type_traits>

#include "decode.cuh"

namespace st {

constexpr int kSelThreads = 256;
constexpr int kSelVecs = 4;        // 16-byte vectors of a chunk per thread
constexpr int kSelChunkBytes = kSelThreads * kSelVecs * 16;
constexpr int kSelPlaces = 4 * 148; // CTAs of the first launch that the GPU holds (three per SM with more registers: 129 us, not 122)
constexpr int kListCap = 2048;     // entries that a stretch collects
constexpr int kMergeThreads = 1024;
constexpr int kMergeCap = 2048;   // pairs sorted at the end
constexpr int kMergeRank = kMergeThreads / 4;  // up to this many are ordered by counting: one pass, no barriers
constexpr int kMergeUnits = 4096; // stretches listed as holding such pairs
constexpr int kHistBins = 256;
constexpr float kSelNear = 16384.f;  // stretches of larger logits are summed the plain way

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
    const uint64_t u = uint64_t(__double_as_longlong(x + 0.0));  // -0 becomes 0
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
    // the bits of word k's elements that are at least x, and which element of which word a bit stands for
    __device__ static uint32_t reach(uint32_t w, uint32_t x, int k) { return __uint_as_float(w) >= __uint_as_float(x) ? 1u << k : 0u; }
    __device__ static int word_of(int bit) { return bit; }
    __device__ static int part_of(int) { return 0; }
    // the next value above
    __device__ static uint32_t up(uint32_t w) { return w << 1 == 0 ? 1u : w >> 31 ? w - 1 : w + 1; }
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
    __device__ static uint32_t reach(uint32_t w, uint32_t x, int k) { return __hge2_mask(as(w), as(x)) & (0x10001u << k); }
    __device__ static int word_of(int bit) { return bit & 15; }
    __device__ static int part_of(int bit) { return bit >> 4; }
    __device__ static uint32_t up(uint32_t w)
    {
        const uint32_t h = w & 0xffffu, n = (h & 0x7fffu) == 0 ? 1u : h & 0x8000u ? h - 1 : h + 1;
        return n | n << 16;
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

// A value surely not above the far edge of histogram bin `bin` below m (every finite value when there is none,
// or it is the last, which also holds what lies further down).
__device__ __forceinline__ float edge_of(float m, float inv, int bin)
{
    if (bin < 0 || bin >= kHistBins - 1 || !(inv > 0.f)) return -FLT_MAX;
    return fmaxf(-FLT_MAX, m - float(bin + 1) / inv * 1.00001f - fabsf(m) * 0x1p-20f);
}

// An entry's order as one number: the logit, then the lower index.
__device__ __forceinline__ uint64_t entry_key(float x, uint32_t index) { return uint64_t(float_key(x)) << 32 | (0xffffffffu - index); }
__device__ __forceinline__ float key_float(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key); }

// The 16 bytes that begin SHIFT bytes behind the 16-byte boundary p, from aligned loads.
template <int SHIFT>
__device__ __forceinline__ void load_shifted(const void* p, uint32_t* out)
{
    constexpr int Q = SHIFT / 4, ODD = SHIFT % 4 != 0, MORE = Q + ODD;  // words taken from the next 16 bytes
    const uint4* q = static_cast<const uint4*>(p);
    const uint4 lo = __ldcs(q);
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, 0, 0, 0, 0};
    if (MORE == 1) {
        w[4] = __ldcs(reinterpret_cast<const uint32_t*>(q + 1));
    } else if (MORE == 2) {
        const uint2 hi = __ldcs(reinterpret_cast<const uint2*>(q + 1));
        w[4] = hi.x;
        w[5] = hi.y;
    } else if (MORE > 2) {
        const uint4 hi = __ldcs(q + 1);
        w[4] = hi.x;
        w[5] = hi.y;
        w[6] = hi.z;
        w[7] = hi.w;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) out[k] = ODD ? __funnelshift_r(w[k + Q], w[k + Q + (ODD ? 1 : 0)], 16) : w[k + Q];
}

// What a CTA of the first launch shares.
struct StretchShared {
    uint2 list[2][kListCap];  // entries (logit, token), in one of the two buffers
    float max[kSelThreads / 32], min[kSelThreads / 32];
    double sum[kSelThreads / 32];
    uint32_t hist[kHistBins];
    uint32_t count[4], total;  // entries found by chunk j: count[j % 4]
    int bin, slow;
};

// The largest key with at least `keep` keys at or above it among the list's n and those that `more` gives to its
// argument, by bisection. All threads of the CTA.
template <bool MORE, typename F>
__device__ uint64_t list_border(StretchShared& sh, const uint2* list, uint32_t n, uint32_t keep, F&& more)
{
    uint64_t border = 0;
    for (int bit = 63; bit >= 0; --bit) {
        const uint64_t mid = border | 1ull << bit;
        uint32_t c = 0;
        for (uint32_t k = threadIdx.x; k < n; k += kSelThreads) c += entry_key(__uint_as_float(list[k].x), list[k].y) >= mid;
        if (MORE) more([&](uint64_t key) { c += key >= mid; });
        c = __reduce_add_sync(0xffffffffu, c);
        if ((threadIdx.x & 31) == 0 && c) atomicAdd(&sh.total, c);
        __syncthreads();
        const uint32_t total = sh.total;
        __syncthreads();
        if (threadIdx.x == 0) sh.total = 0;
        __syncthreads();
        if (total >= keep) border = mid;
    }
    return border;
}

// Narrow a list of n entries in buffer `buf` to those that can be among its best `keep`, by a histogram; they go to
// the other buffer. False (and nothing done) when that cannot be told apart.
__device__ bool list_trim(StretchShared& sh, int buf, uint32_t& n, uint32_t keep, float& edge, bool& above)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float hi = -INFINITY, lo = INFINITY;
    for (uint32_t k = tid; k < n; k += kSelThreads) {
        const float y = __uint_as_float(sh.list[buf][k].x);
        hi = fmaxf(hi, y);
        lo = fminf(lo, y);
    }
    hi = warp_max(hi);
    lo = warp_min(lo);
    __syncthreads();
    if (lane == 0) {
        sh.max[warp] = hi;
        sh.min[warp] = lo;
    }
    sh.hist[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
        hi = fmaxf(hi, sh.max[w]);
        lo = fminf(lo, sh.min[w]);
    }
    const float inv = bin_scale(hi - lo, kHistBins);
    for (uint32_t k = tid; k < n; k += kSelThreads)
        atomicAdd(&sh.hist[min(kHistBins - 1, int((hi - __uint_as_float(sh.list[buf][k].x)) * inv))], 1u);
    __syncthreads();
    find_bin<kHistBins>(sh.hist, keep, &sh.bin);
    __syncthreads();
    const float e = edge_of(hi, inv, sh.bin);
    if (!(e > edge)) return false;  // the same in all threads
    for (uint32_t k = tid; k < n; k += kSelThreads) {  // (the total is 0 between uses)
        const uint2 w = sh.list[buf][k];
        if (__uint_as_float(w.x) >= e) sh.list[buf ^ 1][atomicAdd(&sh.total, 1u)] = w;
    }
    edge = e;
    above = false;
    __syncthreads();
    n = sh.total;
    __syncthreads();
    if (tid == 0) sh.total = 0;
    __syncthreads();
    return true;
}

template <typename T>
__global__ void __launch_bounds__(kSelThreads, 4)
beam_stretch_kernel(SelectArgs a, int stretches, int chunks, int cap, Stretch* res, uint2* lists)
{
    using L = Logit<T>;
    constexpr int PER = L::kPer, IN = L::kIn, VECS = kSelVecs, WORDS = VECS * 4, kSelChunk = kSelChunkBytes / int(sizeof(T));
    __shared__ StretchShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.y;
    const int64_t unit = int64_t(row) * stretches + blockIdx.x;
    const float base = a.scores[row];
    const bool finished = a.ex.finished && a.ex.finished[row];
    if (!(fabsf(base) < INFINITY) || finished) {  // no logit counts
        if (tid == 0) {
            Stretch s{0.0, -INFINITY, 0};
            if (finished && fabsf(base) < INFINITY && blockIdx.x == 0) {  // one candidate of logit 0 with normaliser 0
                s = Stretch{1.0, 0.f, 1};
                lists[unit * cap] = make_uint2(__float_as_uint(0.f), uint32_t(a.ex.end_token));
            }
            res[unit] = s;
        }
        return;
    }

    // Chunk j's first element is the row's element first + j kSelChunk. Which thread takes an element depends on its
    // index in the row alone, not on the row's alignment, so that equal rows have equal sums to the last bit and their
    // pairs stand in the order of the beams.
    const T* x = static_cast<const T*>(a.logits) + row * a.stride;
    const int before = int((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));  // elements behind a 16-byte boundary
    const int first = int(blockIdx.x) * chunks * kSelChunk;
    const uint32_t* allow = nullptr;
    if (a.ex.allow) {
        const int b = row / a.K;
        allow = a.ex.allow + b * a.ex.allow_request_stride + (row - b * a.K) * a.ex.allow_beam_stride;
    }
    // This thread's elements of the chunk at c, from a row that begins `shift` elements behind a 16-byte boundary; -inf
    // for those whose vectors are not all of the row.
    auto load_as = [&](auto shift, int c, uint32_t(&v)[WORDS]) {
        constexpr int SHIFT = decltype(shift)::value;
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int e = c + (j * kSelThreads + tid) * PER;
            v[4 * j] = v[4 * j + 1] = v[4 * j + 2] = v[4 * j + 3] = L::kNone;
            if (e >= SHIFT && e + (SHIFT ? 2 * PER - SHIFT : PER) <= a.V) load_shifted<SHIFT * int(sizeof(T))>(x + e - SHIFT, &v[4 * j]);
        }
    };
    const int reach = before ? 2 * PER - before : PER;
    auto load = [&](int c, uint32_t(&v)[WORDS]) {
        switch (before) {
            case 0: load_as(std::integral_constant<int, 0>{}, c, v); break;
            case 1: load_as(std::integral_constant<int, 1>{}, c, v); break;
            case 2: load_as(std::integral_constant<int, 2>{}, c, v); break;
            case 3: load_as(std::integral_constant<int, 3>{}, c, v); break;
            case 4: load_as(std::integral_constant<int, 4 % PER>{}, c, v); break;
            case 5: load_as(std::integral_constant<int, 5 % PER>{}, c, v); break;
            case 6: load_as(std::integral_constant<int, 6 % PER>{}, c, v); break;
            default: load_as(std::integral_constant<int, 7 % PER>{}, c, v); break;
        }
        const int e0 = c + tid * PER;
        if (e0 < before || e0 + (VECS - 1) * kSelThreads * PER + reach > a.V) {  // the rest, one by one
#pragma unroll
            for (int j = 0; j < VECS; ++j) {
                const int e = e0 + j * kSelThreads * PER;
                if (e >= a.V || (e >= before && e + reach <= a.V)) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w = L::kNone;
#pragma unroll
                    for (int u = 0; u < IN; ++u) {
                        const int at = e + k * IN + u;
                        if (at < a.V) {
                            if (IN == 1) w = L::bits(x, at);
                            else w = (w & (u ? 0xffffu : 0xffff0000u)) | L::bits(x, at) << (16 * u);
                        }
                    }
                    v[4 * j + k] = w;
                }
            }
        }
    };

    if (tid < 4) sh.count[tid] = 0;
    if (tid == 0) {
        sh.total = 0;
        sh.slow = 0;
    }
    __syncthreads();
    const uint32_t keep = uint32_t(a.keep);
    // the lane's power of two 2^(lane/32) as two words, the high one less what adding n << 15 brings from n's low bits
    const double power = kPowers32.v[lane];
    int power_hi = __double2hiint(power) - (lane << 15);
    const int power_lo = __double2loint(power);
    constexpr float kC = 46.166241308446828384f;  // 32 / ln 2
    constexpr float kMagic = 12582912.f;          // 1.5 * 2^23: adding it leaves the nearest integer in the low bits
    constexpr double kStep = 0.0216608493924982908;   // ln 2 / 32
    bool known = false;          // a reference for the exponentials: the maximum of the first chunk that has any
    float ref = 0.f, most = -INFINITY;
    int ref_exp = 0;             // the exponentials are held over 2^ref_exp, about exp(ref)
    double part[2] = {0.0, 0.0};
    uint32_t floor2 = 0;
    float edge = -FLT_MAX;       // entries from here up are candidates (`above`: only those above it)
    bool above = false;
    int buf = 0;
    uint32_t count = 0, fetched = 0;  // entries in the list, and those whose logits have been read into it
    auto fetch = [&]() {         // (an index is enough until then, and a load for each would be waited for)
        for (uint32_t k = fetched + tid; k < count; k += kSelThreads) sh.list[buf][k].x = __float_as_uint(L::one(x, sh.list[buf][k].y));
        fetched = count;
        __syncthreads();
    };

    // Pass 0 goes through the chunks without waiting for one another's candidates. Where they are more than the list
    // holds (equal logits, as a rule), pass 1 goes through them again, a chunk at a time.
    uint32_t v[WORDS];
    for (int pass = 0; pass < 2; ++pass) {
        for (int j = 0; j < chunks; ++j) {
            const int c0 = first + j * kSelChunk;
            if (c0 >= a.V) break;
            load(c0, v);
            // the row's index of element u of this thread's word k
            auto index_of = [&](int k, int u) { return c0 + ((k / 4) * kSelThreads + tid) * PER + (k % 4) * IN + u; };
            if (allow) {
#pragma unroll
                for (int i = 0; i < VECS; ++i) {
                    const int e = c0 + (i * kSelThreads + tid) * PER;  // a multiple of 8 or 4: the bits are one word's
                    if (e >= a.V) continue;
                    const uint32_t bits = allow[e >> 5] >> (e & 31);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[4 * i + k] = L::keep(v[4 * i + k], bits >> (k * IN));
                }
            }
            // this thread's maximum (NaN takes no part); +inf leaves
            uint32_t top = v[0];
#pragma unroll
            for (int k = 1; k < WORDS; ++k) top = L::max2(top, v[k]);
            float tmax = IN == 1 ? L::get(top, 0) : fmaxf(L::get(top, 0), L::get(top, 1));
            if (tmax == INFINITY) {
                tmax = -INFINITY;
#pragma unroll
                for (int k = 0; k < WORDS; ++k) {
                    uint32_t on = 0;
#pragma unroll
                    for (int u = 0; u < IN; ++u) {
                        const float y = L::get(v[k], u);
                        on |= (y < INFINITY ? 1u : 0u) << u;
                        if (y < INFINITY) tmax = fmaxf(tmax, y);
                    }
                    v[k] = L::keep(v[k], on);
                }
            }
            most = fmaxf(most, tmax);
            if (!known) {
                sh.hist[tid] = 0;
                const float wm = warp_max(tmax), wl = warp_min(tmax > -INFINITY ? tmax : INFINITY);
                if (lane == 0) {
                    sh.max[warp] = wm;
                    sh.min[warp] = wl;
                }
                __syncthreads();
                float m = sh.max[0], least = sh.min[0];
#pragma unroll
                for (int w = 1; w < kSelThreads / 32; ++w) {
                    m = fmaxf(m, sh.max[w]);
                    least = fminf(least, sh.min[w]);
                }
                if (!(m > -INFINITY)) {  // nothing allowed in this chunk
                    __syncthreads();
                    continue;
                }
                known = true;
                ref = m;
                ref_exp = __float2int_rn(fminf(fmaxf(m, -kSelNear), kSelNear) * 1.44269504f);
                power_hi -= ref_exp << 20;
                floor2 = L::both(m - 700.f);  // exp(-700) is nothing next to 1; takes the place of -inf and NaN
                if (fabsf(m) > kSelNear && tid == 0) sh.slow = 1;
                // The edge: the chunk's threads' (or, for many, vectors') maxima in a histogram; the bin that `keep` of them
                // reach bounds the chunk's keep-th logit from below.
                const float inv = bin_scale(m - least, kHistBins);
                if (keep <= kSelThreads / 2) {
                    if (tmax > -INFINITY) atomicAdd(&sh.hist[min(kHistBins - 1, int((m - tmax) * inv))], 1u);
                } else {
#pragma unroll
                    for (int i = 0; i < VECS; ++i) {
                        const uint32_t w = L::max2(L::max2(v[4 * i], v[4 * i + 1]), L::max2(v[4 * i + 2], v[4 * i + 3]));
                        const float y = IN == 1 ? L::get(w, 0) : fmaxf(L::get(w, 0), L::get(w, 1));
                        if (y >= least) atomicAdd(&sh.hist[min(kHistBins - 1, int((m - y) * inv))], 1u);
                    }
                }
                __syncthreads();
                find_bin<kHistBins>(sh.hist, keep, &sh.bin);
                __syncthreads();
                edge = edge_of(m, inv, sh.bin);
            }
            // candidates: their indexes go behind the list
            const uint32_t old = count;
            if (edge <= tmax) {  // (false where this thread has none)
                const uint32_t e2 = L::both(edge);
                // above the edge, which is an entry's value then; or from it on, a step further down where the type rounds it up
                const uint32_t from = above ? L::up(e2) : L::get(e2, 0) <= edge ? e2 : L::both(edge - fabsf(edge) * 0.01f - FLT_MIN);
                uint32_t found = 0;
#pragma unroll
                for (int k = 0; k < WORDS; ++k) found |= L::reach(v[k], from, k);
                if (found) {
                    uint32_t at = old + atomicAdd(&sh.count[pass == 0 ? 0 : j & 3], uint32_t(__popc(found)));
                    while (found) {
                        const int bit = __ffs(found) - 1;
                        found &= found - 1;
                        if (at < kListCap) sh.list[buf][at].y = uint32_t(index_of(L::word_of(bit), L::part_of(bit)));
                        ++at;
                    }
                }
            }
            // exp(x - ref)
            if (tmax - ref > 600.f) sh.slow = 1;
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                if (pass > 0 || i * kSelThreads * PER >= a.V - c0) break;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t w = L::max2(v[4 * i + k], floor2);
#pragma unroll
                    for (int u = 0; u < IN; ++u) {
                        const float y = L::get(w, u), t = fmaf(y, kC, kMagic);
                        const int n = __float_as_int(t);
                        const double r = fma(double(t - kMagic), -kStep, double(y));
                        const int hi = __shfl_sync(0xffffffffu, power_hi, n), lo = __shfl_sync(0xffffffffu, power_lo, n);
                        const double scaled = __hiloint2double(hi + (n << 15), lo);
                        const double p = fma(r, fma(r, fma(r, fma(r, 1.0 / 24, 1.0 / 6), 0.5), 1.0), 1.0);
                        part[(k + u) & 1] = fma(scaled, p, part[(k + u) & 1]);
                    }
                }
            }
            if (pass == 0) continue;
            __syncthreads();
            count = old + sh.count[j & 3];
            if (tid == 0) sh.count[(j + 2) & 3] = 0;  // read last two barriers ago
            if (count > kListCap) {
                // Too many: exactly the best `keep` of the list and this chunk's candidates (the logit's order first, then
                // the lower index). Later entries that equal the last of them come behind it.
                count = old;
                fetch();
                const uint64_t border = list_border<true>(sh, sh.list[buf], old, keep, [&](auto&& f) {
#pragma unroll
                    for (int k = 0; k < WORDS; ++k)
#pragma unroll
                        for (int u = 0; u < IN; ++u) {
                            const float y = L::get(v[k], u);
                            if (y > -INFINITY && (above ? y > edge : y >= edge)) f(entry_key(y, uint32_t(index_of(k, u))));
                        }
                });
                if (tid == 0) sh.total = 0;
                __syncthreads();
                auto take = [&](uint64_t key) {
                    if (key >= border) {
                        const uint32_t at = atomicAdd(&sh.total, 1u);
                        if (at < kListCap) sh.list[buf ^ 1][at] = make_uint2(__float_as_uint(key_float(uint32_t(key >> 32))), 0xffffffffu - uint32_t(key));
                    }
                };
                for (uint32_t k = tid; k < old; k += kSelThreads) take(entry_key(__uint_as_float(sh.list[buf][k].x), sh.list[buf][k].y));
#pragma unroll
                for (int k = 0; k < WORDS; ++k)
#pragma unroll
                    for (int u = 0; u < IN; ++u) {
                        const float y = L::get(v[k], u);
                        if (y > -INFINITY && (above ? y > edge : y >= edge)) take(entry_key(y, uint32_t(index_of(k, u))));
                    }
                buf ^= 1;
                edge = key_float(uint32_t(border >> 32));
                above = true;
                __syncthreads();
                count = fetched = min(sh.total, uint32_t(kListCap));
                __syncthreads();
                if (tid == 0) sh.total = 0;
            } else if (count > kListCap / 2 && j + 1 < chunks) {
                fetch();
                if (list_trim(sh, buf, count, keep, edge, above)) buf ^= 1;
                fetched = count;
            }
        }
        if (pass > 0) break;
        __syncthreads();
        count = sh.count[0];
        if (count <= kListCap) break;
        count = 0;
        __syncthreads();
        if (tid == 0) sh.count[0] = 0;
        __syncthreads();
    }
    if (!known) {  // nothing allowed here
        if (tid == 0) res[unit] = Stretch{0.0, -INFINITY, 0};
        return;
    }

    // the sum, over the maximum
    double sum = part[0] + part[1];
    const float wm = warp_max(most);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) {
        sh.max[warp] = wm;
        sh.sum[warp] = sum;
    }
    __syncthreads();
    float m = sh.max[0];
#pragma unroll
    for (int w = 1; w < kSelThreads / 32; ++w) m = fmaxf(m, sh.max[w]);
    double total = 0.0;
    if (sh.slow) {  // logits too far apart for one reference: once more from memory, the plain way
        double s = 0.0;
        const int end = min(a.V, first + chunks * kSelChunk);
#pragma unroll 1
        for (int e = first + tid; e < end; e += kSelThreads) {
            const float y = L::one(x, e);
            const double d = double(y) - double(m);
            if ((!allow || (allow[e >> 5] >> (e & 31) & 1u)) && y < INFINITY && d >= -700.0) s += exp(d);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        __syncthreads();
        if (lane == 0) sh.sum[warp] = s;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSelThreads / 32; ++w) total += sh.sum[w];
    } else {
#pragma unroll
        for (int w = 0; w < kSelThreads / 32; ++w) total += sh.sum[w];
        total *= exp(ref_exp * 0.693147180559945309417 - double(m));
    }
    // the entries: no more than a list holds
    __syncthreads();
    fetch();
    if (count > uint32_t(cap) && list_trim(sh, buf, count, keep, edge, above)) buf ^= 1;
    if (count > uint32_t(cap)) {
        const uint64_t border = list_border<false>(sh, sh.list[buf], count, keep, [](auto&&) {});
        for (uint32_t k = tid; k < count; k += kSelThreads) {
            const uint2 w = sh.list[buf][k];
            if (entry_key(__uint_as_float(w.x), w.y) >= border) {
                const uint32_t at = atomicAdd(&sh.total, 1u);
                if (at < uint32_t(cap)) sh.list[buf ^ 1][at] = w;
            }
        }
        buf ^= 1;
        __syncthreads();
        count = min(sh.total, uint32_t(cap));
    }
    uint2* list = lists + unit * cap;
    for (uint32_t k = tid; k < count; k += kSelThreads) list[k] = sh.list[buf][k];
    if (tid == 0) res[unit] = Stretch{total, m, int32_t(count)};
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

// Chunks per stretch: as many as leave the GPU three CTAs per place (kSelPlaces; a stretch's first chunk and its end
// cost about a chunk more), and their candidates (keep and a few more each) the list's room, at most 16. 
static int select_chunks(int64_t rows, int32_t V, int32_t keep, int size)
{
    const int chunk = kSelChunkBytes / size;
    const int64_t all = (V + chunk - 1) / chunk;
    int64_t chunks = rows * all / (3 * kSelPlaces);
    if (chunks > kListCap / 2 / keep) chunks = kListCap / 2 / keep;
    return int(chunks < 1 ? 1 : chunks > 16 ? 16 : chunks > all ? all : chunks);
}
static int select_stretches(int64_t rows, int32_t V, int32_t keep, int size)
{
    const int64_t stretch = int64_t(select_chunks(rows, V, keep, size)) * (kSelChunkBytes / size);
    return int((V + stretch - 1) / stretch);
}
// Entries a stretch may write: room for the bin that holds the border.
static int select_cap(int32_t V, int32_t keep)
{
    return keep + 64 < V ? keep + 64 : V;
}

int64_t beam_select_workspace(int32_t B, int32_t K, int32_t V, int32_t keep)
{
    // the type is not known here: the longest, whose stretches are the most
    const int64_t rows = int64_t(B) * K;
    const int two = select_stretches(rows, V, keep, 2), four = select_stretches(rows, V, keep, 4);
    const int64_t units = rows * (two > four ? two : four);
    return units * int64_t(sizeof(Stretch)) + units * select_cap(V, keep) * 8;
}

cudaError_t launch_beam_select(const SelectArgs& a, cudaStream_t s)
{
    const int64_t rows = int64_t(a.B) * a.K;
    const int size = a.dtype == ST_F32 ? 4 : 2;
    const int chunks = select_chunks(rows, a.V, a.keep, size), stretches = select_stretches(rows, a.V, a.keep, size);
    const int cap = select_cap(a.V, a.keep);
    Stretch* res = static_cast<Stretch*>(a.workspace);
    uint2* lists = reinterpret_cast<uint2*>(res + rows * stretches);
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(beam_merge_kernel), int(sizeof(MergeShared)));
    if (e != cudaSuccess) return e;
    // grid y is at most 65535 rows
    const int64_t step = 65535 / a.K * int64_t(a.K);
    for (int64_t r0 = 0; r0 < rows; r0 += step) {
        const dim3 grid(unsigned(stretches), unsigned(rows - r0 < step ? rows - r0 : step));
        SelectArgs p = a;
        p.logits = static_cast<const char*>(a.logits) + r0 * a.stride * size;
        p.scores += r0;
        if (p.ex.finished) p.ex.finished += r0;
        if (p.ex.allow) p.ex.allow += r0 / a.K * a.ex.allow_request_stride;
        Stretch* pr = res + r0 * stretches;
        uint2* pl = lists + r0 * stretches * cap;
        switch (a.dtype) {
            case ST_BF16: beam_stretch_kernel<__nv_bfloat16><<<grid, kSelThreads, 0, s>>>(p, stretches, chunks, cap, pr, pl); break;
            case ST_F16: beam_stretch_kernel<__half><<<grid, kSelThreads, 0, s>>>(p, stretches, chunks, cap, pr, pl); break;
            default: beam_stretch_kernel<float><<<grid, kSelThreads, 0, s>>>(p, stretches, chunks, cap, pr, pl); break;
        }
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return launch_dep(beam_merge_kernel, dim3(unsigned(a.B)), dim3(kMergeThreads), sizeof(MergeShared), s, a, stretches, cap,
                      static_cast<const Stretch*>(res), static_cast<const uint2*>(lists));
}

}  // namespace st
