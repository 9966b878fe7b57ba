// Quantise new keys and values into an int8 paged cache with one scale per
// block and head.
//
// Consecutive tokens whose slots follow each other inside one block form a
// run: the unit of work, since they share the block's scale
//   s = max(s0, amax / 127),  codes = rint(x / s),  earlier codes *= s0 / s.
// A run is found where it starts (the token before has another block or does
// not precede in it). A CTA looks at the starts among a few consecutive
// tokens, for one head and one of K and V. Short runs (one token per row in a decode step) go to
// its warps one each; longer ones (prompts) take the whole CTA, and every
// element is read once: it waits in registers while the run's maximum is
// found. Maxima are taken on the 16-bit patterns, two at a time, and codes rounded by adding 1.5 * 2^23:
// with conversions to integers one by one the prompts' case below took 65 us.
//
// Bound by bytes: 2 read and 1 written per new element, and the earlier codes
// of the blocks whose scale grew. 14343 tokens of 8 heads of 128 (88 MB): 20.6 us, 4.3 TB/s of them; the wait between a
// run's loads and its stores, and the instructions of the conversion (issue slots over half busy), keep it from the
// copy's rate. A step of 256 rows: 8 us, two dependent loads and a launch.
#include "decode.cuh"

namespace st {

constexpr int kAppendBlock = 128;
constexpr int kAppendWarpRun = 8;  // longest run (tokens) that one warp takes

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t x);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t x)
{
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t x)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// |x| where x is finite, else 0
__device__ __forceinline__ float finite_abs(float x)
{
    x = fabsf(x);
    return x < INFINITY ? x : 0.f;
}

__device__ __forceinline__ uint32_t code_byte(float y)
{
    // rint, limited; NaN gives 0 (the conversion's result for NaN)
    return uint32_t(max(-127, min(127, __float2int_rn(y)))) & 0xffu;
}

// Magnitudes of 16-bit floats order like their bits without the sign; those from kInf on are infinities and NaN.
template <typename T>
struct Bits;
template <>
struct Bits<__nv_bfloat16> { static constexpr uint32_t kInf = 0x7f80u; };
template <>
struct Bits<__half> { static constexpr uint32_t kInf = 0x7c00u; };

__device__ __forceinline__ uint32_t peak8(const uint4& x)
{
    const uint32_t a = __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), b = __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu);
    return __vmaxu2(a, b);
}

// The largest finite magnitude of eight, one by one.
template <typename T>
__device__ __forceinline__ float amax8(const uint4& x)
{
    float m = 0.f;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T>(w[i]);
        m = fmaxf(m, fmaxf(finite_abs(f.x), finite_abs(f.y)));
    }
    return m;
}

// Adding 1.5 * 2^23 rounds to the nearest integer (ties to even), which then stands in the low bits.
constexpr float kRound = 12582912.f;

__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d)
{
    const uint32_t ab = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
    const uint32_t cd = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040);
    return __byte_perm(ab, cd, 0x5410);
}

// Codes of eight finite values: |x turn| is at most 127 and a rounding, which rounds to 127.
template <typename T>
__device__ __forceinline__ uint2 codes8(const uint4& x, float turn)
{
    const float2 a = unpack2<T>(x.x), b = unpack2<T>(x.y), c = unpack2<T>(x.z), d = unpack2<T>(x.w);
    return make_uint2(low_bytes(__fmul_rn(a.x, turn) + kRound, __fmul_rn(a.y, turn) + kRound, __fmul_rn(b.x, turn) + kRound,
                                __fmul_rn(b.y, turn) + kRound),
                      low_bytes(__fmul_rn(c.x, turn) + kRound, __fmul_rn(c.y, turn) + kRound, __fmul_rn(d.x, turn) + kRound,
                                __fmul_rn(d.y, turn) + kRound));
}

// Codes of eight values of any kind.
template <typename T>
__device__ __noinline__ uint2 codes8_any(uint4 x, float turn)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T>(w[i]);
        out[i >> 1] |= (code_byte(__fmul_rn(f.x, turn)) | code_byte(__fmul_rn(f.y, turn)) << 8) << (16 * (i & 1));
    }
    return make_uint2(out[0], out[1]);
}

// Four codes times a ratio of at most 1. A byte 128 + code below 0x4b0000 is the float 2^23 + 128 + code.
__device__ __forceinline__ uint32_t moved4(uint32_t w, float ratio)
{
    const uint32_t u = w ^ 0x80808080u;
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = __fmul_rn(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.f, ratio) + kRound;
    return low_bytes(f[0], f[1], f[2], f[3]);
}

// Maximum over a group of N threads (a warp, or the whole CTA).
template <int N>
__device__ __forceinline__ uint32_t group_max(uint32_t m, uint32_t* part)
{
    m = __reduce_max_sync(0xffffffffu, m);
    if (N > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N / 32; ++i) m = max(m, part[i]);
    }
    return m;
}

// One run of n tokens from token t, at offset `off` of block `page`, its
// earlier tokens in block `src`, by N threads (rank `me`), up to VEC vectors
// of 8 elements each.
template <typename T, int D, int S, int N, int VEC>
__device__ __forceinline__ void append_run(const T* x, int64_t token_stride, int64_t t, int n, int8_t* codes,
                                           float* scales, int heads, int head, int page, int off, int src, int me,
                                           uint32_t* part)
{
    constexpr int V = D / 8;  // vectors per token
    const int64_t to = int64_t(page) * heads + head, from = int64_t(src) * heads + head;
    const float s0 = off > 0 ? scales[from] : 0.f;
    uint4 held[VEC];
    uint32_t peak = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int j = i * N + me;
        held[i] = make_uint4(0, 0, 0, 0);
        if (j < n * V) held[i] = __ldcs(reinterpret_cast<const uint4*>(x + (t + j / V) * token_stride) + j % V);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) peak = __vmaxu2(peak, peak8(held[i]));
    peak = group_max<N>(max(peak & 0xffffu, peak >> 16), part);  // every thread of the group has read s0 by now
    const bool finite = peak < Bits<T>::kInf;
    float m = unpack2<T>(peak).x;
    if (!finite) {
        m = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = fmaxf(m, amax8<T>(held[i]));
        m = __uint_as_float(group_max<N>(__float_as_uint(m), part));
    }
    float s = fmaxf(s0, __fdiv_rn(m, 127.f));
    s = s > 0x1p-100f ? s : 0.f;
    const float turn = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
    int8_t* out = codes + to * S * D;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int j = i * N + me;
        if (j < n * V) reinterpret_cast<uint2*>(out + off * D)[j] = finite ? codes8<T>(held[i], turn) : codes8_any<T>(held[i], turn);
    }
    if (off > 0 && (s != s0 || src != page)) {
        const float ratio = s > 0.f ? __fdiv_rn(s0, s) : 0.f;
        const uint4* a = reinterpret_cast<const uint4*>(codes + from * S * D);
        uint4* b = reinterpret_cast<uint4*>(out);
        for (int j = me; j < off * D / 16; j += N) {
            uint4 w = a[j];
            w.x = moved4(w.x, ratio);
            w.y = moved4(w.y, ratio);
            w.z = moved4(w.z, ratio);
            w.w = moved4(w.w, ratio);
            b[j] = w;
        }
    }
    if (me == 0) scales[to] = s;
}

// CTAs that an SM shall hold: eight where a thread holds up to eight vectors of a long run (64 registers are enough then:
// 14343 tokens 20.6 us, with the five of 84 registers 24), else as many as come.
constexpr int append_ctas(int D, int S, int per) { return per > 4 && S * D / 8 <= 8 * kAppendBlock ? 8 : 0; }

// PER: tokens whose runs a CTA takes.
template <typename T, int D, int S, int PER>
__global__ void __launch_bounds__(kAppendBlock, append_ctas(D, S, PER)) kv_append_kernel(AppendArgs a)
{
    constexpr int WINDOW = (PER + S + 31) / 32 * 32;  // tokens that runs starting here can reach, and more
    __shared__ int64_t s_slot[WINDOW];
    __shared__ uint32_t s_last[WINDOW / 32];          // bit: the token is the last of its run
    __shared__ uint32_t s_start[(PER + 31) / 32];     // bit: the first
    __shared__ uint32_t part[kAppendBlock / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const int heads = a.c.kv_heads;
    const int64_t limit = int64_t(a.c.num_blocks) * S, t0 = int64_t(blockIdx.x) * PER;

    // slots of the window; -1 for none
    const int64_t before = t0 > 0 ? a.slots[t0 - 1] : -1;
#pragma unroll
    for (int i0 = 0; i0 < WINDOW; i0 += kAppendBlock) {
        const int i = i0 + tid;
        if (i < WINDOW) {
            int64_t slot = t0 + i < a.T ? a.slots[t0 + i] : -1;
            if (slot >= limit) {
                slot = -1;
                if (i < PER) atomicOr(a.err, kDecErrSlot);
            }
            s_slot[i] = slot;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i0 = 0; i0 < WINDOW; i0 += kAppendBlock) {
        const int i = i0 + tid;  // whole warps
        if (i < WINDOW) {
            const int64_t slot = s_slot[i], next = i + 1 < WINDOW ? s_slot[i + 1] : -1, prev = i > 0 ? s_slot[i - 1] : before;
            const unsigned last = __ballot_sync(0xffffffffu, next != slot + 1 || (next & (S - 1)) == 0);
            const unsigned first = __ballot_sync(0xffffffffu, i < PER && slot >= 0 && (prev != slot - 1 || (slot & (S - 1)) == 0));
            if (lane == 0) {
                s_last[i / 32] = last;
                if (i < PER) s_start[i / 32] = first;
            }
        }
    }
    __syncthreads();
    const T* x = static_cast<const T*>(is_v ? a.v : a.k) + head * (is_v ? a.v_head : a.k_head);
    const int64_t stride = is_v ? a.v_token : a.k_token;
    int8_t* codes = is_v ? a.c.v : a.c.k;
    float* scales = is_v ? a.c.v_scale : a.c.k_scale;
    int nth = 0;
    for (int w = 0; w < (PER + 31) / 32; ++w) {
        for (uint32_t starts = s_start[w]; starts; starts &= starts - 1, ++nth) {
            const int at = w * 32 + __ffs(starts) - 1;
            int end = at >> 5;  // word of the run's last token, then that token
            uint32_t lasts = s_last[end] & ~0u << (at & 31);
            while (!lasts) lasts = s_last[++end];
            end = end * 32 + __ffs(lasts) - 1;
            const int n = end - at + 1;
            const int64_t slot = s_slot[at];
            const int page = int(slot / S), off = int(slot & (S - 1));
            const bool small = n <= kAppendWarpRun;
            if (small && (nth & (kAppendBlock / 32 - 1)) != warp) continue;
            const int src = a.sources && off > 0 ? a.sources[t0 + at] : page;
            if (src < 0 || src >= a.c.num_blocks) {
                if (lane == 0) atomicOr(a.err, kDecErrSlot);
                continue;
            }
            if (small)
                append_run<T, D, S, 32, (kAppendWarpRun * D / 8 + 31) / 32>(x, stride, t0 + at, n, codes, scales, heads, head,
                                                                           page, off, src, lane, part);
            else
                append_run<T, D, S, kAppendBlock, (S * D / 8 + kAppendBlock - 1) / kAppendBlock>(
                    x, stride, t0 + at, n, codes, scales, heads, head, page, off, src, tid, part);
        }
    }
}

template <typename T, int D, int S>
static cudaError_t launch_append(const AppendArgs& a, cudaStream_t s)
{
    // Tokens per CTA: 4 while that leaves the CTAs few (a decode step: a run per warp; 256 tokens of 8 heads 8 us, with a
    // block's tokens per CTA 12), else a block's, so that a prompt's CTAs have one run each (14343 tokens: 20.6 us, with 4
    // tokens per CTA 70). The rule sees no run lengths: prompts of few tokens in all are slower than they need be (one of 4096
    // tokens and 8 heads 21 us, one of 4097 6.6).
    const bool few = a.T * a.c.kv_heads <= 32768;
    const int per = few ? 4 : S;
    const dim3 grid(unsigned((a.T + per - 1) / per), unsigned(a.c.kv_heads), 2);
    if (few) kv_append_kernel<T, D, S, 4><<<grid, kAppendBlock, 0, s>>>(a);
    else kv_append_kernel<T, D, S, S><<<grid, kAppendBlock, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t launch_append(const AppendArgs& a, cudaStream_t s)
{
    switch (a.c.block_size) {
        case 16: return launch_append<T, D, 16>(a, s);
        case 32: return launch_append<T, D, 32>(a, s);
        case 64: return launch_append<T, D, 64>(a, s);
        default: return launch_append<T, D, 128>(a, s);
    }
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s)
{
    if (a.c.head_dim == 128)
        return a.dtype == ST_BF16 ? launch_append<__nv_bfloat16, 128>(a, s) : launch_append<__half, 128>(a, s);
    return a.dtype == ST_BF16 ? launch_append<__nv_bfloat16, 64>(a, s) : launch_append<__half, 64>(a, s);
}

}  // namespace st
