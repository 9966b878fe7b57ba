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
// found.
//
// Bound by bytes: 2 read and 1 written per new element, and the earlier codes
// of the blocks whose scale grew.
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

template <typename T>
__device__ __forceinline__ uint2 codes8(const uint4& x, float turn)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T>(w[i]);
        out[i >> 1] |= (code_byte(f.x * turn) | code_byte(f.y * turn) << 8) << (16 * (i & 1));
    }
    return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ uint32_t moved4(uint32_t w, float ratio)
{
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) out |= code_byte(float(int8_t(w >> (8 * i))) * ratio) << (8 * i);
    return out;
}

// Maximum over a group of N threads (a warp, or the whole CTA).
template <int N>
__device__ __forceinline__ float group_max(float m, float* part)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (N > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N / 32; ++i) m = fmaxf(m, part[i]);
    }
    return m;
}

// One run of n tokens from token t, at offset `off` of block `page`, its
// earlier tokens in block `src`, by N threads (rank `me`), up to VEC vectors
// of 8 elements each.
template <typename T, int D, int N, int VEC>
__device__ void append_run(const T* x, int64_t token_stride, int64_t t, int n, int8_t* codes, float* scales,
                           int heads, int head, int S, int page, int off, int src, int me, float* part)
{
    constexpr int V = D / 8;  // vectors per token
    uint4 held[VEC];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int j = i * N + me;
        held[i] = make_uint4(0, 0, 0, 0);
        if (j < n * V) held[i] = __ldg(reinterpret_cast<const uint4*>(x + (t + j / V) * token_stride) + j % V);
    }
    const int64_t to = int64_t(page) * heads + head, from = int64_t(src) * heads + head;
    const float s0 = off > 0 ? scales[from] : 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) m = fmaxf(m, amax8<T>(held[i]));
    m = group_max<N>(m, part);  // every thread of the group has read s0 by now
    float s = fmaxf(s0, __fdiv_rn(m, 127.f));
    s = s > 0x1p-100f ? s : 0.f;
    const float turn = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
    int8_t* out = codes + to * S * D;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int j = i * N + me;
        if (j < n * V) reinterpret_cast<uint2*>(out + int64_t(off) * D)[j] = codes8<T>(held[i], turn);
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

template <typename T, int D>
__global__ void __launch_bounds__(kAppendBlock) kv_append_kernel(AppendArgs a, int per_cta)
{
    __shared__ float part[kAppendBlock / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const T* x = static_cast<const T*>(is_v ? a.v : a.k) + head * (is_v ? a.v_head : a.k_head);
    const int64_t stride = is_v ? a.v_token : a.k_token;
    int8_t* codes = is_v ? a.c.v : a.c.k;
    float* scales = is_v ? a.c.v_scale : a.c.k_scale;
    const int S = a.c.block_size, heads = a.c.kv_heads;
    const int64_t limit = int64_t(a.c.num_blocks) * S;
    const int64_t t0 = int64_t(blockIdx.x) * per_cta;

    // the starts among tokens t0 .. t0 + per_cta (at most 32), the same in every warp
    const int64_t t = t0 + lane;
    int64_t slot = -1;
    bool start = false;
    if (lane < per_cta && t < a.T) {
        slot = a.slots[t];
        if (slot >= limit) {
            slot = -1;
            if (warp == 0) atomicOr(a.err, kDecErrSlot);
        }
        if (slot >= 0) start = slot % S == 0 || t == 0 || a.slots[t - 1] != slot - 1;
    }
    unsigned starts = __ballot_sync(0xffffffffu, start);
    for (int nth = 0; starts; ++nth) {
        const int at = __ffs(starts) - 1;
        starts &= starts - 1;
        const int64_t tr = t0 + at, first = __shfl_sync(0xffffffffu, slot, at);
        const int page = int(first / S), off = int(first - int64_t(page) * S);
        // length: tokens that follow on, inside the block
        int n = 0;
        for (int i0 = 0; i0 < S - off; i0 += 32) {
            const int i = i0 + lane;
            const bool on = i < S - off && tr + i < a.T && a.slots[tr + i] == first + i;
            const unsigned ons = __ballot_sync(0xffffffffu, on);
            const int run = ons == 0xffffffffu ? 32 : __ffs(~ons) - 1;
            n += run;
            if (run < 32) break;
        }
        int src = a.sources ? a.sources[tr] : page;
        if (off > 0 && (src < 0 || src >= a.c.num_blocks)) {
            if (threadIdx.x == 0) atomicOr(a.err, kDecErrSlot);
            continue;
        }
        if (n <= kAppendWarpRun) {
            if (nth % (kAppendBlock / 32) == warp)
                append_run<T, D, 32, kAppendWarpRun * D / 8 / 32>(x, stride, tr, n, codes, scales, heads, head, S,
                                                                  page, off, src, lane, part);
        } else if (n <= 32) {
            append_run<T, D, kAppendBlock, 32 * D / 8 / kAppendBlock>(x, stride, tr, n, codes, scales, heads, head, S,
                                                                      page, off, src, int(threadIdx.x), part);
        } else {
            append_run<T, D, kAppendBlock, 128 * D / 8 / kAppendBlock>(x, stride, tr, n, codes, scales, heads, head, S,
                                                                       page, off, src, int(threadIdx.x), part);
        }
    }
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s)
{
    // Tokens per CTA: 4 while that leaves the GPU's CTAs few (a decode step: a run per warp), else 16, the least
    // block size, so that a prompt's CTAs hold one or two starts.
    const int per_cta = a.T * a.c.kv_heads <= 32768 ? 4 : 16;
    const dim3 grid(unsigned((a.T + per_cta - 1) / per_cta), unsigned(a.c.kv_heads), 2);
    const bool bf = a.dtype == ST_BF16;
    if (a.c.head_dim == 128) {
        if (bf) kv_append_kernel<__nv_bfloat16, 128><<<grid, kAppendBlock, 0, s>>>(a, per_cta);
        else kv_append_kernel<__half, 128><<<grid, kAppendBlock, 0, s>>>(a, per_cta);
    } else {
        if (bf) kv_append_kernel<__nv_bfloat16, 64><<<grid, kAppendBlock, 0, s>>>(a, per_cta);
        else kv_append_kernel<__half, 64><<<grid, kAppendBlock, 0, s>>>(a, per_cta);
    }
    return cudaGetLastError();
}

}  // namespace st
