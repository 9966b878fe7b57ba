// Attention over an int8 paged cache.
#include "decode.cuh"

namespace st {

constexpr int kAttendBlock = 128;

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// A CTA per query token and head: a key per thread, then an output element per thread.
template <typename T, int D>
__global__ void __launch_bounds__(kAttendBlock) kv_attend_kernel(AttendArgs a)
{
    __shared__ float s_q[D], s_w[kAttendBlock], s_vs[kAttendBlock], s_red[kAttendBlock / 32];
    __shared__ int64_t s_at[kAttendBlock];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, hk = h / (a.q_heads / a.c.kv_heads);
    int lo = 0, hi = a.R;  // the row holding token t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.row_start[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    if (lo == a.R || a.row_start[lo] > t) return;
    const int start = a.row_start[lo], n = a.row_start[lo + 1] - start;
    int64_t len = a.lens[lo];
    T* out = static_cast<T*>(a.out) + t * a.out_token + h * a.out_head;
    if (len > a.max_len || n > a.max_q) {
        if (tid == 0) atomicOr(a.err, kDecErrRow);
        len = 0;
    }
    if (a.causal) len = min(len, len - n + (t - start) + 1);
    const T* q = static_cast<const T*>(a.q) + t * a.q_token + h * a.q_head;
    for (int d = tid; d < D; d += kAttendBlock) s_q[d] = to_float(q[d]);
    const int S = a.c.block_size, heads = a.c.kv_heads;
    __syncthreads();
    bool finite = true;
    for (int d = 0; d < D; ++d) finite = finite && fabsf(s_q[d]) < INFINITY;
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int64_t j0 = 0; j0 < len; j0 += kAttendBlock) {
        __syncthreads();
        const int64_t j = j0 + tid;
        float s = -INFINITY;
        if (j < len) {
            const int page = a.table[int64_t(lo) * a.max_blocks + j / S];
            if (page < 0 || page >= a.c.num_blocks) {
                atomicOr(a.err, kDecErrTable);
            } else {
                const int64_t head = int64_t(page) * heads + hk, row = head * S + j % S;
                const int8_t* k = a.c.k + row * D;
                float dot = 0.f;
                for (int d = 0; d < D; d += 16) {
                    const int4 w = *reinterpret_cast<const int4*>(k + d);
                    const int8_t* c = reinterpret_cast<const int8_t*>(&w);
                    for (int u = 0; u < 16; ++u) dot = fmaf(s_q[d + u], float(c[u]), dot);
                }
                s = dot * a.c.k_scale[head] * a.scale_log2;
                s_at[tid] = row * D;
                s_vs[tid] = a.c.v_scale[head];
            }
        }
        float mm = s;
        for (int off = 16; off > 0; off >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, off));
        if (lane == 0) s_red[warp] = mm;
        __syncthreads();
        mm = m;
        for (int w = 0; w < kAttendBlock / 32; ++w) mm = fmaxf(mm, s_red[w]);
        const float shrink = mm > -INFINITY ? exp2f(m - mm) : 1.f;
        m = mm;
        s_w[tid] = s > -INFINITY ? exp2f(s - m) : 0.f;
        __syncthreads();
        o *= shrink;
        l *= shrink;
        const int keys = int(min(int64_t(kAttendBlock), len - j0));
        for (int u = 0; u < keys; ++u) {
            const float w = s_w[u];
            l += w;
            if (tid < D && w > 0.f) o = fmaf(w * s_vs[u], float(a.c.v[s_at[u] + tid]), o);
        }
    }
    if (tid < D) out[tid] = from_float<T>(!finite && len > 0 ? NAN : l > 0.f ? o / l : 0.f);
}

int64_t kv_attend_workspace(const st_kv_cache&, int64_t, int32_t, int32_t, int32_t, int64_t) { return 0; }

cudaError_t launch_kv_attend(const AttendArgs& a, cudaStream_t s)
{
    const dim3 grid(unsigned(a.T), unsigned(a.q_heads));
    const bool bf = a.dtype == ST_BF16;
    if (a.c.head_dim == 128) {
        if (bf) kv_attend_kernel<__nv_bfloat16, 128><<<grid, kAttendBlock, 0, s>>>(a);
        else kv_attend_kernel<__half, 128><<<grid, kAttendBlock, 0, s>>>(a);
    } else {
        if (bf) kv_attend_kernel<__nv_bfloat16, 64><<<grid, kAttendBlock, 0, s>>>(a);
        else kv_attend_kernel<__half, 64><<<grid, kAttendBlock, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace st
