// Small device helpers that the attention kernels share.
#pragma once
#include "decode.cuh"

namespace st {

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// Eight 16-bit floats.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float* x)
{
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = __uint_as_float(a[i] << 16);
            x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// For big in [2^e, 2^(e+1)): 2^-e, which takes it to [1, 2), and 2^e. The exponent
// is limited to what both have normal numbers for (a smaller value, or 0, only
// stays smaller).
__device__ __forceinline__ float pow2_down(float big)
{
    const int e = min(max(int(__float_as_uint(big) >> 23) - 127, -126), 126);
    return __uint_as_float(uint32_t(127 - e) << 23);
}
__device__ __forceinline__ float pow2_up(float big)
{
    const int e = min(max(int(__float_as_uint(big) >> 23) - 127, -126), 126);
    return __uint_as_float(uint32_t(127 + e) << 23);
}

// Scores from here on are rounded before the maximum is taken off: the product that fma(s, factor, -max) holds exactly
// may differ from its rounded value, and so from the maximum, by more than a weight may be off.
constexpr float kScoreFar = 0x1p20f;
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kScoreFar && m > -INFINITY; }
// A little above x, so that no product rounded to x exceeds it (x itself for -inf and where scores are rounded).
__device__ __forceinline__ float just_above(float x) { return fabsf(x) < kScoreFar ? fmaxf(x, fmaf(fabsf(x), 0x1p-22f, x)) : x; }

// Bytes 128 + code (a code with its sign bit flipped) to fp16 codes, two per
// register: 0x64 above a byte b is 1024 + b.
__device__ __forceinline__ void biased_to_half(uint32_t x, uint32_t& lo, uint32_t& hi)
{
    const uint32_t bias = 0x64806480u;  // 1152
    uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 u = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<const __half2*>(&bias));
    const __half2 v = __hsub2(*reinterpret_cast<__half2*>(&b), *reinterpret_cast<const __half2*>(&bias));
    lo = *reinterpret_cast<const uint32_t*>(&u);
    hi = *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void codes_to_half(uint32_t x, uint32_t& lo, uint32_t& hi)
{
    biased_to_half(x ^ 0x80808080u, lo, hi);
}

// Cache codes are read once: a load that does not keep them in L1.
__device__ __forceinline__ uint4 ldg_stream(const uint4* p)
{
    uint4 x;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
    return x;
}
__device__ __forceinline__ uint2 ldg_stream(const uint2* p)
{
    uint2 x;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
    return x;
}

// Zeros for n tokens from `start`, heads h0 .. h0 + heads.
template <typename T, int D>
__device__ void zero_rows(const AttendArgs& a, int start, int n, int h0, int heads)
{
    for (int64_t i = threadIdx.x; i < int64_t(n) * heads * D; i += blockDim.x) {
        const int64_t v = i / D;
        static_cast<T*>(a.out)[(start + v / heads) * a.out_token + (h0 + v % heads) * a.out_head + i % D] = from_float<T>(0.f);
    }
}

// kv_attend.cu: the join of partial results in the workspace, [T][q_heads][splits][D] sums and then
// [T][q_heads][splits] {maximum, sum of weights}; kv_prefill.cu: many query tokens per row.
// per_row: columns per row and cache head to join, or 0: every token's.
cudaError_t launch_kv_join(const AttendArgs& a, int splits, int stretch, int per_row, cudaStream_t s);
int64_t kv_prefill_workspace(const st_kv_cache& c, int64_t T, int32_t q_heads, int32_t R, int32_t max_q, int64_t max_len);
cudaError_t launch_kv_prefill(const AttendArgs& a, cudaStream_t s);

}  // namespace st
