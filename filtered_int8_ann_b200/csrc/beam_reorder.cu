// Take the states of the chosen beams: dst[b][j] = src[b][parents[b][j]] for
// up to 16 arrays in one launch.
//
// A copy: bound by the bytes read and written. Each CTA copies a piece of one
// row of one array, in the widest words that the array's addresses allow (16
// bytes as a rule), four loads in flight per thread. 16 x 8 beams' states in 4 arrays of 512 KB a row
// (537 MB in and out): 73 us, 7.4 TB/s of them, above a plain copy's rate because rows taken more than once come from
// L2. Small states are one launch: 2.8 us.
#include "decode.cuh"

namespace st {

constexpr int kReorderBlock = 256;
constexpr int kReorderUnroll = 4;

struct ReorderArgs {
    st_beam_state s[ST_BEAM_MAX_STATES];
    int64_t first[ST_BEAM_MAX_STATES + 1];  // first CTA of each array
    int32_t pieces[ST_BEAM_MAX_STATES];     // CTAs per row
    int32_t width[ST_BEAM_MAX_STATES];      // bytes per word: 16, 8, 4, 2 or 1
    int32_t n;
    const int32_t* parents;
    int32_t B, K, keep;
    uint32_t* err;
};

template <typename W>
__device__ __forceinline__ void copy_piece(const char* src, char* dst, int64_t bytes, int64_t lo, int64_t hi)
{
    const W* a = reinterpret_cast<const W*>(src);
    W* b = reinterpret_cast<W*>(dst);
    const int64_t end = min(hi, bytes / int64_t(sizeof(W)));
    for (int64_t i0 = lo + threadIdx.x; i0 < end; i0 += kReorderBlock * kReorderUnroll) {
        W x[kReorderUnroll];
#pragma unroll
        for (int u = 0; u < kReorderUnroll; ++u) {
            x[u] = W{};
            if (src && i0 + u * kReorderBlock < end) x[u] = a[i0 + u * kReorderBlock];
        }
#pragma unroll
        for (int u = 0; u < kReorderUnroll; ++u)
            if (i0 + u * kReorderBlock < end) b[i0 + u * kReorderBlock] = x[u];
    }
}

__global__ void __launch_bounds__(kReorderBlock) beam_reorder_kernel(const __grid_constant__ ReorderArgs a)
{
    const int64_t cta = blockIdx.x;
    int k = 0;
    while (k + 1 < a.n && cta >= a.first[k + 1]) ++k;
    const st_beam_state& s = a.s[k];
    const int64_t i = (cta - a.first[k]) / a.pieces[k];
    const int piece = int((cta - a.first[k]) - i * a.pieces[k]);
    const int64_t rows = int64_t(a.B) * a.keep;
    const int64_t outer = i / rows, row = i - outer * rows;
    const int b = int(row / a.keep);
    const int p = a.parents[row];
    const bool real = p >= 0 && p < a.K;
    if (!real && p != -1 && threadIdx.x == 0) atomicOr(a.err, kDecErrParent);
    const char* src = real ? static_cast<const char*>(s.src) + outer * s.src_outer_stride +
                                 (int64_t(b) * a.K + p) * s.src_row_stride
                           : nullptr;
    char* dst = static_cast<char*>(s.dst) + outer * s.dst_outer_stride + row * s.dst_row_stride;
    const int w = a.width[k];
    const int64_t words = (s.row_bytes / w + a.pieces[k] - 1) / a.pieces[k], lo = piece * words, hi = lo + words;
    switch (w) {
        case 16: copy_piece<uint4>(src, dst, s.row_bytes, lo, hi); break;
        case 8: copy_piece<uint2>(src, dst, s.row_bytes, lo, hi); break;
        case 4: copy_piece<uint32_t>(src, dst, s.row_bytes, lo, hi); break;
        case 2: copy_piece<uint16_t>(src, dst, s.row_bytes, lo, hi); break;
        default: copy_piece<uint8_t>(src, dst, s.row_bytes, lo, hi); break;
    }
}

cudaError_t launch_beam_reorder(const st_beam_state* states, int32_t n_states, const int32_t* parents, int32_t B,
                                int32_t K, int32_t keep, uint32_t* err, cudaStream_t s)
{
    ReorderArgs a = {};
    a.parents = parents;
    a.B = B;
    a.K = K;
    a.keep = keep;
    a.err = err;
    for (int i = 0; i < n_states; ++i) {
        const st_beam_state& x = states[i];
        if (x.row_bytes == 0 || x.outer == 0) continue;
        const int k = a.n++;
        a.s[k] = x;
        const uint64_t all = reinterpret_cast<uintptr_t>(x.src) | reinterpret_cast<uintptr_t>(x.dst) |
                             uint64_t(x.row_bytes) | uint64_t(x.src_row_stride) | uint64_t(x.dst_row_stride) |
                             (x.outer > 1 ? uint64_t(x.src_outer_stride) | uint64_t(x.dst_outer_stride) : 0);
        int w = 16;
        while (all % w) w >>= 1;
        a.width[k] = w;
        const int64_t per_cta = int64_t(kReorderBlock) * kReorderUnroll * 4;  // words
        const int64_t pieces = (x.row_bytes / w + per_cta - 1) / per_cta;
        const int64_t ctas = pieces * x.outer * B * keep;
        if (pieces > 0x7fffffff || a.first[k] + ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
        a.pieces[k] = int32_t(pieces);
        a.first[k + 1] = a.first[k] + ctas;
    }
    if (a.n == 0) return cudaSuccess;
    beam_reorder_kernel<<<unsigned(a.first[a.n]), kReorderBlock, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace st
