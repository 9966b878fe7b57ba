// Attention of many query tokens per row over an int8 paged cache (prompts, and
// steps of several tokens) on the 5th-generation tensor cores.
//
// Bound by the products: 4 D flops per (query, head, cached token). A CTA
// takes 256 columns (query token, head) of one cache head, as two tiles of
// 128, and a stretch of the cache, 128 tokens at a time; stretches (long rows, or few columns) are
// joined by the decode kernel's second launch. Roles:
//   * warps 0-3 and 4-7: the softmax of tile 0 and 1, a column per thread, so
//     that maxima and sums need no exchange. Scores come from TMEM; weights go
//     back over them as fp16, the A operand of the second product;
//   * warps 8-11 (K) and 12-15 (V): bring the next tokens' codes into registers,
//     and convert them to fp16 operands in shared memory (128-byte swizzle): K as
//     [token][dim], V transposed as [dim][token] by byte permutes, so both
//     products read K-major operands;
//   * warp 16: issues tcgen05.mma (M = 128, N = 128 tokens or D dims, K = 16, fp32 sums in TMEM). While
//     one tile's products run, the other tile's softmax does: S and its weights
//     share TMEM columns, 2 x 128 for them and 2 x 128 for O fill all 512.
// Codes are exact in fp16; a block's K scale multiplies its scores, and its V scale (over the
// largest of the stretch) the weights, both in fp32. A weight is p = 2^(s - M) with M
// raised only when a score exceeds it by 8 (then O is rescaled in TMEM): p
// is at most 2^8, and 2^7 times it and its V factor fits into fp16 and is held with 11 bits down to 2^-21.
//
// Prompts of 1793 queries over 8192 tokens and of 722 over 6144, 8 cache heads of 128 and 4 query heads each (0.28 TFLOP):
// 469 us, 0.60 PFLOP/s, two rows of one query in the same call and the join of their stretches included; 4 prompts of 2048 over
// 8192 each (0.96 TFLOP) 1283 us, 0.75. A pair of tiles takes 4500 to 5600 cycles per 128 tokens, of which the products are 2570: a tile's S, its
// softmax and its P V follow each other, and two tiles hide only a part of it (without any arithmetic in the softmax
// and the conversions 335 us). Every pair converts its row's K and V anew. The pairs that see most come first, yet the last
// ones leave a fifth of the SMs' time unused; splitting them along the cache cost more (608 us) than it filled.
//
// Up to 128 columns stand in both tiles, which take the steps in turn, instead of leaving one tile empty: 32 rows of
// 8192 tokens with 64 columns 298 us, 431 otherwise.
//
// Waits are bounded: one that runs out sets the error word and an abort flag, the
// roles leave their loops, and the CTA frees its TMEM after a last bounded wait
// for the products in flight.
#include "attend.cuh"
#include "tc_ptx.cuh"

namespace st {

constexpr int kPreTile = 128;                  // tokens per step
constexpr int kPreCols = 256;                  // columns per CTA: two tiles
constexpr int kPreLoaders = 128;               // threads that bring K, and as many for V
constexpr int kPreMmaWarp = 16;
constexpr int kPreBlock = 32 * (kPreMmaWarp + 4);  // whole warpgroups; the last three warps idle
// Registers per thread after the split of the launch's 96: 2 x 128 + 2 x 72 + 80 = 5 x 96.
constexpr int kPreSoftmaxRegs = 128, kPreLoaderRegs = 72, kPreMmaRegs = 80;
constexpr int kPreMaxStretch = 16384;          // tokens: the table of a stretch is held in shared memory
constexpr int kPreMaxBlocks = kPreMaxStretch / 16;
constexpr int kPreStages = 2;  // of K and V operands
constexpr uint32_t kPreWaitLimit = 1u << 22;
constexpr float kPreRaise = 8.f;  // a score this far above the reference raises it
constexpr float kPreUp = 0x1p7f;  // of the weights in fp16

template <int D>
struct PreShared {
    alignas(1024) uint8_t q[2][D / 64][kPreTile * 128];           // two tiles, halves of 64 dims, 128 rows of 128 bytes
    alignas(1024) uint8_t k[kPreStages][D / 64][kPreTile * 128];  // 128 tokens
    alignas(1024) uint8_t v[kPreStages][2][D * 128];              // halves of 64 tokens, D rows of 128 bytes
    // of each 16 tokens of the stretch: where their codes begin (-1: hidden), their block's scales (K: negative
    // when hidden; V: over the largest of the stretch)
    int64_t at[kPreMaxBlocks];
    alignas(16) float ks[kPreMaxBlocks];
    alignas(16) float vs[kPreMaxBlocks];
    float vtop[kPreBlock / 32];
    alignas(8) uint64_t k_full[kPreStages], k_empty[kPreStages], v_full[kPreStages], v_empty[kPreStages];
    uint64_t s_full[2], p_ready[2], pv_done[2];
    uint64_t drain;
    float2 joined[kPreTile];  // taking turns: the second tile's maxima and sums (its O goes over the K operands)
    uint32_t tmem;
    int32_t abort;
};

// D[tmem] (+)= A[smem] x B[smem]^T and A[tmem] x B[smem]^T, fp16 with fp32 sums, issued by one thread.
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::f16: fp32 sums (bits 4-5 = 1), fp16 A and B (0), both K-major, N >> 3
// (bits 17-22), M >> 4 (bits 24-28).
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N)
{
    return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

// 32 consecutive TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32])
{
    uint32_t* x = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]),
          "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]),
          "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]),
          "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&r)[32])
{
    const uint32_t* x = reinterpret_cast<const uint32_t*>(r);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
        ::"r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]),
          "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]), "r"(x[16]), "r"(x[17]), "r"(x[18]),
          "r"(x[19]), "r"(x[20]), "r"(x[21]), "r"(x[22]), "r"(x[23]), "r"(x[24]), "r"(x[25]), "r"(x[26]), "r"(x[27]),
          "r"(x[28]), "r"(x[29]), "r"(x[30]), "r"(x[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&x)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        ::"r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]),
          "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t&>(d)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t&>(d)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}

// Eight columns, as tmem_ld32 and tmem_st32.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&x)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&x)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                 ::"r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(taddr)
                 : "memory");
}

// Wait for this warp's TMEM loads; the registers they fill depend on it.
__device__ __forceinline__ void tmem_wait16(float2 (&s)[8])
{
    uint32_t* x = reinterpret_cast<uint32_t*>(s);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                   "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15])
                 :: "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t taddr, float2 (&s)[8])
{
    tmem_ld16(taddr, reinterpret_cast<uint32_t(&)[16]>(s));
}

// The largest score among the 128 tokens of a step, over the factor sc of their sixteens.
__device__ __forceinline__ float step_max(uint32_t ts, const float (&sc)[8])
{
    float top = -INFINITY;
    float2 s[2][8];
    tmem_load16(ts, s[0]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        float2(&x)[8] = s[c & 1];
        tmem_wait16(x);
        if (c < 7) tmem_load16(ts + 16 * (c + 1), s[(c + 1) & 1]);
        float a = fmaxf(x[0].x, x[0].y), b = fmaxf(x[1].x, x[1].y);
#pragma unroll
        for (int i = 2; i < 8; i += 2) {
            a = fmaxf(fmaxf(a, x[i].x), x[i].y);
            b = fmaxf(fmaxf(b, x[i + 1].x), x[i + 1].y);
        }
        top = fmaxf(top, fmaxf(a, b) * sc[c]);
    }
    return top;
}

// The step's weights 2^(score - base), times their sixteens' V factors, as fp16 over the scores; returns their sum
// before those factors. Straight-line code: the exponentials bound it.
__device__ __forceinline__ float step_weights(uint32_t ts, const float (&sc)[8], const float (&vf)[8], float base)
{
    float2 total[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const float2 down = make_float2(-base, -base);
    float2 s[2][8];
    tmem_load16(ts, s[0]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        float2(&x)[8] = s[c & 1];
        tmem_wait16(x);
        if (c < 7) tmem_load16(ts + 16 * (c + 1), s[(c + 1) & 1]);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float2 y = fma2(x[i], make_float2(sc[c], sc[c]), down);
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            total[i & 1] = add2(total[i & 1], y);
            y = mul2(y, make_float2(vf[c], vf[c]));
            w[i] = pack_half2(y.x, y.y);
        }
        tmem_st8(ts + 8 * c, w);  // over scores that have been read
    }
    total[0] = add2(total[0], total[1]);
    return total[0].x + total[0].y;
}

// Both for a step of which the column sees `see` tokens, without the hidden blocks' (negative factors), and for scores
// that are rounded first.
__device__ __noinline__ float step_max_masked(uint32_t ts, const float* ks, float mult, int see)
{
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        float2 s[8];
        tmem_load16(ts + 16 * c, s);
        tmem_wait16(s);
        const int here = ks[c] >= 0.f ? see - 16 * c : 0;
        const float sc = ks[c] * mult;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (2 * i < here) top = fmaxf(top, s[i].x * sc);
            if (2 * i + 1 < here) top = fmaxf(top, s[i].y * sc);
        }
    }
    return top;
}
__device__ __noinline__ float step_weights_masked(uint32_t ts, const float* ks, const float* vs, float mult, float base, int see, bool far)
{
    // (far: some column's maximum is)
    const auto weight = [&](float s, float sc) { return ex2(far ? __fsub_rn(__fmul_rn(s, sc), base) : fmaf(s, sc, -base)); };
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        float2 s[8];
        tmem_load16(ts + 16 * c, s);
        tmem_wait16(s);
        const int here = ks[c] >= 0.f ? see - 16 * c : 0;
        const float sc = ks[c] * mult, vf = vs[c];
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = 2 * i < here ? weight(s[i].x, sc) : 0.f;
            const float y = 2 * i + 1 < here ? weight(s[i].y, sc) : 0.f;
            sum += x + y;
            w[i] = pack_half2(x * vf, y * vf);
        }
        tmem_st8(ts + 8 * c, w);
    }
    return sum;
}

// Raise the column's reference m to `top` (at least m): what has been summed with it, l and O, shrinks.
template <int D>
__device__ __noinline__ void raise(uint32_t to, float top, bool has_o, float& m, float& l)
{
    const float z = top > m ? ex2(m - top) : 1.f;
    m = top;
    l *= z;
    if (has_o) {
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(to + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * z);
            tmem_st16(to + 16 * c, o);
        }
        tmem_wait_st();
    }
}

// mbar_wait that also ends, without success, when another role has set the abort flag.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, const volatile int32_t* abort)
{
    for (uint32_t i = 0; i < kPreWaitLimit / 256; ++i) {
        if (mbar_wait(bar, parity, 256)) return true;
        if (*abort) return false;
    }
    return false;
}

// True in one lane of the (whole) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t lead;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(lead));
    return lead != 0;
}

template <int REGS>
__device__ __forceinline__ void regs_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

template <typename T, int D>
__global__ void __launch_bounds__(kPreBlock, 1)
kv_prefill_kernel(AttendArgs a, int splits, int stretch)
{
    extern __shared__ unsigned char raw[];
    PreShared<D>& sh = *reinterpret_cast<PreShared<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hk = blockIdx.y;
    const int unit = blockIdx.x / splits, split = blockIdx.x - unit * splits;
    const int G = a.q_heads / a.c.kv_heads, S = a.c.block_size, shift = 31 - __clz(S);

    // Units: row r's pairs of tiles are numbered from floor(row_start[r] G / 256) + r on, which leaves room for all of
    // them whatever the rows' lengths. This unit's row is the last that begins at or before it.
    auto begin_of = [&](int r) { return int(int64_t(min(max(a.row_start[r], 0), int(a.T))) * G / kPreCols) + r; };
    int lo = 0, hi = a.R - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (begin_of(mid) <= unit) lo = mid;
        else hi = mid - 1;
    }
    const int row = lo, nth = unit - begin_of(row);
    const int start = min(max(a.row_start[row], 0), int(a.T)), n = min(max(a.row_start[row + 1], start), int(a.T)) - start;
    const int64_t all_cols = int64_t(n) * G;
    const int row_pairs = int((all_cols + kPreCols - 1) / kPreCols), pair = row_pairs - 1 - nth;  // those that see most first
    if (nth < 0 || pair < 0 || all_cols <= a.above_cols) return;
    int64_t len = max(a.lens[row], 0);
    if (len > a.max_len || n > a.max_q) {
        if (split == 0 && hk == 0 && pair == 0 && tid == 0) atomicOr(a.err, kDecErrRow);
        len = 0;
    }
    const int64_t col0 = int64_t(pair) * kPreCols;
    const int cols = int(min(int64_t(kPreCols), all_cols - col0));
    const int64_t j0 = int64_t(split) * stretch;
    if (j0 >= len && split > 0) return;
    // the stretch's tokens that the last column sees
    int64_t end = len;
    if (a.causal) end = min(end, len - n + (col0 + cols - 1) / G + 1);
    const int tokens = int(max(int64_t(0), min(int64_t(stretch), end - j0)));
    const int steps = (tokens + kPreTile - 1) / kPreTile;
    // Up to 128 columns stand in both tiles, which take the steps in turn; their sums are joined at the end.
    const bool turns = cols <= kPreTile;

    if (warp == kPreMmaWarp) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
        if (lane == 0) {
            for (int i = 0; i < kPreStages; ++i) {
                mbar_init(&sh.k_full[i], kPreLoaders / 32);
                mbar_init(&sh.v_full[i], kPreLoaders / 32);
                mbar_init(&sh.k_empty[i], 1);
                mbar_init(&sh.v_empty[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh.s_full[i], 1);
                mbar_init(&sh.p_ready[i], 4);
                mbar_init(&sh.pv_done[i], 1);
            }
            mbar_init(&sh.drain, 1);
            sh.abort = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    // the stretch's tokens, in sixteens up to the end of the last step
    float vlocal = 0.f;
    {
        const int32_t* table = a.table + int64_t(row) * a.max_blocks + (j0 >> shift);
        for (int i = tid; i < steps * (kPreTile / 16); i += kPreBlock) {
            int p = -1;
            if (16 * i < tokens) {
                p = table[(16 * i) >> shift];
                if (p < 0 || p >= a.c.num_blocks) {
                    atomicOr(a.err, kDecErrTable);
                    p = -1;
                }
            }
            const int64_t block = int64_t(p) * a.c.kv_heads + hk;
            sh.at[i] = p < 0 ? -1 : (block * S + ((16 * i) & (S - 1))) * D;
            sh.ks[i] = p < 0 ? -1.f : a.c.k_scale[block];
            const float vs = p < 0 ? 0.f : a.c.v_scale[block];
            sh.vs[i] = vs;
            vlocal = fmaxf(vlocal, vs);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) vlocal = fmaxf(vlocal, __shfl_xor_sync(0xffffffffu, vlocal, off));
        if (lane == 0) sh.vtop[warp] = vlocal;
    }
    // the queries, a column per softmax thread
    const int tile = warp >> 2, r = tid & 127;  // warps 0-7
    const int64_t col = col0 + (turns ? 0 : tile * kPreTile) + r;
    const bool mine = warp < 8 && col < col0 + cols;
    float mult = 0.f;
    int64_t token = 0, head = 0;
    if (warp < 8) {
        uint4 w[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] = make_uint4(0, 0, 0, 0);
        if (mine) {
            token = start + col / G;
            head = hk * G + col % G;
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + token * a.q_token + head * a.q_head);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) w[i] = p[i];
        }
        float big = 0.f;
        bool finite = true;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            float x[8];
            unpack8<T>(w[i], x);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                big = fmaxf(big, fabsf(x[u]));
                finite = finite && fabsf(x[u]) < INFINITY;
            }
        }
        // a negative scale's sign goes to the query: block scores are then multiplied by positive numbers
        const float down = finite ? copysignf(pow2_down(big), a.scale_log2) : 0.f;
        mult = finite ? fabsf(a.scale_log2) * pow2_up(big) : NAN;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            float x[8];
            unpack8<T>(w[i], x);
            uint4 y = make_uint4(0, 0, 0, 0);
            if (finite) {
                y.x = pack_half2(x[0] * down, x[1] * down);
                y.y = pack_half2(x[2] * down, x[3] * down);
                y.z = pack_half2(x[4] * down, x[5] * down);
                y.w = pack_half2(x[6] * down, x[7] * down);
            }
            *reinterpret_cast<uint4*>(&sh.q[tile][i / 8][r * 128 + (((i & 7) ^ (r & 7)) << 4)]) = y;
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    float vtop = 0.f;
#pragma unroll
    for (int w = 0; w < kPreBlock / 32; ++w) vtop = fmaxf(vtop, sh.vtop[w]);
    {
        for (int i = tid; i < steps * (kPreTile / 16); i += kPreBlock) sh.vs[i] = vtop > 0.f ? __fdiv_rn(sh.vs[i], vtop) * kPreUp : 0.f;
    }
    __syncthreads();
    volatile int32_t* abort = &sh.abort;
    auto give_up = [&]() {
        *abort = 1;
        atomicOr(a.err, kDecErrWait);
    };

    float m = -INFINITY, l = 0.f;  // softmax threads
    if (warp >= kPreMmaWarp) {
        // ------------------------------------------------------------ products --
        regs_down<kPreMmaRegs>();
        if (warp == kPreMmaWarp && steps > 0) {
            // The whole warp walks the steps, so that addresses stay in uniform registers; one lane issues.
            constexpr uint32_t idS = idesc_f16(128, kPreTile), idO = idesc_f16(128, D);
            constexpr uint64_t kQHalf = sizeof(sh.q[0][0]) >> 4, kVHalf = sizeof(sh.v[0][0]) >> 4;
            const uint64_t dq = smem_desc_kmajor(smem_u32(sh.q), 128), dk = smem_desc_kmajor(smem_u32(sh.k), 128),
                           dv = smem_desc_kmajor(smem_u32(sh.v), 128);
            const bool lead = elect_one();
            auto scores = [&](int x, int j) {  // S of tile x, step j
                if (lead) {
                    const uint64_t q = dq + x * (sizeof(sh.q[0]) >> 4), k = dk + (j & 1) * (sizeof(sh.k[0]) >> 4);
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        tc_mma_f16(tmem + x * 128, q + s / 4 * kQHalf + (s & 3) * 2, k + s / 4 * kQHalf + (s & 3) * 2, idS, s > 0);
                    tc_commit(&sh.s_full[x]);
                }
            };
            auto values = [&](int x, int j, bool first) {  // O += P V
                if (lead) {
                    const uint64_t v = dv + (j & 1) * (sizeof(sh.v[0]) >> 4);
#pragma unroll
                    for (int s = 0; s < kPreTile / 16; ++s)
                        tc_mma_f16_ts(tmem + 256 + x * 128, tmem + x * 128 + s * 8, v + s / 4 * kVHalf + (s & 3) * 2, idO, !first || s > 0);
                    tc_commit(&sh.pv_done[x]);
                }
            };
            auto done = [&](uint64_t* bar) {
                if (lead) tc_commit(bar);
            };
            bool ok = wait_or_abort(&sh.k_full[0], 0, abort);
            if (turns) {
#pragma unroll 1
                for (int j = 0; j < 2 && j < steps && ok; ++j) {
                    ok = wait_or_abort(&sh.k_full[j], 0, abort);
                    if (!ok) break;
                    tc_fence_after();
                    scores(j, j);
                    done(&sh.k_empty[j]);
                }
#pragma unroll 1
                for (int j = 0; j < steps && ok; ++j) {
                    const int st = j & 1;
                    ok = wait_or_abort(&sh.v_full[st], j >> 1 & 1, abort) && wait_or_abort(&sh.p_ready[st], j >> 1 & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    values(st, j, j < 2);
                    done(&sh.v_empty[st]);
                    if (j + 2 < steps) {
                        ok = wait_or_abort(&sh.k_full[st], (j + 2) >> 1 & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                        scores(st, j + 2);
                        done(&sh.k_empty[st]);
                    }
                }
            } else {
                if (ok) {
                    tc_fence_after();
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) scores(x, 0);
                    done(&sh.k_empty[0]);
                }
#pragma unroll 1
                for (int j = 0; j < steps && ok; ++j) {
                    const int st = j & 1, nx = st ^ 1;
                    ok = wait_or_abort(&sh.v_full[st], j >> 1 & 1, abort);
                    if (ok && j + 1 < steps) ok = wait_or_abort(&sh.k_full[nx], (j + 1) >> 1 & 1, abort);
#pragma unroll 1
                    for (int x = 0; x < 2 && ok; ++x) {
                        ok = wait_or_abort(&sh.p_ready[x], j & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                        values(x, j, j == 0);
                        if (j + 1 < steps) scores(x, j + 1);
                    }
                    if (ok) {
                        done(&sh.v_empty[st]);
                        if (j + 1 < steps) done(&sh.k_empty[nx]);
                    }
                }
            }
            if (!__all_sync(0xffffffffu, ok)) give_up();
            __syncwarp();
            done(&sh.drain);  // all products issued are done before the TMEM is freed
            if (!mbar_wait(&sh.drain, 0, kPreWaitLimit)) give_up();
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------------ V --
        regs_down<kPreLoaderRegs>();
        constexpr int VN = D / 32;  // turns of 32 dims each, for the warp's 32 tokens
        uint32_t vr[VN][8];
        // lane bits 0, 3, 4: a word of the turn's 32 dims; bits 1, 2: a group of 8 of the warp's 32 tokens
        const int vword = (lane & 1) | (lane >> 3 & 3) << 1, vrow = (warp - 12) * 32 + (lane >> 1 & 3) * 8;
        const int8_t* const from = a.c.v + (vrow & 8) * D + vword * 4;
        auto load = [&](int j) {
            const int64_t at = sh.at[j * 8 + vrow / 16];
            const bool on = at >= 0;
            const int8_t* x = from + (on ? at : 0);
#pragma unroll
            for (int i = 0; i < VN; ++i)
#pragma unroll
                for (int u = 0; u < 8; ++u) vr[i][u] = __ldg(reinterpret_cast<const uint32_t*>(x + u * D + i * 32));
            if (!on) {
#pragma unroll
                for (int i = 0; i < VN; ++i)
#pragma unroll
                    for (int u = 0; u < 8; ++u) vr[i][u] = 0u;
            }
        };
        // piece of 8 tokens vrow / 8 % 8 of half vrow / 64; rows 4 vword .. of the turn, whose low bits are u and vword's
        uint8_t* const vto = sh.v[0][vrow / 64] + vword * 4 * 128;
        const int vc = (vrow / 8 & 7) ^ (vword & 1) << 2;
        bool ok = true;
        if (steps > 0) load(0);
        for (int j = 0; j < steps; ++j) {
            ok = wait_or_abort(&sh.v_empty[j & 1], (j >> 1 & 1) ^ 1, abort);
            if (!ok) break;
            uint8_t* to = vto + (j & 1) * int(sizeof(sh.v[0]));
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                uint32_t out[4][4];  // [dim][pairs of tokens]
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t x = vr[i][2 * u] ^ 0x80808080u, y = vr[i][2 * u + 1] ^ 0x80808080u;
                    biased_to_half(__byte_perm(x, y, 0x5140), out[0][u], out[1][u]);
                    biased_to_half(__byte_perm(x, y, 0x7362), out[2][u], out[3][u]);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    *reinterpret_cast<uint4*>(to + (i * 32 + u) * 128 + ((vc ^ u) << 4)) =
                        make_uint4(out[u][0], out[u][1], out[u][2], out[u][3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.v_full[j & 1]);
            if (j + 1 < steps) load(j + 1);  // (behind the fence, which would wait for these loads)
        }
        if (!ok) give_up();
    } else if (warp >= 8) {
        // ------------------------------------------------------------------ K --
        regs_down<kPreLoaderRegs>();
        constexpr int ROWP = D / 16;                 // 16-byte pieces of a row
        constexpr int ROWS = kPreLoaders / ROWP;     // rows per turn: 16 (D = 128) or 32
        constexpr int KN = kPreTile / ROWS;          // turns
        uint4 kr[KN];
        const int p = tid - 256, piece = p % ROWP, krow = p / ROWP;
        const int8_t* const from = a.c.k + (krow & 15) * D + piece * 16;
        auto load = [&](int j) {
#pragma unroll
            for (int i = 0; i < KN; ++i) {
                const int64_t at = sh.at[j * 8 + (krow + i * ROWS) / 16];
                kr[i] = ldg_stream(reinterpret_cast<const uint4*>(from + (at >= 0 ? at : 0)));
                if (at < 0) kr[i] = make_uint4(0, 0, 0, 0);
            }
        };
        // dims 16 piece .. are pieces 2 (piece % 4) and the next of half piece / 4; the second half's lanes store them
        // in the other order, so that eight lanes fill eight different pieces
        const int swap = piece >> 2 & 1, kc = (piece & 3) * 2;
        uint8_t* const kto = sh.k[0][piece / 4] + krow * 128;
        const int k0 = ((kc + swap) ^ (krow & 7)) << 4, k1 = ((kc + (swap ^ 1)) ^ (krow & 7)) << 4;
        bool ok = true;
        if (steps > 0) load(0);
        for (int j = 0; j < steps; ++j) {
            ok = wait_or_abort(&sh.k_empty[j & 1], (j >> 1 & 1) ^ 1, abort);
            if (!ok) break;
            uint8_t* to = kto + (j & 1) * int(sizeof(sh.k[0]));
#pragma unroll
            for (int i = 0; i < KN; ++i) {
                uint4 lo, hi;
                codes_to_half(kr[i].x, lo.x, lo.y);
                codes_to_half(kr[i].y, lo.z, lo.w);
                codes_to_half(kr[i].z, hi.x, hi.y);
                codes_to_half(kr[i].w, hi.z, hi.w);
                *reinterpret_cast<uint4*>(to + i * ROWS * 128 + k0) = swap ? hi : lo;
                *reinterpret_cast<uint4*>(to + i * ROWS * 128 + k1) = swap ? lo : hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.k_full[j & 1]);
            if (j + 1 < steps) load(j + 1);  // (behind the fence, which would wait for these loads)
        }
        if (!ok) give_up();
    } else {
        // ------------------------------------------------------------- softmax --
        regs_up<kPreSoftmaxRegs>();
        const uint32_t lanes = uint32_t(warp & 3) << 21;  // TMEM lane 32 (warp % 4) in bits 16 on
        const uint32_t ts = tmem + lanes + tile * 128, to = tmem + lanes + 256 + tile * 128;
        int see = tokens;  // tokens of the stretch that this column sees
        if (mine && a.causal) see = int(max(int64_t(0), min(int64_t(tokens), len - n + col / G + 1 - j0)));
        const int least = __reduce_min_sync(0xffffffffu, see);
        bool ok = true, far = false;  // far: some column's maximum is
        int i = 0;  // steps of this tile
        for (int j = turns ? tile : 0; j < steps && ok; j += turns ? 2 : 1, ++i) {
            const int left = see - j * kPreTile;
            const float *ks = sh.ks + j * 8, *vs = sh.vs + j * 8;
            float sc[8], vf[8];  // before the wait: shared memory is slow while products read it
#pragma unroll
            for (int b = 0; b < 8; b += 4) {
                const float4 x = *reinterpret_cast<const float4*>(ks + b), y = *reinterpret_cast<const float4*>(vs + b);
                sc[b] = x.x, sc[b + 1] = x.y, sc[b + 2] = x.z, sc[b + 3] = x.w;
                vf[b] = y.x, vf[b + 1] = y.y, vf[b + 2] = y.z, vf[b + 3] = y.w;
            }
            bool whole = (j + 1) * kPreTile <= least;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                whole = whole && sc[b] >= 0.f;
                sc[b] *= mult;
            }
            ok = wait_or_abort(&sh.s_full[tile], i & 1, abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();  // the products of the tile's step before are done too
            const float top = just_above(whole ? step_max(ts, sc) : step_max_masked(ts, ks, mult, left));
            if (m == -INFINITY) m = top;  // nothing seen before: l and O are 0
            if (__any_sync(0xffffffffu, top > m + kPreRaise)) raise<D>(to, top > m + kPreRaise ? top : m, i > 0, m, l);
            far = __any_sync(0xffffffffu, is_far(m));
            const float base = m > -INFINITY ? m : 0.f;
            l += whole && !far ? step_weights(ts, sc, vf, base) : step_weights_masked(ts, ks, vs, mult, base, left, far);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_ready[tile]);
        }
        if (ok && i > 0) ok = wait_or_abort(&sh.pv_done[tile], (i - 1) & 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) give_up();
        tc_fence_after();
        float z0 = 1.f, z1 = 0.f;  // weights of this tile's sums and the other's
        float* const other = reinterpret_cast<float*>(sh.k);  // [dim][column]
        if (turns) {
            if (tile == 1) {
                // Every score product is done when one of the last two steps' value products is, so the K operands'
                // memory is free by now (or, without a step, left alone: nothing was seen then).
                sh.joined[r] = make_float2(m, l);
                if (ok && i > 0) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tmem_ld32(to + 32 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int d = 0; d < 32; ++d) other[(32 * c + d) * kPreTile + r] = o[d];
                    }
                }
            }
            named_barrier(1, 256);
            if (tile == 0) {
                const float2 y = sh.joined[r];
                const float top = fmaxf(m, y.x);
                z0 = m > -INFINITY ? ex2(m - top) : 0.f;
                z1 = y.x > -INFINITY ? ex2(y.x - top) : 0.f;
                l = l * z0 + y.y * z1;
                m = top;
            }
        }
        if (ok && !*abort && (tile == 0 || !turns)) {
            const bool direct = splits == 1 || n > a.max_q;  // (the join leaves out rows that are too long)
            const float scale = direct ? (l == 0.f ? 0.f : 1.f / (kPreUp * l)) : 1.f / kPreUp;  // vtop may be next to nothing
            T* out = static_cast<T*>(a.out) + token * a.out_token + head * a.out_head;
            const int64_t part = (token * a.q_heads + head) * splits + split;
            float* po = static_cast<float*>(a.workspace);
            if (mine && !direct) {
                float* pm = po + a.parts * splits * D;
                pm[2 * part] = m;
                pm[2 * part + 1] = l;
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                if (steps > 0) {
                    tmem_ld32(to + 32 * c, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int d = 0; d < 32; ++d) o[d] = 0.f;
                }
                if (turns) {
#pragma unroll
                    for (int d = 0; d < 32; ++d) {
                        o[d] *= z0;
                        if (z1 > 0.f) o[d] = fmaf(other[(32 * c + d) * kPreTile + r], z1, o[d]);
                    }
                }
                if (!mine) {
                    // the loads above are the whole warp's
                } else if (direct) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        T y[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) y[u] = from_float<T>(l == 0.f ? 0.f : o[8 * k + u] * scale * vtop);
                        *reinterpret_cast<uint4*>(out + 32 * c + 8 * k) = *reinterpret_cast<const uint4*>(y);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<float4*>(po + part * D + 32 * c + 4 * k) =
                            make_float4(o[4 * k] * scale * vtop, o[4 * k + 1] * scale * vtop, o[4 * k + 2] * scale * vtop,
                                        o[4 * k + 3] * scale * vtop);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kPreMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

struct PrePlan {
    int splits, stretch;
    int64_t units;
};

// Stretches: one while the columns alone fill the GPU (a join would only add to the work), else enough for two CTAs
// per SM, none longer than the table that fits, of at least 1024 tokens. Every row counts as work here, short ones that the
// decode kernel takes too: few prompt columns beside many such rows get fewer stretches than they would alone (a prompt of 64
// tokens over 16384, 4 query heads each, 53 us; beside 63 rows of one token, which alone take 370, both take 898).
static PrePlan pre_plan(const st_kv_cache& c, int64_t T, int32_t q_heads, int32_t R, int64_t max_len)
{
    PrePlan p;
    p.units = T * (q_heads / c.kv_heads) / kPreCols + R;
    const int64_t units = p.units * c.kv_heads, wanted = 2 * 148;
    int64_t stretch = max_len;
    if (units < wanted) {
        const int64_t each = (wanted + units - 1) / units;
        stretch = (max_len + each - 1) / each;
        if (stretch < 1024) stretch = 1024;
    }
    if (stretch > kPreMaxStretch) stretch = kPreMaxStretch;
    stretch = (stretch + kPreTile - 1) / kPreTile * kPreTile;
    p.splits = int((max_len + stretch - 1) / stretch);
    p.stretch = int(stretch);
    return p;
}

int64_t kv_prefill_workspace(const st_kv_cache& c, int64_t T, int32_t q_heads, int32_t R, int32_t, int64_t max_len)
{
    const PrePlan p = pre_plan(c, T, q_heads, R, max_len);
    if (p.splits == 1) return 0;
    // T q_heads is below 2^47, its multiples need not be within 64 bits
    const int64_t parts = T * q_heads, each = p.splits * (int64_t(c.head_dim) + 2) * 4;
    return parts > kAttendMaxBytes / each ? kAttendMaxBytes + 1 : parts * each;
}

template <typename T, int D>
static cudaError_t launch_prefill(const AttendArgs& a, const PrePlan& p, cudaStream_t s)
{
    const int bytes = int(sizeof(PreShared<D>)) + 1024;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kv_prefill_kernel<T, D>), bytes);
    if (e != cudaSuccess) return e;
    if (p.units * p.splits > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kv_prefill_kernel<T, D><<<dim3(unsigned(p.units * p.splits), unsigned(a.c.kv_heads)), kPreBlock, bytes, s>>>(a, p.splits, p.stretch);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_kv_join(a, p.splits, p.stretch, 0, s);
}

cudaError_t launch_kv_prefill(const AttendArgs& a, cudaStream_t s)
{
    const PrePlan p = pre_plan(a.c, a.T, a.q_heads, a.R, a.max_len);
    const bool bf = a.dtype == ST_BF16;
    if (a.c.head_dim == 128) return bf ? launch_prefill<__nv_bfloat16, 128>(a, p, s) : launch_prefill<__half, 128>(a, p, s);
    return bf ? launch_prefill<__nv_bfloat16, 64>(a, p, s) : launch_prefill<__half, 64>(a, p, s);
}

}  // namespace st
