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
//   * warps 8-15: bring the next tokens' codes into registers, and convert them to fp16 operands in
//     shared memory (128-byte swizzle): K as [token][dim], V transposed as
//     [dim][token] by byte permutes, so both products read K-major operands;
//   * warp 16: issues tcgen05.mma (M = 128, N = 128 tokens or D dims, K = 16, fp32 sums in TMEM). While
//     one tile's products run, the other tile's softmax does: S and its weights
//     share TMEM columns, 2 x 128 for them and 2 x 128 for O fill all 512.
// Codes are exact in fp16; a block's K scale multiplies its scores, and its V scale (over the
// largest of the stretch) the weights, both in fp32. A weight is p = 2^(s - M) with M
// raised only when a score exceeds it by 8 (then O is rescaled in TMEM): p
// stays below 2^8, fine for fp16 and for the fp32 sum.
//
// Waits are bounded: one that runs out sets the error word and an abort flag, the
// roles leave their loops, and the CTA frees its TMEM after a last bounded wait
// for the products in flight.
#include "attend.cuh"
#include "tc_ptx.cuh"

namespace st {

constexpr int kPreTile = 128;                  // tokens per step
constexpr int kPreCols = 256;                  // columns per CTA: two tiles
constexpr int kPreProducers = 256;
constexpr int kPreBlock = 512 + 32;
constexpr int kPreMaxStretch = 16384;          // tokens: the table of a stretch is held in shared memory
constexpr int kPreMaxBlocks = kPreMaxStretch / 16;
constexpr int kPreStages = 2;
constexpr uint32_t kPreWaitLimit = 1u << 22;
constexpr float kPreRaise = 8.f;

template <int D>
struct PreShared {
    alignas(1024) uint8_t q[2][D / 64][kPreTile * 128];           // two tiles, halves of 64 dims, 128 rows of 128 bytes
    alignas(1024) uint8_t k[kPreStages][D / 64][kPreTile * 128];  // 128 tokens
    alignas(1024) uint8_t v[kPreStages][2][D * 128];              // halves of 64 tokens, D rows of 128 bytes
    int32_t page[kPreMaxBlocks];
    float ks[kPreMaxBlocks], vs[kPreMaxBlocks];                   // ks < 0: the block is hidden
    float vtop[kPreBlock / 32];
    alignas(8) uint64_t k_full[kPreStages], k_empty[kPreStages], v_full[kPreStages], v_empty[kPreStages];
    uint64_t s_full[2], p_ready[2], pv_done[2];
    uint64_t drain;
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

template <typename T, int D>
__global__ void __launch_bounds__(kPreBlock, 1)
kv_prefill_kernel(AttendArgs a, int splits, int stretch, int pairs)
{
    extern __shared__ unsigned char raw[];
    PreShared<D>& sh = *reinterpret_cast<PreShared<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hk = blockIdx.y;
    const int unit = blockIdx.x / splits, split = blockIdx.x - unit * splits;
    const int row = unit / pairs, pair = pairs - 1 - (unit - row * pairs);  // the columns that see most first
    const int G = a.q_heads / a.c.kv_heads, S = a.c.block_size, shift = 31 - __clz(S);

    const int start = min(max(a.row_start[row], 0), int(a.T)), n = min(max(a.row_start[row + 1], start), int(a.T)) - start;
    int64_t len = max(a.lens[row], 0);
    if (len > a.max_len || n > a.max_q) {
        if (split == 0 && hk == 0 && pair == 0 && tid == 0) atomicOr(a.err, kDecErrRow);
        len = 0;
        if (n > a.max_q) {  // more tokens than pairs: the first writes all its zeros
            if (split == 0 && pair == 0) zero_rows<T, D>(a, start, n, hk * G, G);
            return;
        }
    }
    const int64_t col0 = int64_t(pair) * kPreCols, all_cols = int64_t(n) * G;
    if (col0 >= all_cols) return;
    const int cols = int(min(int64_t(kPreCols), all_cols - col0));
    const int64_t j0 = int64_t(split) * stretch;
    if (j0 >= len && split > 0) return;
    // the stretch's tokens that the last column sees
    int64_t end = len;
    if (a.causal) end = min(end, len - n + (col0 + cols - 1) / G + 1);
    const int tokens = int(max(int64_t(0), min(int64_t(stretch), end - j0)));
    const int steps = (tokens + kPreTile - 1) / kPreTile;
    const int tiles = cols > kPreTile ? 2 : 1;

    if (warp == 16) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
        if (lane == 0) {
            for (int i = 0; i < kPreStages; ++i) {
                mbar_init(&sh.k_full[i], kPreProducers / 32);
                mbar_init(&sh.v_full[i], kPreProducers / 32);
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
    // the stretch's blocks
    {
        const int pages = (tokens + S - 1) >> shift;
        const int32_t* table = a.table + int64_t(row) * a.max_blocks + (j0 >> shift);
        float vtop = 0.f;
        for (int i = tid; i < pages; i += kPreBlock) {
            int p = table[i];
            if (p < 0 || p >= a.c.num_blocks) {
                atomicOr(a.err, kDecErrTable);
                p = -1;
            }
            const int64_t at = int64_t(p) * a.c.kv_heads + hk;
            sh.page[i] = p;
            sh.ks[i] = p < 0 ? -1.f : a.c.k_scale[at];
            const float vs = p < 0 ? 0.f : a.c.v_scale[at];
            sh.vs[i] = vs;
            vtop = fmaxf(vtop, vs);
        }
        // up to the end of the last step
        for (int i = pages + tid; i < (steps * kPreTile) >> shift; i += kPreBlock) {
            sh.page[i] = -1;
            sh.ks[i] = -1.f;
            sh.vs[i] = 0.f;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, off));
        if (lane == 0) sh.vtop[warp] = vtop;
    }
    // the queries, a column per softmax thread
    const int tile = warp >> 2, r = tid & 127;  // warps 0-7
    const int64_t col = col0 + tile * kPreTile + r;
    const bool mine = warp < 8 && tile * kPreTile + r < cols;
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
    const float vinv = vtop > 0.f ? 1.f / vtop : 0.f;
    volatile int32_t* abort = &sh.abort;
    auto give_up = [&]() {
        *abort = 1;
        atomicOr(a.err, kDecErrWait);
    };

    float m = -INFINITY, l = 0.f;  // softmax threads
    if (warp == 16) {
        // ------------------------------------------------------------ products --
        if (lane == 0 && steps > 0) {
            constexpr uint32_t idS = idesc_f16(128, kPreTile), idO = idesc_f16(128, D);
            bool ok = true;
            auto scores = [&](int x, int j) {  // S of tile x, step j
                const int st = j % kPreStages;
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    tc_mma_f16(tmem + x * 128, smem_desc_kmajor(smem_u32(sh.q[x][s / 4]) + (s & 3) * 32, 128),
                               smem_desc_kmajor(smem_u32(sh.k[st][s / 4]) + (s & 3) * 32, 128), idS, s > 0);
                tc_commit(&sh.s_full[x]);
            };
            auto values = [&](int x, int j) {  // O += P V
                const int st = j % kPreStages;
#pragma unroll
                for (int s = 0; s < kPreTile / 16; ++s)
                    tc_mma_f16_ts(tmem + 256 + x * 128, tmem + x * 128 + s * 8,
                                  smem_desc_kmajor(smem_u32(sh.v[st][s / 4]) + (s & 3) * 32, 128), idO, j > 0 || s > 0);
                tc_commit(&sh.pv_done[x]);
            };
            ok = mbar_wait(&sh.k_full[0], 0, kPreWaitLimit);
            if (ok) {
                tc_fence_after();
                for (int x = 0; x < tiles; ++x) scores(x, 0);
                tc_commit(&sh.k_empty[0]);
            }
            for (int j = 0; j < steps && ok; ++j) {
                const int st = j % kPreStages, nx = (j + 1) % kPreStages;
                ok = mbar_wait(&sh.v_full[st], j / kPreStages & 1, kPreWaitLimit);
                if (ok && j + 1 < steps) ok = mbar_wait(&sh.k_full[nx], (j + 1) / kPreStages & 1, kPreWaitLimit);
                for (int x = 0; x < tiles && ok; ++x) {
                    ok = !*abort && mbar_wait(&sh.p_ready[x], j & 1, kPreWaitLimit);
                    if (!ok) break;
                    tc_fence_after();
                    values(x, j);
                    if (j + 1 < steps) scores(x, j + 1);
                }
                if (ok) {
                    tc_commit(&sh.v_empty[st]);
                    if (j + 1 < steps) tc_commit(&sh.k_empty[nx]);
                }
            }
            if (!ok) give_up();
            tc_commit(&sh.drain);  // all products issued are done before the TMEM is freed
            if (!mbar_wait(&sh.drain, 0, kPreWaitLimit)) give_up();
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------------ operands --
        const int p = tid - 256, pw = p >> 5;
        constexpr int KN = kPreTile * (D / 16) / kPreProducers;  // 16-byte pieces of K per thread
        constexpr int VN = (D / 32) * 4 / (kPreProducers / 32);  // V tasks (32 dims x 32 tokens) per warp
        constexpr int ROWP = D / 16;
        const int64_t head_bytes = int64_t(S) * D;
        uint4 kr[KN];
        uint32_t vr[VN][8];
        auto rows_at = [&](const int8_t* base, int jj) -> const int8_t* {
            const int page = sh.page[jj >> shift];
            return page < 0 ? nullptr : base + (int64_t(page) * a.c.kv_heads + hk) * head_bytes + (jj & (S - 1)) * D;
        };
        // V task: lane bits 0, 3, 4: a word of the 32 dims; bits 1, 2: a group of 8 tokens
        const int vword = (lane & 1) | (lane >> 3 & 3) << 1, vgroup = lane >> 1 & 3;
        auto load = [&](int j) {
#pragma unroll
            for (int i = 0; i < KN; ++i) {
                const int piece = p % ROWP, t = p / ROWP + i * (kPreProducers / ROWP);
                const int8_t* x = rows_at(a.c.k, j * kPreTile + t);
                kr[i] = x ? ldg_stream(reinterpret_cast<const uint4*>(x + piece * 16)) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const int task = pw * VN + i, dims = (task % (D / 32)) * 32, t0 = (task / (D / 32)) * 32 + vgroup * 8;
                const int8_t* x = rows_at(a.c.v, j * kPreTile + t0);
#pragma unroll
                for (int u = 0; u < 8; ++u) vr[i][u] = x ? __ldg(reinterpret_cast<const uint32_t*>(x + u * D + dims) + vword) : 0u;
            }
        };
        bool ok = true;
        if (steps > 0) load(0);
        for (int j = 0; j < steps && ok; ++j) {
            const int st = j % kPreStages;
            const uint32_t phase = (j / kPreStages & 1) ^ 1;
            ok = !*abort && mbar_wait(&sh.k_empty[st], phase, kPreWaitLimit);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < KN; ++i) {
                const int piece = p % ROWP, t = p / ROWP + i * (kPreProducers / ROWP);
                uint4 lo, hi;
                codes_to_half(kr[i].x, lo.x, lo.y);
                codes_to_half(kr[i].y, lo.z, lo.w);
                codes_to_half(kr[i].z, hi.x, hi.y);
                codes_to_half(kr[i].w, hi.z, hi.w);
                // dims 16 piece ..: pieces 2 (piece % 4) and the next of half piece / 4; the second half's lanes
                // store in the other order, so that eight lanes fill eight different pieces
                uint8_t* to = &sh.k[st][piece / 4][t * 128];
                const int c = (piece & 3) * 2, swap = piece >> 2 & 1;
                *reinterpret_cast<uint4*>(to + (((c + swap) ^ (t & 7)) << 4)) = swap ? hi : lo;
                *reinterpret_cast<uint4*>(to + (((c + (swap ^ 1)) ^ (t & 7)) << 4)) = swap ? lo : hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.k_full[st]);
            ok = !*abort && mbar_wait(&sh.v_empty[st], phase, kPreWaitLimit);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                const int task = pw * VN + i, dims = (task % (D / 32)) * 32, t0 = (task / (D / 32)) * 32 + vgroup * 8;
                uint32_t out[4][4];  // [dim][pairs of tokens]
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t x = vr[i][2 * u] ^ 0x80808080u, y = vr[i][2 * u + 1] ^ 0x80808080u;
                    biased_to_half(__byte_perm(x, y, 0x5140), out[0][u], out[1][u]);
                    biased_to_half(__byte_perm(x, y, 0x7362), out[2][u], out[3][u]);
                }
                const int half = t0 / 64, c = t0 % 64 / 8;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int d = dims + vword * 4 + u;
                    *reinterpret_cast<uint4*>(&sh.v[st][half][d * 128 + ((c ^ (d & 7)) << 4)]) =
                        make_uint4(out[u][0], out[u][1], out[u][2], out[u][3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.v_full[st]);
            if (j + 1 < steps) load(j + 1);
        }
        if (!ok) give_up();
    } else if (tile < tiles) {
        // ------------------------------------------------------------- softmax --
        const uint32_t lanes = uint32_t(warp & 3) << 21;  // TMEM lane 32 (warp % 4) in bits 16 on
        const uint32_t ts = tmem + lanes + tile * 128, to = tmem + lanes + 256 + tile * 128;
        int see = tokens;  // tokens of the stretch that this column sees
        if (mine && a.causal) see = int(max(int64_t(0), min(int64_t(tokens), len - n + col / G + 1 - j0)));
        const int least = __reduce_min_sync(0xffffffffu, see);
        bool ok = true;
        for (int j = 0; j < steps && ok; ++j) {
            ok = !*abort && mbar_wait(&sh.s_full[tile], j & 1, kPreWaitLimit);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int jj0 = j * kPreTile;
            float ks[8], vs[8];  // of each 16 tokens
            bool whole = jj0 + kPreTile <= least;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                ks[b] = sh.ks[(jj0 + 16 * b) >> shift];
                whole = whole && ks[b] >= 0.f;
            }
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float s[32];
                tmem_ld32(ts + 32 * c, s);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float sc = ks[2 * c + h] * mult;
                    float x = -INFINITY;
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x = fmaxf(x, s[16 * h + i]);
                        top = fmaxf(top, x * sc);
                    } else if (ks[2 * c + h] >= 0.f) {
                        const int left = see - (jj0 + 32 * c + 16 * h);
#pragma unroll
                        for (int i = 0; i < 16; ++i) x = i < left ? fmaxf(x, s[16 * h + i]) : x;
                        if (left > 0) top = fmaxf(top, x * sc);
                    }
                }
            }
            // the reference: raised when a score is far above it
            const bool first = m == -INFINITY;
            const bool raise = first ? top > -INFINITY : top > m + kPreRaise;
            if (__any_sync(0xffffffffu, raise && !first)) {
                ok = mbar_wait(&sh.pv_done[tile], (j - 1) & 1, kPreWaitLimit);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float z = raise && !first ? ex2(m - top) : 1.f;
                l *= z;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(to + 32 * c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= z;
                    tmem_st32(to + 32 * c, o);
                }
                tmem_wait_st();
            }
            if (raise) m = top;
            const float base = m > -INFINITY ? m : 0.f;
#pragma unroll
            for (int b = 0; b < 8; ++b) vs[b] = sh.vs[(jj0 + 16 * b) >> shift] * vinv;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float s[32];
                tmem_ld32(ts + 32 * c, s);
                tmem_wait_ld();
                uint32_t p[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float sc = ks[2 * c + h] * mult, vf = vs[2 * c + h];
                    const int left = see - (jj0 + 32 * c + 16 * h);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float2 x = fma2(make_float2(s[16 * h + 2 * i], s[16 * h + 2 * i + 1]), make_float2(sc, sc), make_float2(-base, -base));
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        if (!whole) {
                            const bool on = ks[2 * c + h] >= 0.f;
                            x.x = on && 2 * i < left ? x.x : 0.f;
                            x.y = on && 2 * i + 1 < left ? x.y : 0.f;
                        }
                        sum = add2(sum, x);
                        x = mul2(x, make_float2(vf, vf));
                        p[8 * h + i] = pack_half2(x.x, x.y);
                    }
                }
                // over the scores just read: tokens 32 c .. 32 c + 31 take columns 16 c ..
                tmem_st16(ts + 16 * c, p);
            }
            l += sum.x + sum.y;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_ready[tile]);
        }
        if (ok && steps > 0) ok = mbar_wait(&sh.pv_done[tile], (steps - 1) & 1, kPreWaitLimit);
        if (!__all_sync(0xffffffffu, ok)) {
            give_up();
        } else {
            tc_fence_after();
            const float scale = splits == 1 ? (l == 0.f ? 0.f : vtop / l) : vtop;
            T* out = static_cast<T*>(a.out) + token * a.out_token + head * a.out_head;
            const int64_t part = (token * a.q_heads + head) * splits + split;
            float* po = static_cast<float*>(a.workspace);
            if (mine && splits > 1) {
                float* pm = po + a.T * a.q_heads * splits * D;
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
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
                if (!mine) {
                    // the loads above are the whole warp's
                } else if (splits == 1) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        T y[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) y[u] = from_float<T>(l == 0.f ? 0.f : o[8 * i + u] * scale);
                        *reinterpret_cast<uint4*>(out + 32 * c + 8 * i) = *reinterpret_cast<const uint4*>(y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(po + part * D + 32 * c + 4 * i) =
                            make_float4(o[4 * i] * scale, o[4 * i + 1] * scale, o[4 * i + 2] * scale, o[4 * i + 3] * scale);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

struct PrePlan {
    int splits, stretch, pairs;
};

// Stretches: one while the columns alone fill the GPU, else enough for two CTAs per SM, none longer than the
// table that fits, of at least 1024 tokens.
static PrePlan pre_plan(const st_kv_cache& c, int32_t q_heads, int32_t R, int32_t max_q, int64_t max_len)
{
    PrePlan p;
    const int64_t cols = int64_t(max_q) * (q_heads / c.kv_heads);
    p.pairs = int((cols + kPreCols - 1) / kPreCols);
    const int64_t units = int64_t(R) * c.kv_heads * p.pairs, wanted = 2 * 148;
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

int64_t kv_prefill_workspace(const st_kv_cache& c, int64_t T, int32_t q_heads, int32_t R, int32_t max_q, int64_t max_len)
{
    const PrePlan p = pre_plan(c, q_heads, R, max_q, max_len);
    return p.splits == 1 ? 0 : T * q_heads * p.splits * (int64_t(c.head_dim) + 2) * 4;
}

template <typename T, int D>
static cudaError_t launch_prefill(const AttendArgs& a, const PrePlan& p, cudaStream_t s)
{
    const int bytes = int(sizeof(PreShared<D>)) + 1024;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kv_prefill_kernel<T, D>), bytes);
    if (e != cudaSuccess) return e;
    const int64_t ctas = int64_t(a.R) * p.pairs * p.splits;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kv_prefill_kernel<T, D><<<dim3(unsigned(ctas), unsigned(a.c.kv_heads)), kPreBlock, bytes, s>>>(a, p.splits, p.stretch, p.pairs);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_kv_join(a, p.splits, p.stretch, s);
}

cudaError_t launch_kv_prefill(const AttendArgs& a, cudaStream_t s)
{
    const PrePlan p = pre_plan(a.c, a.q_heads, a.R, a.max_q, a.max_len);
    const bool bf = a.dtype == ST_BF16;
    if (a.c.head_dim == 128) return bf ? launch_prefill<__nv_bfloat16, 128>(a, p, s) : launch_prefill<__half, 128>(a, p, s);
    return bf ? launch_prefill<__nv_bfloat16, 64>(a, p, s) : launch_prefill<__half, 64>(a, p, s);
}

}  // namespace st
