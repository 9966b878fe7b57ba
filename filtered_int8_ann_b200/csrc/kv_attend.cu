// Attention of a few query tokens per row over an int8 paged cache (a decode step).
//
// Bound by the cache's bytes: every code is read once per group of query
// heads that share it. The work is split along the cache: a CTA takes one row, one cache
// head, up to 16 "columns" (query token, head) and a stretch of tokens; its four
// warps take 32 tokens at a time, and the stretches are joined by a second
// launch when there are several.
//
// One pass with a running maximum, in powers of two:
//   s_j = scale log2(e) ks <q, k_j>, M = max s_j, p_j = 2^(s_j - M), l = sum p_j, O = sum p_j v_j.
// Products run on mma.sync (m16n8k16, fp16 with fp32 sums): with at most 16 columns a tcgen05 tile
// of 128 rows would be almost empty, and the converted codes would have to go back through
// shared memory; here they go from there to registers in the order the fragments want:
//   S^T = K Q^T    A = 16 tokens x 16 dims: lane (g, t) loads 16 dims of tokens g and g + 8 as
//                  one vector; which dims stand at which k index is free as long as Q agrees
//   O^T = V^T P^T  A = 16 dims x 16 tokens: lane (g, t) loads D/8 dims of four tokens and pairs
//                  the tokens' bytes with byte permutes; B = P^T is S^T's accumulator transposed by movmatrix
// Each warp copies its next 32 tokens (cp.async, 16 bytes a lane) while it works on
// the last: 12 warps per SM keep 96 KB of codes under way, where loads to registers kept too
// few (64 rows of up to 16384 tokens, 8 cache heads of 128, 4 query heads each: 404 us; 240 so). The 16-byte pieces of
// a 128-byte line are permuted by the token so that both kinds of loads are free of bank conflicts.
// That case reads 1.33 GB at 5.5 TB/s, 85% of a plain copy's rate: blocks of 32 tokens are pieces of 4 KB anywhere in
// memory, which costs about 7% against neighbouring ones, and the last wave of CTAs is not full. One row of 100003
// tokens (205 MB): 50 us against 31 at that rate; each CTA's way to its first product and the join are 12 of them.
// A code becomes fp16 exactly: with the sign bit flipped it is the low byte of 1024 + 128 + code.
// A query is scaled by a power of two to below 2 (exact in fp16 down to 2^-24 of
// its largest element). The V operand's weight is 2^15 p_j vs_j / max vs: p_j is at most 1, so that fp16 holds
// it with 11 bits down to 2^-29 of the largest and to 2^-40 of it below (many small weights may make up a
// sum); maxima, sums and O stay in fp32.
#include "attend.cuh"

namespace st {

constexpr int kDecWarps = 4;
constexpr int kDecBlock = 32 * kDecWarps;
// Columns (query tokens x heads per cache head) up to which this kernel is taken, 16 at a time: with 24 to 32 it took
// 256 to 270 us for 32 rows of 8192 tokens and the prompts' kernel 340, with 40 it took 380 and that one 297. A block of 16
// columns copies and converts the cache for itself: such rows (8 cache heads of 128, 4 query heads each) take 104 us with one
// query token, 110 with 2, 151 with 4, 283 with 8 and 301 with 16; their bytes are 82.
constexpr int kDecMaxCols = 32;
constexpr int kDecGroup = 32;             // tokens a warp takes at a time
constexpr int kDecSixteens = 4096 / 16 + 2 * kDecWarps * kDecGroup / 16;  // of the longest stretch, and of the stages copied past it
constexpr int kDecMaxStretch = 4096;      // tokens
constexpr int64_t kDecRoom = int64_t(128) << 20;  // bytes of partial sums beside prompts
constexpr float kDecUp = 0x1p15f;         // of the weights in fp16

template <int D, int NT>
struct DecShared {
    // of each 16 tokens of the stretch: where their codes begin (-1: none), their block's K scale, its V scale over
    // the largest of the stretch
    int64_t at[kDecSixteens];
    float ks[kDecSixteens], vs[kDecSixteens];
    float m[kDecWarps][8 * NT], l[kDecWarps][8 * NT];
    union {
        alignas(128) uint8_t codes[kDecWarps][2][2][kDecGroup * D];  // per warp: two stages of K and V codes
        float o[kDecWarps][8 * NT][D + 4];              // at the end: the warps' sums
    };
};

// Where 16-byte piece `c` of token r stands among its warp's codes: in line r
// (two tokens per line for D = 64), pieces permuted.
template <int D>
__device__ __forceinline__ int piece_at(int r, int c)
{
    if (D == 128) return r * 128 + ((c ^ ((r & 1) << 2 | (r >> 1 & 3))) << 4);
    return (r >> 1) * 128 + ((((r & 1) << 2 | c) ^ (r >> 1 & 3) << 1) << 4);
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// A lane's dims of a V row: 16 (D = 128) or 8 (D = 64)
template <int D>
struct VecV;
template <>
struct VecV<128> { using type = uint4; };
template <>
struct VecV<64> { using type = uint2; };

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kDecBlock, 3)
kv_decode_kernel(AttendArgs a, int splits, int stretch, int col_blocks)
{
    constexpr int KV = D / 64;    // 16-byte vectors of a K row per lane
    constexpr int MT = D / 16;    // m-tiles of O^T
    constexpr int VW = D / 32;    // words of a V row per lane
    constexpr int COLS = 8 * NT;
    using V = typename VecV<D>::type;
    extern __shared__ __align__(16) unsigned char raw[];
    DecShared<D, NT>& sh = *reinterpret_cast<DecShared<D, NT>*>(raw);
    __shared__ float s_vmax[kDecWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    // the cache heads of one stretch run together: their codes lie side by side in each block
    const int hk = blockIdx.x % a.c.kv_heads, part_id = blockIdx.x / a.c.kv_heads, unit = part_id / splits, split = part_id - unit * splits;
    const int row = unit / col_blocks, col0 = (unit - row * col_blocks) * COLS;
    const int G = a.q_heads / a.c.kv_heads, S = a.c.block_size;

    const int start = min(max(a.row_start[row], 0), int(a.T)), n = min(max(a.row_start[row + 1], start), int(a.T)) - start;
    int64_t len = max(a.lens[row], 0);
    if (int64_t(n) * G <= a.above_cols || int64_t(n) * G > a.most_cols) return;  // another launch's row
    if (len > a.max_len || n > a.max_q) {
        if (split == 0 && hk == 0 && col0 == 0 && tid == 0) atomicOr(a.err, kDecErrRow);
        len = 0;
        if (n > a.max_q) {  // more tokens than column blocks: the first writes all its zeros
            if (split == 0 && col0 == 0) zero_rows<T, D>(a, start, n, hk * G, G);
            return;
        }
    }
    const int cols = min(COLS, n * G - col0);  // of this block
    if (cols <= 0) return;
    const int64_t j0 = int64_t(split) * stretch;
    if (j0 >= len && split > 0) return;  // the join knows how many stretches a row has
    const int tokens = int(min(int64_t(stretch), len - j0));

    // the stretch's tokens in sixteens, and as many more as stages are copied ahead
    const int shift = 31 - __clz(S), sixteens = (tokens + 15) / 16;
    const int32_t* table = a.table + int64_t(row) * a.max_blocks + (j0 >> shift);
    for (int i = tid; i < sixteens + 2 * kDecWarps * kDecGroup / 16; i += kDecBlock) {
        int p = -1;
        if (i < sixteens) {
            p = table[(16 * i) >> shift];
            if (p < 0 || p >= a.c.num_blocks) {
                atomicOr(a.err, kDecErrTable);
                p = -1;
            }
        }
        sh.at[i] = p < 0 ? -1 : ((int64_t(p) * a.c.kv_heads + hk) * S + ((16 * i) & (S - 1))) * D;
    }
    __syncthreads();
    // Codes of the 32 tokens of sixteens i and i + 1 into stage `st`: each sixteen is one run of bytes.
    uint8_t* codes = sh.codes[warp][0][0];
    const uint32_t codes_at = smem_u32(codes);
    constexpr int kStage = 2 * kDecGroup * D, kHalf = 16 * D, kCopies = kHalf / 512;
    constexpr int kLaneRows = 512 / D;  // tokens that a warp's copy covers
    uint32_t dst[2];  // of copies with even and odd numbers
#pragma unroll
    for (int i = 0; i < 2; ++i)
        dst[i] = codes_at + piece_at<D>(i * kLaneRows + lane / (D / 16), lane % (D / 16)) - i * 512;
    const int8_t *const from_k = a.c.k + lane * 16, *const from_v = a.c.v + lane * 16;
    auto copy_stage = [&](int i16, int st) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t at = sh.at[i16 + h];
            if (at >= 0) {
                const int8_t *k = from_k + at, *v = from_v + at;
                const uint32_t to = uint32_t(st * kStage + h * kHalf);
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    copy_async(dst[i & 1] + to + i * 512, k + i * 512);
                    copy_async(dst[i & 1] + to + kDecGroup * D + i * 512, v + i * 512);
                }
            }
        }
        cp_async_commit();
    };
    copy_stage(warp * (kDecGroup / 16), 0);  // on its way while scales and queries come
    float vmax = 0.f;
    for (int i = tid; i < sixteens + 2 * kDecWarps * kDecGroup / 16; i += kDecBlock) {
        const int64_t at = sh.at[i], block = at >> (shift + (D == 128 ? 7 : 6));
        sh.ks[i] = at < 0 ? 0.f : a.c.k_scale[block];
        const float vs = at < 0 ? 0.f : a.c.v_scale[block];
        sh.vs[i] = vs;
        vmax = fmaxf(vmax, vs);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
    if (lane == 0) s_vmax[warp] = vmax;

    // queries: lane (g, t) holds dims 16 t .. 16 t + 15 (and 64 on) of columns g, g + 8, ...
    uint32_t q[NT][KV][8];
    float mult[NT][2];  // of columns 8 nt + 2 t and the next: scale log2(e) and the query's power of two
    int seen[NT][2];    // tokens of the stretch that the column sees
    float own_mult[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int c = 8 * nt + g, col = col0 + c;
        float x[KV * 16];
#pragma unroll
        for (int i = 0; i < KV * 16; ++i) x[i] = 0.f;
        if (c < cols) {
            const T* p = static_cast<const T*>(a.q) + int64_t(start + col / G) * a.q_token +
                         int64_t(hk * G + col % G) * a.q_head + 16 * t;
#pragma unroll
            for (int v = 0; v < KV; ++v) {
                unpack8<T>(*reinterpret_cast<const uint4*>(p + 64 * v), x + 16 * v);
                unpack8<T>(*reinterpret_cast<const uint4*>(p + 64 * v + 8), x + 16 * v + 8);
            }
        }
        float big = 0.f;
        bool finite = true;
#pragma unroll
        for (int i = 0; i < KV * 16; ++i) {
            big = fmaxf(big, fabsf(x[i]));
            finite = finite && fabsf(x[i]) < INFINITY;
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const unsigned ok = __ballot_sync(0xffffffffu, finite) >> (lane & 28) & 15u;
        // a negative scale's sign goes to the query: scores are then multiplied by positive numbers
        const float down = ok == 15u ? copysignf(pow2_down(big), a.scale_log2) : 0.f, up = ok == 15u ? pow2_up(big) : NAN;
#pragma unroll
        for (int v = 0; v < KV; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[nt][v][i] = ok == 15u ? pack_half2(x[16 * v + 2 * i] * down, x[16 * v + 2 * i + 1] * down) : 0u;
        own_mult[nt] = fabsf(a.scale_log2) * up;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = 2 * t + i;
            mult[nt][i] = __shfl_sync(0xffffffffu, own_mult[nt], 4 * c);
            const int col = col0 + 8 * nt + c;
            int64_t see = len - j0;
            if (a.causal) see = len - n + col / G + 1 - j0;
            seen[nt][i] = 8 * nt + c < cols ? int(max(int64_t(0), min(int64_t(tokens), see))) : 0;
        }
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may come up meanwhile
    float vtop = s_vmax[0];
#pragma unroll
    for (int w = 1; w < kDecWarps; ++w) vtop = fmaxf(vtop, s_vmax[w]);
    {
        for (int i = tid; i < sixteens; i += kDecBlock) sh.vs[i] = vtop > 0.f ? __fdiv_rn(sh.vs[i], vtop) * kDecUp : 0.f;
    }
    __syncthreads();
    int least_seen = 0x7fffffff;  // of the whole warp's columns: tiles below it need no mask
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (8 * nt + 2 * t + i < cols) least_seen = min(least_seen, seen[nt][i]);
    }
    least_seen = __reduce_min_sync(0xffffffffu, least_seen);

    float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }

    // lane (g, t)'s pieces: K pieces t (and t + 4) of tokens g, g + 8; V dims of tokens 2t, 2t+1 (and + 8)
    const int vdim = D == 128 ? (g >> 1 | (g & 1) << 2) * 16 : g * 8;  // first of the lane's D/8 dims of V
    const int k_at[2] = {piece_at<D>(g, t), D == 128 ? piece_at<D>(g, t + 4) : 0};
    const int v_at[2] = {kDecGroup * D + piece_at<D>(2 * t, vdim / 16) + vdim % 16,
                         kDecGroup * D + piece_at<D>(2 * t + 1, vdim / 16) + vdim % 16};
    int stage = 0;
    for (int jj0 = warp * kDecGroup; jj0 < tokens; jj0 += kDecWarps * kDecGroup, stage ^= 1) {
        copy_stage(jj0 / 16 + kDecWarps * (kDecGroup / 16), stage ^ 1);
        cp_async_wait_group<1>();
        __syncwarp();
        const uint8_t* from = codes + stage * kStage;
        float s[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[h][nt][0] = s[h][nt][1] = s[h][nt][2] = s[h][nt][3] = 0.f;
#pragma unroll
            for (int v = 0; v < KV; ++v) {
                const uint4 x0 = *reinterpret_cast<const uint4*>(from + h * kHalf + k_at[v]);
                const uint4 x1 = *reinterpret_cast<const uint4*>(from + h * kHalf + 8 * D + k_at[v]);
                const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t f[4];
                    codes_to_half(w0[i], f[0], f[2]);
                    codes_to_half(w1[i], f[1], f[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma16816(s[h][nt], f, q[nt][v][2 * i], q[nt][v][2 * i + 1]);
                }
            }
        }
        // the columns' maxima; a sixteen's factor takes its products to scores
        float f[2], sc[2][NT][2];
        float mx[NT][2];
        const bool whole = jj0 + kDecGroup <= least_seen && sh.at[jj0 / 16] >= 0 && sh.at[jj0 / 16 + 1] >= 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mx[nt][0] = m[nt][0];
            mx[nt][1] = m[nt][1];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float ks = sh.ks[jj0 / 16 + h];
            f[h] = sh.vs[jj0 / 16 + h];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                sc[h][nt][0] = ks * mult[nt][0];
                sc[h][nt][1] = ks * mult[nt][1];
            }
        }
        if (!whole) {  // scores now (rounded), those that the column does not see masked
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int jj = jj0 + 16 * h;
                const bool none = sh.at[jj / 16] < 0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[h][nt][i] = !none && jj + g + 8 * (i >> 1) < seen[nt][i & 1] ? __fmul_rn(s[h][nt][i], sc[h][nt][i & 1]) : -INFINITY;
                    sc[h][nt][0] = sc[h][nt][1] = 1.f;
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) mx[nt][i] = fmaxf(mx[nt][i], fmaxf(s[h][nt][i], s[h][nt][2 + i]) * sc[h][nt][i]);
        bool grew = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1)
                    mx[nt][i] = fmaxf(mx[nt][i], __shfl_xor_sync(0xffffffffu, mx[nt][i], off));
                grew = grew || mx[nt][i] > m[nt][i];
            }
        if (__any_sync(0xffffffffu, grew)) {
            bool some = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float shrink[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float up = mx[nt][i] > m[nt][i] ? just_above(mx[nt][i]) : m[nt][i];
                    shrink[i] = up > m[nt][i] ? ex2(m[nt][i] - up) : 1.f;
                    m[nt][i] = up;
                    l[nt][i] *= shrink[i];
                    some = some || is_far(up);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[nt][i][0] *= shrink[0];
                    o[nt][i][1] *= shrink[1];
                    o[nt][i][2] *= shrink[0];
                    o[nt][i][3] *= shrink[1];
                }
            }
            if (__any_sync(0xffffffffu, some)) {  // this step's scores are rounded now, later ones as those of a masked step
                least_seen = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[h][nt][i] = __fmul_rn(s[h][nt][i], sc[h][nt][i & 1]);
                        sc[h][nt][0] = sc[h][nt][1] = 1.f;
                    }
            }
        }
        // weights, transposed to the B fragments of 16 tokens x 8 columns
        uint32_t p[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float b0 = m[nt][0] > -INFINITY ? m[nt][0] : 0.f, b1 = m[nt][1] > -INFINITY ? m[nt][1] : 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float p0 = ex2(fmaf(s[h][nt][2 * r], sc[h][nt][0], -b0)), p1 = ex2(fmaf(s[h][nt][2 * r + 1], sc[h][nt][1], -b1));
                    l[nt][0] += p0;
                    l[nt][1] += p1;
                    p[h][nt][r] = transpose8x8(pack_half2(p0 * f[h], p1 * f[h]));
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            V vreg[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) vreg[i] = *reinterpret_cast<const V*>(from + h * kHalf + (i >> 1) * 8 * D + v_at[i & 1]);
            const uint32_t* w[4] = {reinterpret_cast<const uint32_t*>(&vreg[0]), reinterpret_cast<const uint32_t*>(&vreg[1]),
                                    reinterpret_cast<const uint32_t*>(&vreg[2]), reinterpret_cast<const uint32_t*>(&vreg[3])};
#pragma unroll
            for (int i = 0; i < VW; ++i) {  // four dims of the four tokens
                const uint32_t x0 = w[0][i] ^ 0x80808080u, x1 = w[1][i] ^ 0x80808080u, x2 = w[2][i] ^ 0x80808080u,
                               x3 = w[3][i] ^ 0x80808080u;
                const uint32_t a01 = __byte_perm(x0, x1, 0x5140), b01 = __byte_perm(x0, x1, 0x7362);
                const uint32_t a23 = __byte_perm(x2, x3, 0x5140), b23 = __byte_perm(x2, x3, 0x7362);
                uint32_t f0[4], f1[4];
                biased_to_half(a01, f0[0], f0[1]);
                biased_to_half(a23, f0[2], f0[3]);
                biased_to_half(b01, f1[0], f1[1]);
                biased_to_half(b23, f1[2], f1[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma16816(o[nt][2 * i], f0, p[h][nt][0], p[h][nt][1]);
                    mma16816(o[nt][2 * i + 1], f1, p[h][nt][0], p[h][nt][1]);
                }
            }
        }
        __syncwarp();  // the stage is copied into again
    }

    // join the warps
    cp_async_wait_group<0>();
    __syncthreads();  // the codes' memory is used again
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], off);
            const int c = 8 * nt + 2 * t + i;
            if (g == 0) {
                sh.m[warp][c] = m[nt][i];
                sh.l[warp][c] = l[nt][i];
            }
#pragma unroll
            for (int k = 0; k < MT; ++k) {  // dims vdim + 2 k and the next
                sh.o[warp][c][vdim + 2 * k] = o[nt][k][i];
                sh.o[warp][c][vdim + 2 * k + 1] = o[nt][k][2 + i];
            }
        }
    __syncthreads();
    for (int i = tid; i < cols * D; i += kDecBlock) {
        const int c = i / D, d = i - c * D, col = col0 + c;
        float top = sh.m[0][c];
#pragma unroll
        for (int w = 1; w < kDecWarps; ++w) top = fmaxf(top, sh.m[w][c]);
        const float base = top > -INFINITY ? top : 0.f;
        float sum = 0.f, val = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            const float z = sh.m[w][c] > -INFINITY ? ex2(sh.m[w][c] - base) : 0.f;
            sum += sh.l[w][c] * z;
            val += sh.o[w][c][d] * z;
        }
        // a column whose query is not finite has NaN scores, a NaN sum and no maximum
        const int64_t token = start + col / G, head = hk * G + col % G;
        if (splits == 1) {
            static_cast<T*>(a.out)[token * a.out_token + head * a.out_head + d] =
                from_float<T>(sum == 0.f ? 0.f : val / (kDecUp * sum) * vtop);
        } else {
            const int64_t of = a.row_cols > 0 ? (int64_t(row) * a.c.kv_heads + hk) * a.row_cols + col : token * a.q_heads + head;
            const int64_t part = of * splits + split;
            float* po = static_cast<float*>(a.workspace);
            float* pm = po + a.parts * splits * D;
            po[part * D + d] = val * (1.f / kDecUp) * vtop;
            if (d == 0) {
                pm[2 * part] = top;
                pm[2 * part + 1] = sum;
            }
        }
    }
}

// Join a query head's stretches: groups of D threads take every so many of them each.
template <typename T, int D, int kJoinBlock>
__global__ void __launch_bounds__(kJoinBlock) kv_join_kernel(AttendArgs a, int splits, int stretch, int per_row)
{
    constexpr int GROUPS = kJoinBlock / D, kChunk = kJoinBlock;
    __shared__ float s_w[kChunk], s_red[kJoinBlock / 32], s_o[GROUPS][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, d = tid % D, group = tid / D;
    const int G = a.q_heads / a.c.kv_heads;
    int lo;
    int64_t token, head;
    // Every CTA waits for the stretches' launch, those without work too: what follows this launch then follows that one.
    auto wait = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
    if (per_row > 0) {  // per_row columns of each row and cache head
        const int64_t unit = blockIdx.x / per_row;
        const int col = int(blockIdx.x - unit * per_row);
        lo = int(unit / a.c.kv_heads);
        token = int64_t(max(a.row_start[lo], 0)) + col / G;
        head = (unit - int64_t(lo) * a.c.kv_heads) * G + col % G;
        if (token >= min(a.row_start[lo + 1], int(a.T))) return wait();
    } else {  // the query heads of every token
        token = blockIdx.x / a.q_heads;
        head = blockIdx.x - token * a.q_heads;
        int hi = a.R;  // the row holding the token
        lo = 0;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.row_start[mid + 1] > token) hi = mid;
            else lo = mid + 1;
        }
        if (lo == a.R || a.row_start[lo] > token) return wait();
    }
    const int n = a.row_start[lo + 1] - a.row_start[lo];
    const int64_t cols = int64_t(n) * G;
    int64_t len = max(a.lens[lo], 0);
    if (n > a.max_q || cols <= a.above_cols || cols > a.most_cols) return wait();  // written already, or another launch's
    if (len > a.max_len) len = 0;
    const int64_t unit = a.row_cols > 0 ? int64_t(blockIdx.x) : token * a.q_heads + head;  // (the CTAs are numbered so)
    const int used = int(max(int64_t(1), (len + stretch - 1) / stretch));
    const float* po = static_cast<const float*>(a.workspace);
    const float* pm = po + a.parts * splits * D + 2 * unit * splits;
    po += unit * splits * D + d;
    wait();  // what the stretches' launch wrote is read from here on
    float top = -INFINITY;
    for (int i = tid; i < used; i += kJoinBlock) top = fmaxf(top, pm[2 * i]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) s_red[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinBlock / 32; ++w) top = fmaxf(top, s_red[w]);
    const float base = top > -INFINITY ? top : 0.f;
    float sum = 0.f, val = 0.f;
    for (int c0 = 0; c0 < used; c0 += kChunk) {
        const int c = min(kChunk, used - c0);
        __syncthreads();
        if (tid < c) {
            const float m = pm[2 * (c0 + tid)];
            s_w[tid] = m > -INFINITY ? ex2(m - base) : 0.f;
            sum += pm[2 * (c0 + tid) + 1] * s_w[tid];
        }
        __syncthreads();
#pragma unroll 8
        for (int i = group; i < c; i += GROUPS) val += po[int64_t(c0 + i) * D] * s_w[i];
    }
    // sums over the threads and groups
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    __syncthreads();
    if (lane == 0) s_red[warp] = sum;
    s_o[group][d] = val;
    __syncthreads();
    if (group == 0) {
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinBlock / 32; ++w) sum += s_red[w];
        val = 0.f;
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) val += s_o[k][d];
        static_cast<T*>(a.out)[token * a.out_token + head * a.out_head + d] = from_float<T>(sum == 0.f ? 0.f : val / sum);
    }
}

struct DecPlan {
    int splits, stretch, cols, col_blocks;
    int per_row;    // most columns of a row
    int64_t parts;  // columns with partial sums, and how they are numbered (AttendArgs)
    int row_cols;
    int64_t bytes;  // of the workspace: a multiple of 16, the prompts' kernel's part may follow
};

// Stretches, multiples of the longest block, from the bound that the host knows: rows much shorter than max_len use few of
// the CTAs (one row of 32768 tokens 22 us, under a bound of 131072 30). One row fills the GPU's places (3 CTAs per SM) once, all with
// the same work (100003 tokens: 49 us; in two to four turns 52 to 62). Several rows, which may be uneven, get about
// three CTAs per place, of 256 to 1024 tokens, so that the long ones' stretches fill in behind the short ones.
// A short row is one stretch, which needs no join.
// Partial sums are numbered by token, or by row where that takes less room: beside prompts, and with tokens behind the
// last row's. Where short rows stand beside prompts, the host knows only that each of them may have kDecMaxCols columns:
// a workspace above kDecRoom then takes longer stretches (63 rows of up to 65536 tokens beside a prompt of 2048, 8 cache
// heads of 128, 4 query heads each: 130 MiB and, prompt included, 1198 us; with stretches of 1024 520 MiB and 1504 us).
static DecPlan dec_plan(const st_kv_cache& c, int64_t T, int32_t q_heads, int32_t R, int32_t max_q, int64_t max_len, bool mixed)
{
    DecPlan p;
    const int64_t cols = int64_t(max_q) * (q_heads / c.kv_heads);
    p.per_row = int(cols);
    p.cols = cols <= 8 ? 8 : 16;
    p.col_blocks = int((cols + p.cols - 1) / p.cols);
    const int64_t places = 3 * 148;
    const int64_t units = int64_t(R) * c.kv_heads * p.col_blocks;
    int64_t stretch;
    if (R == 1) {
        const int64_t each = places / units > 1 ? places / units : 1;
        stretch = (max_len + each - 1) / each;
        stretch = stretch < 256 ? 256 : stretch > kDecMaxStretch ? 1024 : stretch;
    } else {
        stretch = (max_len * units + 3 * places - 1) / (3 * places);
        stretch = stretch < 256 ? 256 : stretch > 1024 ? 1024 : stretch;
    }
    stretch = (stretch + 127) / 128 * 128;
    if (max_len <= 512) stretch = 512;
    const int64_t by_token = T * q_heads, by_row = int64_t(R) * c.kv_heads * cols;
    p.row_cols = by_row < by_token ? int(cols) : 0;
    p.parts = by_row < by_token ? by_row : by_token;
    while (true) {
        p.splits = int((max_len + stretch - 1) / stretch);
        p.bytes = p.splits == 1 ? 0 : (p.parts * p.splits * (int64_t(c.head_dim) + 2) * 4 + 15) / 16 * 16;
        if (!mixed || p.bytes <= kDecRoom || 2 * stretch > kDecMaxStretch) break;
        stretch *= 2;
    }
    p.stretch = int(stretch);
    return p;
}

template <typename T, int D, int NT>
static cudaError_t launch_decode(const AttendArgs& a, const DecPlan& p, cudaStream_t s)
{
    const int bytes = int(sizeof(DecShared<D, NT>));
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kv_decode_kernel<T, D, NT>), bytes);
    if (e != cudaSuccess) return e;
    const int64_t ctas = int64_t(a.R) * p.col_blocks * p.splits * a.c.kv_heads;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kv_decode_kernel<T, D, NT><<<unsigned(ctas), kDecBlock, bytes, s>>>(a, p.splits, p.stretch, p.col_blocks);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.splits == 1) return e;
    return launch_kv_join(a, p.splits, p.stretch, p.per_row, s);
}

template <typename T, int D>
static cudaError_t launch_join(const AttendArgs& a, int splits, int stretch, int per_row, int64_t ctas, cudaStream_t s)
{
    const dim3 grid{unsigned(ctas)};
    // few stretches are joined faster by small CTAs, many heads at a time (2048 heads of up to 16: the call took 236 us, by
    // 512 threads 256), many by large ones (64 heads of 53: 49 us, by 128 threads 51)
    if (splits <= 16) return launch_dep(kv_join_kernel<T, D, 128>, grid, dim3(128), 0, s, a, splits, stretch, per_row);
    return launch_dep(kv_join_kernel<T, D, 512>, grid, dim3(512), 0, s, a, splits, stretch, per_row);
}

cudaError_t launch_kv_join(const AttendArgs& a, int splits, int stretch, int per_row, cudaStream_t s)
{
    const int64_t ctas = per_row > 0 ? int64_t(a.R) * a.c.kv_heads * per_row : a.T * a.q_heads;
    if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const bool bf = a.dtype == ST_BF16;
    if (a.c.head_dim == 128)
        return bf ? launch_join<__nv_bfloat16, 128>(a, splits, stretch, per_row, ctas, s)
                  : launch_join<__half, 128>(a, splits, stretch, per_row, ctas, s);
    return bf ? launch_join<__nv_bfloat16, 64>(a, splits, stretch, per_row, ctas, s)
              : launch_join<__half, 64>(a, splits, stretch, per_row, ctas, s);
}

static cudaError_t launch_kv_decode(const AttendArgs& a, const DecPlan& p, cudaStream_t s)
{
    const bool bf = a.dtype == ST_BF16, wide = a.c.head_dim == 128, two = p.cols > 8;
    if (wide && two) return bf ? launch_decode<__nv_bfloat16, 128, 2>(a, p, s) : launch_decode<__half, 128, 2>(a, p, s);
    if (wide) return bf ? launch_decode<__nv_bfloat16, 128, 1>(a, p, s) : launch_decode<__half, 128, 1>(a, p, s);
    if (two) return bf ? launch_decode<__nv_bfloat16, 64, 2>(a, p, s) : launch_decode<__half, 64, 2>(a, p, s);
    return bf ? launch_decode<__nv_bfloat16, 64, 1>(a, p, s) : launch_decode<__half, 64, 1>(a, p, s);
}

// Which kernels a call takes: rows of up to kDecMaxCols columns go to the decode kernel, the others to the
// prompts' kernel; a batch that may hold both kinds takes both.
struct AttendPlan {
    bool decode, prefill;
    DecPlan dec;
};

static AttendPlan attend_plan(const st_kv_cache& c, int64_t T, int32_t q_heads, int32_t R, int32_t max_q, int64_t max_len)
{
    const int64_t G = q_heads / c.kv_heads;
    AttendPlan p;
    p.prefill = max_q * G > kDecMaxCols;
    p.decode = !p.prefill || (R > 1 && G <= kDecMaxCols);
    p.dec = DecPlan{};
    if (p.decode) p.dec = dec_plan(c, T, q_heads, R, p.prefill ? int32_t(kDecMaxCols / G) : max_q, max_len, p.prefill);
    return p;
}

int64_t kv_attend_workspace(const st_kv_cache& c, int64_t T, int32_t q_heads, int32_t R, int32_t max_q, int64_t max_len)
{
    const AttendPlan p = attend_plan(c, T, q_heads, R, max_q, max_len);
    return p.dec.bytes + (p.prefill ? kv_prefill_workspace(c, T, q_heads, R, max_q, max_len) : 0);
}

cudaError_t launch_kv_attend(const AttendArgs& args, cudaStream_t s)
{
    const AttendPlan p = attend_plan(args.c, args.T, args.q_heads, args.R, args.max_q, args.max_len);
    AttendArgs a = args;
    if (p.prefill) {
        a.above_cols = p.decode ? kDecMaxCols : 0;
        a.workspace = static_cast<char*>(args.workspace) + p.dec.bytes;
        a.parts = args.T * args.q_heads;
        const cudaError_t e = launch_kv_prefill(a, s);
        if (e != cudaSuccess) return e;
        a.above_cols = 0;
        a.most_cols = kDecMaxCols;
        a.workspace = args.workspace;
    }
    a.parts = p.dec.parts;
    a.row_cols = p.dec.row_cols;
    return p.decode ? launch_kv_decode(a, p.dec, s) : cudaSuccess;
}

}  // namespace st
