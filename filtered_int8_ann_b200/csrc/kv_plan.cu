// Block tables and slot maps of a paged cache, from the rows' lengths.
//
// Which blocks are free follows from the tables: those that no stored token of
// any row uses. One pass over the used table entries marks them in a bitmap
// (and in a second one those met twice: a partly filled last block that
// others use too must not be written). Prefix sums over the rows (blocks
// needed, tokens added) and over the bitmap (free blocks) give every row its
// blocks: the free block of rank j goes to the row whose range of needed
// blocks holds j. Everything is whole numbers, so results are the same
// whatever the order of the atomics.
//
// A single cluster does all of that in one launch: the bitmaps are split over its
// CTAs' shared memory (2 x 64 KB in each of 8 CTAs for the largest pool of 4M
// blocks), the marks are distributed-shared-memory atomics, and the cluster barrier
// orders the steps. Small pools and tables take one CTA: no remote atomics and cheap barriers.
// The new tokens' slots (12 bytes each) are written there too, a warp per
// row, when the rows get few tokens each; prompts' are written by a second
// launch over the whole GPU, since the cluster's SMs alone store too slowly.
#include <cooperative_groups.h>

#include "decode.cuh"

namespace cg = cooperative_groups;

namespace st {

constexpr int kPlanCtas = 8;      // CTAs of the cluster for large calls
constexpr int kPlanBlock = 1024;
// Calls up to these sizes take one CTA.
constexpr int kPlanSmallRows = 1024;
constexpr int kPlanSmallBlocks = 131072;
constexpr int64_t kPlanSmallEntries = 32768;
constexpr int kPlanWarps = kPlanBlock / 32;

struct PlanShared {
    uint32_t part[32];
    unsigned long long part64[32];
    unsigned long long tokens;  // sum of add over this CTA's rows
    uint32_t need, free;        // blocks its rows need, free blocks in its part of the pool
    uint32_t failed, refused;   // CTA 0: rows not served, rows refused
};

// Inclusive scan of a 64-bit value per thread over the block.
__device__ __forceinline__ unsigned long long block_incl_scan64(unsigned long long v, unsigned long long* part,
                                                                unsigned long long& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long t = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += t;
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    if (warp == 0) {
        unsigned long long w = lane < kPlanWarps ? part[lane] : 0ull;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const unsigned long long t = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += t;
        }
        part[lane] = w;
    }
    __syncthreads();
    v += warp > 0 ? part[warp - 1] : 0ull;
    total = part[kPlanWarps - 1];
    __syncthreads();
    return v;
}

// CTAS: CTAs of the (only) cluster. all_slots: every token's slot is written
// here, else only those in the rows' partly filled blocks (whose sources only
// this kernel knows).
template <int CTAS>
__global__ void __launch_bounds__(kPlanBlock) kv_plan_kernel(PlanArgs a, int rows_per, int words_per, bool all_slots)
{
    extern __shared__ uint32_t smem[];
    __shared__ PlanShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int me = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // this CTA's part of the pool (bitmaps of words_per words) and of the rows
    uint32_t* used_bits = smem;
    uint32_t* twice_bits = smem + words_per;
    uint32_t* row_end = smem + 2 * words_per;       // [rows_per] blocks needed by rows up to this one, within the CTA
    uint32_t* row_need = row_end + rows_per;        // [rows_per] blocks this row needs; bit 31: its last block is replaced
    int32_t* row_tail = reinterpret_cast<int32_t*>(row_need + rows_per);  // [rows_per] that last block
    const int r0 = min(a.R, me * rows_per), r1 = min(a.R, r0 + rows_per);
    const int pages_per = words_per * 32;
    const int S = a.block_size;

    for (int i = tid; i < 2 * words_per; i += kPlanBlock) smem[i] = 0;
    if (tid == 0) sh.failed = sh.refused = 0;
    __syncthreads();
    cluster.sync();

    // 1. mark the blocks of the stored tokens, a warp per row; row_need holds the row's state meanwhile:
    // 0 in order, 1 refused, 2 no room in its table row
    for (int r = r0 + warp; r < r1; r += kPlanWarps) {
        const int64_t have = a.have[r], add = a.add[r], room = int64_t(a.max_blocks) * S;
        int state = have < 0 || add < 0 || have > room ? 1 : have + add > room ? 2 : 0;
        if (have >= 0 && have <= room) {
            const int n = int((have + S - 1) / S);
            const int32_t* row = a.table + int64_t(r) * a.max_blocks;
            bool bad = false;
            for (int c = lane; c < n; c += 32) {
                const int32_t p = row[c];
                if (p < 0 || p >= a.num_blocks) {
                    bad = true;
                    continue;
                }
                const int owner = p / pages_per, w = (p - owner * pages_per) >> 5;
                const uint32_t bit = 1u << (p & 31);
                const uint32_t old = atomicOr(cluster.map_shared_rank(used_bits, owner) + w, bit);
                if (old & bit) atomicOr(cluster.map_shared_rank(twice_bits, owner) + w, bit);
            }
            if (__any_sync(0xffffffffu, bad)) {
                state = 1;
                if (lane == 0) atomicOr(a.err, kDecErrTable);
            }
        }
        if (lane == 0) row_need[r - r0] = uint32_t(state);
    }
    __syncthreads();
    cluster.sync();

    // 2a. rows: blocks needed and tokens, with prefix sums inside the CTA
    unsigned long long tok_base = 0;
    uint32_t need_base = 0;
    for (int i0 = 0; i0 < rows_per; i0 += kPlanBlock) {
        const int r = r0 + i0 + tid;
        const bool mine = i0 + tid < rows_per && r < r1;
        uint32_t need = 0;
        int32_t tail = -1;
        unsigned long long tok = 0;
        if (mine) {
            const int state = int(row_need[r - r0]);
            const int have = a.have[r], add = a.add[r];
            tok = add > 0 ? (unsigned long long)(add) : 0ull;
            if (state == 0) {
                const int used = int((int64_t(have) + S - 1) / S);
                need = uint32_t((int64_t(have) + add + S - 1) / S) - uint32_t(used);
                if (have % S != 0 && add > 0) {
                    const int32_t p = a.table[int64_t(r) * a.max_blocks + used - 1];
                    const int owner = p / pages_per, w = (p - owner * pages_per) >> 5;
                    if (cluster.map_shared_rank(twice_bits, owner)[w] >> (p & 31) & 1u) {
                        tail = p;
                        ++need;
                    }
                }
            }
            if (state == 1) atomicAdd(&cluster.map_shared_rank(&sh, 0)->refused, 1u);
            // state in the top bits: not to be served whatever the pool holds
            row_need[r - r0] = need | (tail >= 0 ? 1u << 31 : 0u) | (state ? 1u << 30 : 0u) | (state == 1 ? 1u << 29 : 0u);
            row_tail[r - r0] = tail;
        }
        unsigned long long tok_total = 0;
        const unsigned long long tok_incl = block_incl_scan64(tok, sh.part64, tok_total);
        uint32_t need_total = 0;
        const uint32_t need_excl = block_excl_scan<kPlanBlock>(need, sh.part, need_total);
        if (mine) row_end[r - r0] = need_base + need_excl + need;
        // the row's token end within the CTA waits in row_start until the CTAs' bases are known
        if (mine) a.row_start[r + 1] = int32_t(min((unsigned long long)(0x7fffffff), tok_base + tok_incl));
        tok_base += tok_total;
        need_base += need_total;
    }
    // 2b. free blocks of this CTA's part, a run of words per thread
    const int per_thread = (words_per + kPlanBlock - 1) / kPlanBlock;
    const int w0 = min(words_per, tid * per_thread), w1 = min(words_per, w0 + per_thread);
    auto free_word = [&](int w) {
        const int64_t first = int64_t(me) * pages_per + int64_t(w) * 32;
        const int64_t left = int64_t(a.num_blocks) - first;
        if (left <= 0) return 0u;
        return ~used_bits[w] & (left >= 32 ? 0xffffffffu : (1u << left) - 1u);
    };
    uint32_t nfree = 0;
    for (int w = w0; w < w1; ++w) nfree += __popc(free_word(w));
    uint32_t free_total = 0;
    uint32_t rank = block_excl_scan<kPlanBlock>(nfree, sh.part, free_total);
    if (tid == 0) {
        sh.tokens = tok_base;
        sh.need = need_base;
        sh.free = free_total;
    }
    __syncthreads();
    cluster.sync();

    // 3. bases of the CTAs; token starts; which rows are served
    unsigned long long tok_before = 0, tok_all = 0;
    uint32_t need_before = 0, free_before = 0, free_all = 0;
    unsigned long long need_all = 0;
    uint32_t need_ends[CTAS];  // blocks needed by the rows of CTAs 0..c
#pragma unroll
    for (int c = 0; c < CTAS; ++c) {
        const PlanShared* o = cluster.map_shared_rank(&sh, c);
        if (c < me) {
            tok_before += o->tokens;
            need_before += o->need;
            free_before += o->free;
        }
        tok_all += o->tokens;
        need_all += o->need;
        free_all += o->free;
        need_ends[c] = uint32_t(need_all);
    }
    rank += free_before;
    for (int i = tid; i < r1 - r0; i += kPlanBlock) {
        const int r = r0 + i;
        const unsigned long long end = tok_before + (unsigned long long)(uint32_t(a.row_start[r + 1]));
        const uint32_t word = row_need[i], need = word & 0x1fffffffu;
        const int have = a.have[r], add = a.add[r];
        bool served = !(word >> 30 & 1u);
        if (served && need > 0 && uint32_t(need_before + row_end[i]) > free_all) served = false;
        if (served && add > 0 && end > (unsigned long long)(a.T)) served = false;
        a.lens[r] = served ? have + add : -1;
        if (!served && !(word >> 29 & 1u)) atomicAdd(&cluster.map_shared_rank(&sh, 0)->failed, 1u);
        if (!served) row_need[i] |= 1u << 30;
        a.row_start[r + 1] = int32_t(min(end, (unsigned long long)(a.T)));
        if (r == 0) a.row_start[0] = 0;
    }
    __syncthreads();
    cluster.sync();

    // 4. the free block of rank j goes to the row whose needed blocks hold j
    for (int w = w0; w < w1 && rank < need_all; ++w) {
        uint32_t bits = free_word(w);
        while (bits && rank < need_all) {
            const int b = __ffs(bits) - 1;
            bits &= bits - 1;
            const uint32_t j = rank++;
            int c = 0;
#pragma unroll
            for (int i = 0; i < CTAS - 1; ++i) c += need_ends[i] <= j;
            uint32_t before = 0;
#pragma unroll
            for (int i = 0; i < CTAS - 1; ++i)
                if (i < c) before = need_ends[i];
            const uint32_t* ends = cluster.map_shared_rank(row_end, c);
            int lo = 0, hi = min(a.R, (c + 1) * rows_per) - c * rows_per - 1;  // first row whose end is above j
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (before + ends[mid] > j) hi = mid;
                else lo = mid + 1;
            }
            const int r = c * rows_per + lo;
            const uint32_t word = cluster.map_shared_rank(row_need, c)[lo];
            if (word >> 30 & 1u) continue;  // not served
            const uint32_t need = word & 0x1fffffffu;
            const int used = int((int64_t(a.have[r]) + S - 1) / S) - int(word >> 31);
            a.table[int64_t(r) * a.max_blocks + used + int(j - (before + ends[lo] - need))] =
                int32_t(int64_t(me) * pages_per + int64_t(w) * 32 + b);
        }
    }
    __syncthreads();
    cluster.sync();

    // 5. slots, a warp per row
    for (int r = r0 + warp; r < r1; r += kPlanWarps) {
        const int64_t start = __ldcg(a.row_start + r), end = __ldcg(a.row_start + r + 1);
        const bool served = !(row_need[r - r0] >> 30 & 1u);
        const int have = a.have[r], into = have % S;
        const int32_t tail = row_tail[r - r0];
        const int64_t n = !served || all_slots ? end - start : into ? min(end - start, int64_t(S - into)) : 0;
        const int32_t* row = a.table + int64_t(r) * a.max_blocks;
        for (int64_t i = lane; i < n; i += 32) {
            int64_t slot = -1;
            int32_t src = -1;
            if (served) {
                const int p = have + int(i), c = p / S;
                src = __ldcg(row + c);
                slot = int64_t(src) * S + (p - c * S);
                if (c == have / S && tail >= 0) src = tail;
            }
            a.slots[start + i] = slot;
            a.sources[start + i] = src;
        }
    }
    if (all_slots)  // behind the last row's tokens
        for (int64_t t = int64_t(min(tok_all, (unsigned long long)(a.T))) + me * kPlanBlock + tid; t < a.T; t += CTAS * kPlanBlock) {
            a.slots[t] = -1;
            a.sources[t] = -1;
        }
    if (me == 0 && tid == 0) {
        a.report[0] = int32_t(min(need_all, 0x7fffffffull));
        a.report[1] = int32_t(free_all);
        a.report[2] = int32_t(sh.failed);
        a.report[3] = int32_t(sh.refused);
    }
    cluster.sync();  // the CTAs' shared memory stays until all are done with it
}

// The slots of rows that get many tokens: each warp walks a stretch of tokens,
// its lanes holding the ends of the next 32 rows.
constexpr int kSlotBlock = 256;
constexpr int kSlotStretch = 256;  // tokens per warp

__global__ void __launch_bounds__(kSlotBlock) kv_slots_kernel(PlanArgs a)
{
    dep_enter();
    const int lane = threadIdx.x & 31, S = a.block_size;
    const int64_t t0 = (int64_t(blockIdx.x) * (kSlotBlock / 32) + (threadIdx.x >> 5)) * kSlotStretch;
    const int64_t t1 = min(a.T, t0 + kSlotStretch);
    if (t0 >= t1) return;
    int lo = 0, hi = a.R;  // first row that ends behind t0 (R: none)
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.row_start[mid + 1] > t0) hi = mid;
        else lo = mid + 1;
    }
    constexpr int64_t kNever = int64_t(1) << 40;
    int base = lo;  // lane i: the end of row base + i
    int64_t end = base + lane < a.R ? int64_t(a.row_start[base + lane + 1]) : kNever;
    for (int64_t t = t0 + lane; t - lane < t1; t += 32) {
        int row = 0;
        bool found = false;
        while (true) {  // the first row that ends behind t
            int pos = 0;
#pragma unroll
            for (int step = 16; step > 0; step >>= 1) {
                const int64_t e = __shfl_sync(0xffffffffu, end, pos + step - 1);
                if (e <= t) pos += step;
            }
            const int64_t e = __shfl_sync(0xffffffffu, end, pos);
            if (!found && e > t) {
                row = base + pos;
                found = true;
            }
            if (__all_sync(0xffffffffu, found)) break;
            base += 32;
            end = base + lane < a.R ? int64_t(a.row_start[base + lane + 1]) : kNever;
        }
        const int last_row = __shfl_sync(0xffffffffu, row, 31);
        if (t < t1) {
            int64_t slot = -1;
            int32_t src = -1;
            bool mine = true;
            if (row < a.R && a.lens[row] >= 0) {
                const int have = a.have[row];
                const int p = have + int(t - a.row_start[row]), c = p / S;
                mine = have % S == 0 || c != have / S;
                if (mine) {
                    src = a.table[int64_t(row) * a.max_blocks + c];
                    slot = int64_t(src) * S + (p - c * S);
                }
            }
            if (mine) {
                a.slots[t] = slot;
                a.sources[t] = src;
            }
        }
        if (last_row >= base + 16 && last_row < a.R) {  // keep the window ahead of the walk
            base = last_row;
            end = base + lane < a.R ? int64_t(a.row_start[base + lane + 1]) : kNever;
        }
    }
}

template <int CTAS>
static cudaError_t launch_plan(const PlanArgs& a, bool all_slots, cudaStream_t s)
{
    const int rows_per = (a.R + CTAS - 1) / CTAS;
    const int words_per = ((a.num_blocks + 31) / 32 + CTAS - 1) / CTAS;
    // the largest: 2 x 16384 words and 3 x 4096 rows
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kv_plan_kernel<CTAS>),
                                     (2 * (ST_KV_MAX_BLOCKS / 32 / kPlanCtas) + 3 * (ST_KV_MAX_ROWS / kPlanCtas)) * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CTAS);
    cfg.blockDim = dim3(kPlanBlock);
    cfg.dynamicSmemBytes = size_t(2 * words_per + 3 * rows_per) * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {CTAS, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_plan_kernel<CTAS>, a, rows_per, words_per, all_slots);
}

cudaError_t launch_kv_plan(const PlanArgs& a, cudaStream_t s)
{
    const bool all_slots = a.T <= 4 * int64_t(a.R) + 1024;
    const bool small = a.R <= kPlanSmallRows && a.num_blocks <= kPlanSmallBlocks &&
                       int64_t(a.R) * a.max_blocks <= kPlanSmallEntries;
    cudaError_t e = small ? launch_plan<1>(a, all_slots, s) : launch_plan<kPlanCtas>(a, all_slots, s);
    if (e != cudaSuccess || all_slots) return e;
    const int64_t per_cta = int64_t(kSlotBlock / 32) * kSlotStretch;
    return launch_dep(kv_slots_kernel, dim3(unsigned((a.T + per_cta - 1) / per_cta)), dim3(kSlotBlock), 0, s, a);
}

}  // namespace st
