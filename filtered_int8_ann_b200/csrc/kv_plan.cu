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
// The new tokens' slots (12 bytes each) are written there too, eight lanes per
// row, when the rows get few tokens each; prompts' are written by a second
// launch over the whole GPU, since the cluster's SMs alone store too slowly.
//
// Bound by latency: a dozen steps that wait for one another, each a barrier and one or two loads; the bytes (a few
// hundred KB at most) take under 1 us. 64 rows of 2000 tokens get one more in 8.2 us on the device, 1024 prompts of up to 1000
// tokens their slots in 20 us (two launches).
#include <cooperative_groups.h>

#include "decode.cuh"

namespace cg = cooperative_groups;

namespace st {

constexpr int kPlanCtas = 8;      // CTAs of the cluster for large calls
constexpr int kPlanBlock = 1024;
// Calls up to these sizes take one CTA (64 rows of 2000 tokens: 8.2 us, a cluster 15.7), larger ones the cluster (1024
// rows: 20 us, one CTA 33).
constexpr int kPlanSmallRows = 256;
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
    const int me = CTAS > 1 ? int(cluster.block_rank()) : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto sync_all = [&]() {
        if (CTAS > 1) cluster.sync();
        else __syncthreads();
    };
    auto of = [&](auto* p, int rank) { return CTAS > 1 ? cluster.map_shared_rank(p, rank) : p; };
    // this CTA's part of the pool (bitmaps of words_per words) and of the rows
    uint32_t* used_bits = smem;
    uint32_t* twice_bits = smem + words_per;        // later: free blocks before each word
    uint32_t* row_end = smem + 2 * words_per;       // [rows_per] blocks needed by rows up to this one, within the CTA
    uint32_t* row_need = row_end + rows_per;        // [rows_per] blocks this row needs, and flags
    int32_t* row_tail = reinterpret_cast<int32_t*>(row_need + rows_per);  // [rows_per] last block; later -1 if it stays
    int32_t* row_have = row_tail + rows_per;
    int32_t* row_tok = row_have + rows_per;         // [rows_per] end of the row's tokens
    constexpr uint32_t kUnserved = 1u << 30, kRefused = 1u << 29, kNeed = kRefused - 1;
    const int r0 = min(a.R, me * rows_per), r1 = min(a.R, r0 + rows_per), rows = r1 - r0;
    const int pages_per = words_per * 32, width = a.max_blocks;
    const int S = a.block_size, shift = 31 - __clz(S);
    const int64_t room = int64_t(width) << shift;

    for (int i = tid; i < 2 * words_per; i += kPlanBlock) smem[i] = 0;
    if (tid == 0) sh.failed = sh.refused = 0;
    for (int i = tid; i < rows; i += kPlanBlock) {
        const int64_t have = a.have[r0 + i], add = a.add[r0 + i];
        row_have[i] = int32_t(have);
        row_need[i] = have < 0 || add < 0 || have > room ? kUnserved | kRefused : have + add > room ? kUnserved : 0u;
        row_tail[i] = -1;
    }
    sync_all();

    // 1. mark the blocks of the stored tokens: eight lanes per row, a few entries each at a time
    for (int i0 = warp * 4; i0 < rows; i0 += kPlanWarps * 4) {
        const int i = i0 + (lane >> 3);
        const int64_t have = i < rows ? row_have[i] : 0;
        const int n = have > 0 && have <= room ? int((have + S - 1) >> shift) : 0;
        const int32_t* row = a.table + int64_t(r0 + i) * width;
        bool bad = false;
        for (int c0 = lane & 7; c0 < n; c0 += 32) {
            int32_t p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) p[u] = c0 + 8 * u < n ? row[c0 + 8 * u] : 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int c = c0 + 8 * u;
                if (c >= n) continue;
                if (p[u] < 0 || p[u] >= a.num_blocks) {
                    bad = true;
                    continue;
                }
                const int owner = CTAS > 1 ? p[u] / pages_per : 0, w = (p[u] - owner * pages_per) >> 5;
                const uint32_t bit = 1u << (p[u] & 31);
                const uint32_t old = atomicOr(of(used_bits, owner) + w, bit);
                if (old & bit) atomicOr(of(twice_bits, owner) + w, bit);
                if (c == n - 1) row_tail[i] = p[u];
            }
        }
        if (bad) {
            atomicOr(&row_need[i], kUnserved | kRefused);
            atomicOr(a.err, kDecErrTable);
        }
    }
    sync_all();

    // 2a. rows: blocks needed and tokens, with prefix sums inside the CTA
    unsigned long long tok_base = 0;
    uint32_t need_base = 0;
    for (int i0 = 0; i0 < rows_per; i0 += kPlanBlock) {
        const int i = i0 + tid;
        const bool mine = i < rows;
        uint32_t need = 0;
        unsigned long long tok = 0;
        if (mine) {
            const uint32_t state = row_need[i];
            const int have = row_have[i], add = a.add[r0 + i];
            int32_t tail = -1;
            tok = add > 0 ? (unsigned long long)(add) : 0ull;
            if (!(state & kUnserved)) {
                need = uint32_t(((int64_t(have) + add + S - 1) >> shift) - ((int64_t(have) + S - 1) >> shift));
                if ((have & (S - 1)) != 0 && add > 0) {
                    const int32_t p = row_tail[i];
                    const int owner = CTAS > 1 ? p / pages_per : 0, w = (p - owner * pages_per) >> 5;
                    if (of(twice_bits, owner)[w] >> (p & 31) & 1u) {  // the last block is replaced
                        tail = p;
                        ++need;
                    }
                }
            }
            if (state & kRefused) atomicAdd(&of(&sh, 0)->refused, 1u);
            row_need[i] = need | state;
            row_tail[i] = tail;
        }
        unsigned long long tok_total = 0;
        const unsigned long long tok_incl = block_incl_scan64(tok, sh.part64, tok_total);
        uint32_t need_total = 0;
        const uint32_t need_excl = block_excl_scan<kPlanBlock>(need, sh.part, need_total);
        if (mine) {
            row_end[i] = need_base + need_excl + need;
            row_tok[i] = int32_t(min((unsigned long long)(0x7fffffff), tok_base + tok_incl));
        }
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
    sync_all();

    // 3. bases of the CTAs; token starts; which rows are served; free blocks before each word
    unsigned long long tok_before = 0, tok_all = 0, need_all = 0;
    uint32_t need_before = 0, free_before = 0, free_all = 0;
    uint32_t need_ends[CTAS];  // blocks needed by the rows of CTAs 0..c
#pragma unroll
    for (int c = 0; c < CTAS; ++c) {
        const PlanShared* o = of(&sh, c);
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
    for (int w = w0; w < w1; ++w) {
        twice_bits[w] = rank;
        rank += __popc(free_word(w));
    }
    if (me == 0 && tid == 0) a.row_start[0] = 0;
    for (int i = tid; i < rows; i += kPlanBlock) {
        const unsigned long long end = tok_before + (unsigned long long)(uint32_t(row_tok[i]));
        const uint32_t word = row_need[i];
        const int have = row_have[i], add = a.add[r0 + i];
        bool served = !(word & kUnserved);
        if (served && (word & kNeed) > 0 && need_before + row_end[i] > free_all) served = false;
        if (served && add > 0 && end > (unsigned long long)(a.T)) served = false;
        if (!served && !(word & kRefused)) atomicAdd(&of(&sh, 0)->failed, 1u);
        if (!served) row_need[i] = word | kUnserved;
        const int tok = int(min(end, (unsigned long long)(a.T)));
        row_tok[i] = tok;
        a.row_start[r0 + i + 1] = tok;
        a.lens[r0 + i] = served ? have + add : -1;
    }
    sync_all();

    // 4. the free block of rank j goes to the row whose needed blocks hold j: a warp per word, a lane per block
    for (int w = warp; w < words_per; w += kPlanWarps) {
        const uint32_t bits = free_word(w), j = twice_bits[w] + __popc(bits & lanemask_lt());
        if (twice_bits[w] >= need_all) break;
        if (!(bits >> lane & 1u) || j >= need_all) continue;
        int c = 0;
        uint32_t before = 0;
#pragma unroll
        for (int i = 0; i < CTAS - 1; ++i)
            if (need_ends[i] <= j) {
                c = i + 1;
                before = need_ends[i];
            }
        const uint32_t* ends = of(row_end, c);
        int lo = 0, hi = min(a.R, (c + 1) * rows_per) - c * rows_per - 1;  // first row whose end is above j
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (before + ends[mid] > j) hi = mid;
            else lo = mid + 1;
        }
        const uint32_t word = of(row_need, c)[lo];
        if (word & kUnserved) continue;
        const int used = int((int64_t(of(row_have, c)[lo]) + S - 1) >> shift) - (of(row_tail, c)[lo] >= 0);
        a.table[int64_t(c * rows_per + lo) * width + used + int(j - (before + ends[lo] - (word & kNeed)))] =
            int32_t(int64_t(me) * pages_per + int64_t(w) * 32 + lane);
    }
    sync_all();

    // 5. slots: rows of a few tokens have eight lanes each
    const int per_row = all_slots ? 8 : 32;
    for (int i0 = warp * (32 / per_row); i0 < rows; i0 += kPlanWarps * (32 / per_row)) {
        const int i = i0 + lane / per_row;
        if (i >= rows) continue;
        const int start = i > 0 ? row_tok[i - 1] : int(min(tok_before, (unsigned long long)(a.T))), end = row_tok[i];
        const bool served = !(row_need[i] & kUnserved);
        const int have = row_have[i], into = have & (S - 1);
        const int32_t tail = row_tail[i];
        const int n = !served || all_slots ? end - start : into ? min(end - start, S - into) : 0;
        const int32_t* row = a.table + int64_t(r0 + i) * width;
        for (int k = lane % per_row; k < n; k += per_row) {
            int64_t slot = -1;
            int32_t src = -1;
            if (served) {
                const int p = have + k, c = p >> shift;
                src = __ldcg(row + c);
                slot = (int64_t(src) << shift) + (p & (S - 1));
                if (c == have >> shift && tail >= 0) src = tail;
            }
            a.slots[start + k] = slot;
            a.sources[start + k] = src;
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
    if (CTAS > 1) cluster.sync();  // the CTAs' shared memory stays until all are done with it
}

// The slots of rows that get many tokens: each warp walks a stretch of tokens,
// its lanes holding the ends of the next 32 rows.
constexpr int kSlotBlock = 256;
constexpr int kSlotStretch = 64;   // tokens per warp: more of them wait longer for each other than for the row search

__global__ void __launch_bounds__(kSlotBlock) kv_slots_kernel(PlanArgs a)
{
    dep_enter();
    const int lane = threadIdx.x & 31, S = a.block_size, shift = 31 - __clz(S);
    const int64_t t0 = (int64_t(blockIdx.x) * (kSlotBlock / 32) + (threadIdx.x >> 5)) * kSlotStretch;
    const int64_t t1 = min(a.T, t0 + kSlotStretch);
    if (t0 >= t1) return;
    // first row that ends behind t0 (R: none), among lo .. lo + n: 32 rows are looked at a time, since each look waits for
    // memory
    int lo = 0;
    for (int n = a.R; n > 0;) {
        const int step = (n + 31) / 32, at = lo + (lane + 1) * step - 1;
        const int before = __popc(__ballot_sync(0xffffffffu, at < lo + n && a.row_start[at + 1] <= t0));
        n = min(step - 1, n - before * step);
        lo += before * step;
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
                const int p = have + int(t - a.row_start[row]), c = p >> shift;
                mine = (have & (S - 1)) == 0 || c != have >> shift;
                if (mine) {
                    src = a.table[int64_t(row) * a.max_blocks + c];
                    slot = (int64_t(src) << shift) + (p & (S - 1));
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
    // the largest: 2 x 16384 words and 5 x 4096 rows
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kv_plan_kernel<CTAS>),
                                     (2 * (ST_KV_MAX_BLOCKS / 32 / kPlanCtas) + 5 * (ST_KV_MAX_ROWS / kPlanCtas)) * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CTAS);
    cfg.blockDim = dim3(kPlanBlock);
    cfg.dynamicSmemBytes = size_t(2 * words_per + 5 * rows_per) * 4;
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
    // Few tokens per row need no second launch (64 rows of one token: 8.2 us, with it 13.1); many do (1024 rows of 1000:
    // 20 us, without it 48). Few rows of many tokens would need it sooner than this rule gives it (one row of 1028 tokens 28 us,
    // of 1029 7).
    const bool all_slots = a.T <= 4 * int64_t(a.R) + 1024;
    const bool small = a.R <= kPlanSmallRows && a.num_blocks <= kPlanSmallBlocks &&
                       int64_t(a.R) * a.max_blocks <= kPlanSmallEntries;
    cudaError_t e = small ? launch_plan<1>(a, all_slots, s) : launch_plan<kPlanCtas>(a, all_slots, s);
    if (e != cudaSuccess || all_slots) return e;
    const int64_t per_cta = int64_t(kSlotBlock / 32) * kSlotStretch;
    return launch_dep(kv_slots_kernel, dim3(unsigned((a.T + per_cta - 1) / per_cta)), dim3(kSlotBlock), 0, s, a);
}

}  // namespace st
