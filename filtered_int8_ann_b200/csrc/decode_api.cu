// Host side of the decode operators declared in include/st.h: argument checks
// and the device's decode error word.
#include <cmath>
#include <mutex>
#include <new>
#include <numeric>

#include "decode.cuh"

namespace st {

// Kernels record an index outside its array here; st_decode_check reads and clears it.
static __device__ uint32_t g_decode_err;

cudaError_t decode_error_address(uint32_t** word)
{
    constexpr int kDevices = 64;
    static std::mutex mu;
    static uint32_t* known[kDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < kDevices && known[dev]) {
        *word = known[dev];
        return cudaSuccess;
    }
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_decode_err);
    if (e != cudaSuccess) return e;
    *word = static_cast<uint32_t*>(p);
    if (dev < kDevices) known[dev] = *word;
    return cudaSuccess;
}

cudaError_t decode_error_word(uint32_t* value)
{
    cudaError_t e = cudaMemcpyFromSymbol(value, g_decode_err, sizeof(uint32_t));
    if (e == cudaSuccess && *value) {
        const uint32_t z = 0;
        e = cudaMemcpyToSymbol(g_decode_err, &z, sizeof(uint32_t));
    }
    return e;
}

}  // namespace st

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int64_t kLimit31 = int64_t(1) << 31;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Device (or managed) memory that the current device `device` holds, aligned to `a`.
bool on_device(const void* p, int device, size_t a)
{
    if (p == nullptr || !aligned(p, a)) return false;
    cudaPointerAttributes attr;
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (attr.type == cudaMemoryTypeManaged) return true;
    return attr.type == cudaMemoryTypeDevice && attr.device == device;
}

st_status to_status(cudaError_t e)
{
    if (e == cudaSuccess) return ST_OK;
    cudaGetLastError();
    if (e == cudaErrorInvalidConfiguration) return ST_ERR_UNSUPPORTED;  // more CTAs than a grid holds
    return e == cudaErrorMemoryAllocation ? ST_ERR_OOM : ST_ERR_CUDA;
}

// Do the byte ranges [p, p + n) and [q, q + m) share a byte?
bool overlap(const void* p, int64_t n, const void* q, int64_t m)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && a < b + uintptr_t(m) && b < a + uintptr_t(n);
}

// n0 x n1 vectors of `bytes` bytes, the strides between them in bytes (not negative).
struct Vectors {
    const void* p;
    int64_t n0, s0, n1, s1, bytes;
    __int128 at() const { return reinterpret_cast<uintptr_t>(p); }
    __int128 inner() const { return (n1 > 1 ? __int128(n1 - 1) * s1 : 0) + bytes; }  // what the vectors of one n0 span
    __int128 span() const { return (n0 > 1 ? __int128(n0 - 1) * s0 : 0) + inner(); }
    Vectors swapped() const { return {p, n1, s1, n0, s0, bytes}; }
};
Vectors dense(const void* p, int64_t bytes) { return {p, 1, 0, 1, 0, bytes}; }

// The vectors do not share a byte among themselves: one dimension inside the other.
bool separate(const Vectors& v)
{
    const Vectors w = v.swapped();
    return (v.n0 <= 1 || v.s0 >= v.bytes) && (v.n1 <= 1 || v.s1 >= v.bytes) &&
           (v.n0 <= 1 || v.n1 <= 1 || v.s0 >= v.inner() || w.s0 >= w.inner());
}

// Do a and b lie in different bytes of each turn of length `turn`?
bool apart_in_turns(const Vectors& a, __int128 na, const Vectors& b, __int128 nb, __int128 turn)
{
    const __int128 d = ((b.at() - a.at()) % turn + turn) % turn;
    return d >= na && d + nb <= turn;
}

// a and b share no byte: their spans do not, or they are interleaved with equal outer strides (slices of one
// projection), or with strides that are multiples of a length in which both have their place (every other head).
bool apart(const Vectors& a, const Vectors& b)
{
    if (a.n0 <= 1 && a.n1 <= 1 && b.n0 <= 1 && b.n1 <= 1) return !overlap(a.p, a.bytes, b.p, b.bytes);
    if (a.span() <= 0 || b.span() <= 0 || a.at() >= b.at() + b.span() || b.at() >= a.at() + a.span()) return true;
    const auto outer = [](const Vectors& x, const Vectors& y) {
        return x.n0 > 1 && y.n0 > 1 && x.s0 == y.s0 && x.s0 > 0 && x.inner() <= x.s0 && y.inner() <= y.s0 &&
               apart_in_turns(x, x.inner(), y, y.inner(), x.s0);
    };
    if (outer(a, b) || outer(a.swapped(), b.swapped())) return true;
    int64_t g = 0;
    for (const Vectors& v : {a, b}) {
        if (v.n0 > 1) g = std::gcd(g, v.s0);
        if (v.n1 > 1) g = std::gcd(g, v.s1);
    }
    return g > 0 && apart_in_turns(a, a.bytes, b, b.bytes, g);
}

// The same vectors in the same places.
bool same(const Vectors& a, const Vectors& b)
{
    return a.p == b.p && a.n0 == b.n0 && a.n1 == b.n1 && a.bytes == b.bytes && (a.n0 <= 1 || a.s0 == b.s0) &&
           (a.n1 <= 1 || a.s1 == b.s1);
}

// No exception leaves the library: what the host side's containers and locks may throw becomes a status.
template <typename F>
st_status guarded(F&& f) noexcept
{
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return ST_ERR_OOM;
    } catch (...) {
        return ST_ERR_CUDA;
    }
}

bool block_size_ok(int32_t s) { return s == 16 || s == 32 || s == 64 || s == 128; }

// Sizes of a cache: INVALID_ARG for what no cache has, UNSUPPORTED for what this one cannot be.
st_status cache_sizes(const st_kv_cache* c)
{
    if (c == nullptr || c->num_blocks < 1 || c->kv_heads < 1 || c->block_size < 1 || c->head_dim < 1)
        return ST_ERR_INVALID_ARG;
    if (c->num_blocks > ST_KV_MAX_BLOCKS || c->kv_heads > 1024 || !block_size_ok(c->block_size) ||
        (c->head_dim != 64 && c->head_dim != 128))
        return ST_ERR_UNSUPPORTED;
    return ST_OK;
}

int64_t code_bytes(const st_kv_cache* c) { return int64_t(c->num_blocks) * c->kv_heads * c->block_size * c->head_dim; }
int64_t scale_bytes(const st_kv_cache* c) { return int64_t(c->num_blocks) * c->kv_heads * 4; }

bool cache_arrays(const st_kv_cache* c, int dev)
{
    return on_device(c->k, dev, 16) && on_device(c->v, dev, 16) && on_device(c->k_scale, dev, 4) &&
           on_device(c->v_scale, dev, 4);
}

// Strides (elements of 16 bits) of an array of 16-byte vectors.
bool strides_ok(int64_t token, int64_t head)
{
    constexpr int64_t far = int64_t(1) << 56;
    return token >= 0 && head >= 0 && token % 8 == 0 && head % 8 == 0 && token < far && head < far;
}

st_status attend_sizes(const st_kv_cache* c, int64_t T, int32_t q_heads, int32_t R, int32_t max_q, int64_t max_len)
{
    const st_status s = cache_sizes(c);
    if (s == ST_ERR_INVALID_ARG) return s;
    if (T < 0 || q_heads < 1 || R < 1 || max_q < 1 || max_q > (1 << 20) || max_len < 1) return ST_ERR_INVALID_ARG;
    if (q_heads % c->kv_heads != 0) return ST_ERR_INVALID_ARG;
    if (s != ST_OK) return s;
    if (R > ST_KV_MAX_ROWS || T >= kLimit31 || max_len >= kLimit31 || q_heads > 65535) return ST_ERR_UNSUPPORTED;
    return ST_OK;
}

st_status select_sizes(int32_t B, int32_t K, int32_t V, int32_t keep)
{
    if (B < 1 || K < 1 || V < 1 || keep < 1) return ST_ERR_INVALID_ARG;
    if (B > ST_MAX_B || K > ST_BEAM_MAX_BEAMS || V > ST_BEAM_MAX_VOCAB || keep > ST_BEAM_MAX_KEEP)
        return ST_ERR_UNSUPPORTED;
    return ST_OK;
}

}  // namespace

extern "C" {

st_status st_kv_plan(int32_t* table, const int32_t* have, const int32_t* add, int32_t R, int32_t max_blocks,
                     int32_t num_blocks, int32_t block_size, int64_t T, int64_t* slots, int32_t* sources,
                     int32_t* row_start, int32_t* lens, int32_t* report, cudaStream_t stream)
{
    return guarded([&]() -> st_status {
        if (R < 1 || max_blocks < 1 || num_blocks < 1 || T < 0 || !block_size_ok(block_size)) return ST_ERR_INVALID_ARG;
        if (R > ST_KV_MAX_ROWS || num_blocks > ST_KV_MAX_BLOCKS || int64_t(R) * max_blocks >= kLimit31 || T >= kLimit31 - 1 ||
            int64_t(max_blocks) * block_size >= kLimit31)
            return ST_ERR_UNSUPPORTED;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return ST_ERR_CUDA;
        if (!on_device(table, dev, 4) || !on_device(have, dev, 4) || !on_device(add, dev, 4) ||
            !on_device(row_start, dev, 4) || !on_device(lens, dev, 4) || !on_device(report, dev, 4))
            return ST_ERR_INVALID_ARG;
        if (T > 0 && (!on_device(slots, dev, 8) || !on_device(sources, dev, 4))) return ST_ERR_INVALID_ARG;
        // a launch of two kernels reads the inputs while it writes the outputs
        const struct {
            const void* p;
            int64_t bytes;
        } part[] = {{table, int64_t(R) * max_blocks * 4}, {slots, T * 8}, {sources, T * 4}, {row_start, (int64_t(R) + 1) * 4},
                    {lens, int64_t(R) * 4}, {report, 16}, {have, int64_t(R) * 4}, {add, int64_t(R) * 4}};
        for (int i = 0; i < 6; ++i)
            for (int j = i + 1; j < 8; ++j)
                if (overlap(part[i].p, part[i].bytes, part[j].p, part[j].bytes)) return ST_ERR_INVALID_ARG;
        st::PlanArgs a{table, have, add, R, max_blocks, num_blocks, block_size, T, slots, sources, row_start, lens, report, nullptr};
        cudaError_t e = st::decode_error_address(&a.err);
        if (e == cudaSuccess) e = st::launch_kv_plan(a, stream);
        return to_status(e);
    });
}

st_status st_kv_append(const st_kv_cache* cache, const void* k, const void* v, st_dtype dtype, int64_t T,
                       int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                       int64_t v_head_stride, const int64_t* slots, const int32_t* sources,
                       cudaStream_t stream)
{
    return guarded([&]() -> st_status {
        if (cache_sizes(cache) == ST_ERR_INVALID_ARG || T < 0 || (dtype != ST_BF16 && dtype != ST_F16) ||
            !strides_ok(k_token_stride, k_head_stride) || !strides_ok(v_token_stride, v_head_stride))
            return ST_ERR_INVALID_ARG;
        if (cache_sizes(cache) != ST_OK || T >= kLimit31) return ST_ERR_UNSUPPORTED;
        if (T == 0) return ST_OK;
        // the cache's arrays are written while the others are read
        const int64_t row = cache->head_dim * 2;
        const Vectors part[] = {dense(cache->k, code_bytes(cache)), dense(cache->v, code_bytes(cache)), dense(cache->k_scale, scale_bytes(cache)),
                                dense(cache->v_scale, scale_bytes(cache)), {k, T, k_token_stride * 2, cache->kv_heads, k_head_stride * 2, row},
                                {v, T, v_token_stride * 2, cache->kv_heads, v_head_stride * 2, row}, dense(slots, T * 8),
                                dense(sources, sources ? T * 4 : 0)};
        for (int i = 0; i < 4; ++i)
            for (int j = i + 1; j < 8; ++j)
                if (!apart(part[i], part[j])) return ST_ERR_INVALID_ARG;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return ST_ERR_CUDA;
        if (!cache_arrays(cache, dev) || !on_device(k, dev, 16) || !on_device(v, dev, 16) || !on_device(slots, dev, 8) ||
            (sources != nullptr && !on_device(sources, dev, 4)))
            return ST_ERR_INVALID_ARG;
        st::AppendArgs a{*cache, k, v, dtype, T, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots, sources, nullptr};
        cudaError_t e = st::decode_error_address(&a.err);
        if (e == cudaSuccess) e = st::launch_kv_append(a, stream);
        return to_status(e);
    });
}

st_status st_kv_attend_workspace(const st_kv_cache* cache, int64_t T, int32_t q_heads, int32_t R, int32_t max_q,
                                 int64_t max_len, int64_t* bytes)
{
    if (bytes == nullptr) return ST_ERR_INVALID_ARG;
    *bytes = 0;
    const st_status s = attend_sizes(cache, T, q_heads, R, max_q, max_len);
    if (s != ST_OK) return s;
    const int64_t need = st::kv_attend_workspace(*cache, T, q_heads, R, max_q, max_len);
    if (need > st::kAttendMaxBytes) return ST_ERR_UNSUPPORTED;
    *bytes = need;
    return ST_OK;
}

st_status st_kv_attend(const st_kv_cache* cache, const void* q, st_dtype dtype, int64_t T, int32_t q_heads,
                       int64_t q_token_stride, int64_t q_head_stride, const int32_t* table, int32_t max_blocks,
                       const int32_t* row_start, const int32_t* lens, int32_t R, int32_t max_q, int64_t max_len,
                       float scale, int32_t causal, void* out, int64_t out_token_stride,
                       int64_t out_head_stride, void* workspace, int64_t workspace_bytes, cudaStream_t stream)
{
    return guarded([&]() -> st_status {
        const st_status s = attend_sizes(cache, T, q_heads, R, max_q, max_len);
        if (s == ST_ERR_INVALID_ARG) return s;
        if ((dtype != ST_BF16 && dtype != ST_F16) || max_blocks < 1 || !std::isfinite(scale * kLog2e) ||
            !strides_ok(q_token_stride, q_head_stride) || !strides_ok(out_token_stride, out_head_stride) ||
            max_len > int64_t(max_blocks) * cache->block_size)
            return ST_ERR_INVALID_ARG;
        if (s != ST_OK) return s;
        if (int64_t(R) * max_blocks >= kLimit31) return ST_ERR_UNSUPPORTED;
        if (T == 0) return ST_OK;
        const int64_t need = st::kv_attend_workspace(*cache, T, q_heads, R, max_q, max_len);
        if (need > st::kAttendMaxBytes) return ST_ERR_UNSUPPORTED;
        // out and the workspace are written while the rest is read; out may be q itself
        const Vectors vq{q, T, q_token_stride * 2, q_heads, q_head_stride * 2, cache->head_dim * 2};
        const Vectors vo{out, T, out_token_stride * 2, q_heads, out_head_stride * 2, cache->head_dim * 2}, vw = dense(workspace, need);
        if (!separate(vo) || !(same(vo, vq) || apart(vo, vq)) || !apart(vw, vq) || !apart(vw, vo)) return ST_ERR_INVALID_ARG;
        for (const Vectors& x : {dense(cache->k, code_bytes(cache)), dense(cache->v, code_bytes(cache)), dense(cache->k_scale, scale_bytes(cache)),
                                 dense(cache->v_scale, scale_bytes(cache)), dense(table, int64_t(R) * max_blocks * 4),
                                 dense(row_start, (int64_t(R) + 1) * 4), dense(lens, int64_t(R) * 4)})
            if (!apart(vo, x) || !apart(vw, x)) return ST_ERR_INVALID_ARG;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return ST_ERR_CUDA;
        if (!cache_arrays(cache, dev) || !on_device(q, dev, 16) || !on_device(out, dev, 16) || !on_device(table, dev, 4) ||
            !on_device(row_start, dev, 4) || !on_device(lens, dev, 4))
            return ST_ERR_INVALID_ARG;
        if (need > 0 && (workspace_bytes < need || !on_device(workspace, dev, 16))) return ST_ERR_INVALID_ARG;
        st::AttendArgs a{*cache, q, dtype, T, q_heads, q_token_stride, q_head_stride, table, max_blocks, row_start, lens,
                         R, max_q, max_len, scale * kLog2e, causal, out, out_token_stride, out_head_stride,
                         workspace, nullptr};
        cudaError_t e = st::decode_error_address(&a.err);
        if (e == cudaSuccess) e = st::launch_kv_attend(a, stream);
        return to_status(e);
    });
}

st_status st_beam_select_workspace(int32_t B, int32_t K, int32_t V, int32_t keep, int64_t* bytes)
{
    if (bytes == nullptr) return ST_ERR_INVALID_ARG;
    *bytes = 0;
    const st_status s = select_sizes(B, K, V, keep);
    if (s == ST_OK) *bytes = st::beam_select_workspace(B, K, V, keep);
    return s;
}

st_status st_beam_select(const void* logits, st_dtype dtype, int64_t logits_stride, const float* scores,
                         int32_t B, int32_t K, int32_t V, int32_t keep, float* out_scores, int32_t* out_parents,
                         int32_t* out_tokens, const st_beam_extras* extras, void* workspace,
                         int64_t workspace_bytes, cudaStream_t stream)
{
    return guarded([&]() -> st_status {
        const st_status s = select_sizes(B, K, V, keep);
        if (s == ST_ERR_INVALID_ARG) return s;
        if ((dtype != ST_BF16 && dtype != ST_F16 && dtype != ST_F32) || logits_stride < V) return ST_ERR_INVALID_ARG;
        st::SelectArgs a{logits, dtype, logits_stride, scores, B, K, V, keep, out_scores, out_parents, out_tokens, {}, workspace};
        if (extras) a.ex = *extras;
        constexpr int64_t far = int64_t(1) << 56;
        if (a.ex.allow_request_stride < 0 || a.ex.allow_beam_stride < 0 || logits_stride >= far || a.ex.allow_request_stride >= far ||
            a.ex.allow_beam_stride >= far ||
            (a.ex.finished == nullptr) != (a.ex.out_finished == nullptr) ||
            (a.ex.finished && (a.ex.end_token < 0 || a.ex.end_token >= V)))
            return ST_ERR_INVALID_ARG;
        if (s != ST_OK) return s;
        const int64_t need = st::beam_select_workspace(B, K, V, keep);
        // the outputs and the workspace are written while the rest is read
        const int64_t pairs = int64_t(B) * keep, size = dtype == ST_F32 ? 4 : 2;
        const Vectors part[] = {dense(out_scores, pairs * 4), dense(out_parents, pairs * 4), dense(out_tokens, pairs * 4),
                                dense(a.ex.out_finished, a.ex.out_finished ? pairs : 0), dense(workspace, need),
                                {logits, 1, 0, int64_t(B) * K, logits_stride * size, V * size}, dense(scores, int64_t(B) * K * 4),
                                {a.ex.allow, B, a.ex.allow_request_stride * 4, K, a.ex.allow_beam_stride * 4, a.ex.allow ? (V + 31) / 32 * 4 : 0},
                                dense(a.ex.finished, a.ex.finished ? int64_t(B) * K : 0)};
        for (int i = 0; i < 5; ++i)
            for (int j = i + 1; j < 9; ++j)
                if (part[i].bytes > 0 && part[j].bytes > 0 && !apart(part[i], part[j])) return ST_ERR_INVALID_ARG;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return ST_ERR_CUDA;
        if (!on_device(logits, dev, dtype == ST_F32 ? 4 : 2) || !on_device(scores, dev, 4) ||
            !on_device(out_scores, dev, 4) || !on_device(out_parents, dev, 4) || !on_device(out_tokens, dev, 4) ||
            (a.ex.allow && !on_device(a.ex.allow, dev, 4)) || (a.ex.finished && !on_device(a.ex.finished, dev, 1)) ||
            (a.ex.out_finished && !on_device(a.ex.out_finished, dev, 1)))
            return ST_ERR_INVALID_ARG;
        if (need > 0 && (workspace_bytes < need || !on_device(workspace, dev, 16))) return ST_ERR_INVALID_ARG;
        return to_status(st::launch_beam_select(a, stream));
    });
}

st_status st_beam_reorder(const st_beam_state* states, int32_t n_states, const int32_t* parents, int32_t B,
                          int32_t K, int32_t keep, cudaStream_t stream)
{
    return guarded([&]() -> st_status {
        if (states == nullptr || n_states < 1 || B < 1 || K < 1 || keep < 1) return ST_ERR_INVALID_ARG;
        const int64_t n_src = int64_t(B) * K, n_dst = int64_t(B) * keep;
        const int64_t far = int64_t(1) << 62;
        for (int i = 0; i < n_states; ++i) {
            const st_beam_state& x = states[i];
            if (x.row_bytes < 0 || x.outer < 0 || x.src_row_stride < 0 || x.dst_row_stride < 0 ||
                x.src_outer_stride < 0 || x.dst_outer_stride < 0)
                return ST_ERR_INVALID_ARG;
        }
        if (n_states > ST_BEAM_MAX_STATES || n_src >= kLimit31 || n_dst >= kLimit31) return ST_ERR_UNSUPPORTED;
        // the bytes that each array's rows span, for the overlap checks
        struct Span {
            __int128 lo, hi;
        } src[ST_BEAM_MAX_STATES], dst[ST_BEAM_MAX_STATES];
        for (int i = 0; i < n_states; ++i) {
            const st_beam_state& x = states[i];
            src[i] = dst[i] = Span{0, 0};
            if (x.row_bytes == 0 || x.outer == 0) continue;
            const __int128 ls = __int128(x.outer - 1) * x.src_outer_stride + __int128(n_src - 1) * x.src_row_stride + x.row_bytes;
            const __int128 ld = __int128(x.outer - 1) * x.dst_outer_stride + __int128(n_dst - 1) * x.dst_row_stride + x.row_bytes;
            if (ls > far || ld > far) return ST_ERR_INVALID_ARG;
            // rows of dst apart from each other: rows inside outer parts, or outer parts inside rows
            const bool rows_inside = (n_dst == 1 || x.dst_row_stride >= x.row_bytes) &&
                                     (x.outer == 1 || __int128(x.dst_outer_stride) >= __int128(n_dst - 1) * x.dst_row_stride + x.row_bytes);
            const bool outer_inside = (x.outer == 1 || x.dst_outer_stride >= x.row_bytes) &&
                                      (n_dst == 1 || __int128(x.dst_row_stride) >= __int128(x.outer - 1) * x.dst_outer_stride + x.row_bytes);
            if (!rows_inside && !outer_inside) return ST_ERR_INVALID_ARG;
            src[i].lo = reinterpret_cast<uintptr_t>(x.src);
            src[i].hi = src[i].lo + ls;
            dst[i].lo = reinterpret_cast<uintptr_t>(x.dst);
            dst[i].hi = dst[i].lo + ld;
        }
        const Span by{__int128(reinterpret_cast<uintptr_t>(parents)), __int128(reinterpret_cast<uintptr_t>(parents)) + n_dst * 4};
        for (int i = 0; i < n_states; ++i)
            if (dst[i].lo < by.hi && by.lo < dst[i].hi) return ST_ERR_INVALID_ARG;
        for (int i = 0; i < n_states; ++i)
            for (int j = 0; j < n_states; ++j) {
                if (dst[i].lo < src[j].hi && src[j].lo < dst[i].hi) return ST_ERR_INVALID_ARG;
                if (i < j && dst[i].lo < dst[j].hi && dst[j].lo < dst[i].hi) return ST_ERR_INVALID_ARG;
            }
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return ST_ERR_CUDA;
        if (!on_device(parents, dev, 4)) return ST_ERR_INVALID_ARG;
        for (int i = 0; i < n_states; ++i)
            if (states[i].row_bytes > 0 && states[i].outer > 0 && (!on_device(states[i].src, dev, 1) || !on_device(states[i].dst, dev, 1)))
                return ST_ERR_INVALID_ARG;
        uint32_t* err = nullptr;
        cudaError_t e = st::decode_error_address(&err);
        if (e == cudaSuccess) e = st::launch_beam_reorder(states, n_states, parents, B, K, keep, err, stream);
        return to_status(e);
    });
}

st_status st_decode_check(cudaStream_t stream)
{
    return guarded([&]() -> st_status {
        if (cudaStreamSynchronize(stream) != cudaSuccess) return ST_ERR_CUDA;
        uint32_t word = 0;
        if (st::decode_error_word(&word) != cudaSuccess) return ST_ERR_CUDA;
        return word ? ST_ERR_DEVICE : ST_OK;
    });
}

}  // extern "C"
