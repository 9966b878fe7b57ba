// What the decode operators (kv_plan.cu, kv_append.cu, kv_attend.cu,
// beam_select.cu, beam_reorder.cu) share with their host side (decode_api.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "st_internal.cuh"

namespace st {

// Bits of the decode error word (st_decode_check reports any of them).
enum : uint32_t {
    kDecErrTable = 1u << 0,   // a used block table entry is outside the cache
    kDecErrSlot = 1u << 1,    // a slot or source block is outside the cache
    kDecErrRow = 1u << 2,     // a row is longer than the launch was sized for
    kDecErrParent = 1u << 3,  // a parent beam is outside its request
    kDecErrWait = 1u << 4,    // a wait for a copy or a product ran out
};

// ------------------------------------------------------------------- plan --
struct PlanArgs {
    int32_t* table;
    const int32_t* have;
    const int32_t* add;
    int32_t R, max_blocks, num_blocks, block_size;
    int64_t T;
    int64_t* slots;
    int32_t* sources;
    int32_t* row_start;
    int32_t* lens;
    int32_t* report;
    uint32_t* err;
};
cudaError_t launch_kv_plan(const PlanArgs& a, cudaStream_t s);

// ----------------------------------------------------------------- append --
struct AppendArgs {
    st_kv_cache c;
    const void* k;
    const void* v;
    st_dtype dtype;
    int64_t T, k_token, k_head, v_token, v_head;  // strides in elements
    const int64_t* slots;
    const int32_t* sources;  // or null
    uint32_t* err;
};
cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t s);

// ----------------------------------------------------------------- attend --
struct AttendArgs {
    st_kv_cache c;
    const void* q;
    st_dtype dtype;
    int64_t T;
    int32_t q_heads;
    int64_t q_token, q_head;
    const int32_t* table;
    int32_t max_blocks;
    const int32_t* row_start;
    const int32_t* lens;
    int32_t R, max_q;
    int64_t max_len;
    float scale_log2;  // scale * log2(e): the softmax works in powers of two
    int32_t causal;
    void* out;
    int64_t out_token, out_head;
    void* workspace;
    uint32_t* err;
    // rows that a launch takes, by their columns (query tokens x heads per cache head): more than the first, up to
    // the second
    int32_t above_cols = 0, most_cols = 0x7fffffff;
    // the columns that have partial sums in the workspace: T * q_heads, numbered by token and head, or, with row_cols > 0,
    // that many for each row and cache head
    int64_t parts = 0;
    int32_t row_cols = 0;
};
constexpr int64_t kAttendMaxBytes = int64_t(1) << 48;  // of workspace: sizes that need more are refused
int64_t kv_attend_workspace(const st_kv_cache& c, int64_t T, int32_t q_heads, int32_t R, int32_t max_q,
                            int64_t max_len);
cudaError_t launch_kv_attend(const AttendArgs& a, cudaStream_t s);

// ----------------------------------------------------------------- select --
struct SelectArgs {
    const void* logits;
    st_dtype dtype;
    int64_t stride;
    const float* scores;
    int32_t B, K, V, keep;
    float* out_scores;
    int32_t* out_parents;
    int32_t* out_tokens;
    st_beam_extras ex;
    void* workspace;
};
int64_t beam_select_workspace(int32_t B, int32_t K, int32_t V, int32_t keep);
cudaError_t launch_beam_select(const SelectArgs& a, cudaStream_t s);

// ---------------------------------------------------------------- reorder --
cudaError_t launch_beam_reorder(const st_beam_state* states, int32_t n_states, const int32_t* parents, int32_t B,
                                int32_t K, int32_t keep, uint32_t* err, cudaStream_t s);

// The current device's decode error word: its address, and its value (cleared).
cudaError_t decode_error_address(uint32_t** word);
cudaError_t decode_error_word(uint32_t* value);

}  // namespace st
