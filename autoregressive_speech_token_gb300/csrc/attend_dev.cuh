// Shared by the kernels behind sd_attend_pages and sd_attend_cross.
#pragma once
#include "pages_dev.cuh"

// Partial results of the split kernel: two records a block, one arrival counter.
// The counters are zero between calls (the last arriver of a unit clears its own).
struct sd_attn_ws {
    int device = 0, sms = 0;
    float* part = nullptr;
    int* cnt = nullptr;
    int* err = nullptr;              // pinned: a kernel's expired wait
};

namespace sd {

struct AttendArgs {
    const void *q, *k, *v;
    void* out;
    float* lse;
    const int32_t *table, *len;      // table NULL: positions by strides
    const float *k_scale, *v_scale;
    FastDiv by_ps;
    int64_t batch_stride, page_stride, head_stride, pos_stride, q_batch, q_stride, o_batch, o_stride;
    int32_t B, Lq, H, Hkv, n_pages, table_stride, max_len, dtype, kv_dtype;
    float scale;
    float* part;
    int *cnt, *err;
};

constexpr int kSplitBlocksPerSm = 2;                              // at most
constexpr int kSplitRows = 8;                                     // query rows of a unit
constexpr int kSplitRecord = kSplitRows * (128 + 2);              // floats of a partial record

constexpr int kMaxPositions = INT32_MAX - 1023;                   // of a row: tile arithmetic stays within int32

cudaError_t prepare_attend_split();                               // shared-memory limits on the current device
cudaError_t prepare_attend_tc();
cudaError_t launch_attend_tc(const AttendArgs& a, int hd, int sms, cudaStream_t st, bool* taken);
cudaError_t launch_attend_split(const AttendArgs& a, int hd, int sms, cudaStream_t st);

}  // namespace sd
