// Shared by the kernels behind sd_attend_pages and sd_attend_cross.
#pragma once
#include <cuda.h>

#include "pages_dev.cuh"

// Partial results: a record a block of the tensor-core kernel, or two of the split kernel with its arrival counters.
// The counters are zero between calls (the last arriver of a unit clears its own).
namespace sd {
struct SharedRow;
}
struct sd_attn_ws {
    int device = 0, sms = 0;
    float* part = nullptr;
    int* cnt = nullptr;              // the counters, and behind them the word of AttendArgs::dead
    int* err = nullptr;              // pinned: a kernel's expired wait, for the host
    float* recs = nullptr;           // shared pages: partial results
    sd::SharedRow* desc = nullptr;   // and of which each request has its own, behind them the word of AttendArgs::shared
    long long share_bytes = 0;       // key and value bytes that sharing has to save (SD_SHARE_MIN_BYTES for the tests)
    long long test_stall = 0;        // test hook (SD_TEST_STALL_US): cycles for one wait of the first uncaptured call
};

namespace sd {

// Of a request whose first `skip` pages are attended to for its whole group of `size` requests from r0 on: the rows
// (request - r0, head) of a kv head are in items of `rows`, each of `tiles` tiles behind kShareLead empty ones; the group's
// first tile is `base` of all, and a block took `per` of them.
struct alignas(16) SharedRow {
    int32_t skip, r0, size, tiles, rows, unused[3];
    int64_t base, per;
};
constexpr int kShareLead = 8;                                     // what beginning and ending an item costs, in tiles
constexpr int kSharedRecord = 128 + 4;                            // floats of a row's partial result: output, maximum, sum
constexpr int kSharedRows = 65536;                                // query rows (request, head) that a workspace has records for
constexpr int kSharedBlock = 256;                                 // and more for each block, for the item that it continues

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
    int* dead;                       // set with err.  A launch that finds it set (a replayed graph: no host call looks at err)
                                     // leaves the counters alone, which are not zero then, and writes NaN
    float* recs;                     // shared pages
    SharedRow* desc;
    int32_t* shared;                 // 1: the kernels for shared pages serve this call, 0: the split kernel does; NULL: it does
    long long stall;                 // test hook: a block waits as many cycles for a barrier that nothing arrives at
};

constexpr int kSplitRows = 8;                                     // query rows of a unit
constexpr int kSplitRecord = kSplitRows * (128 + 2);              // floats of a partial record
constexpr int kTcRecord = 2 * 128 * (128 + 2);                    // of the tensor-core kernel: two tiles of 128 queries

constexpr int kMaxPositions = INT32_MAX - 1023;                   // of a row: tile arithmetic stays within int32

cudaError_t prepare_attend_split();                               // shared-memory limits on the current device
cudaError_t prepare_attend_tc();
cudaError_t launch_attend_tc(const AttendArgs& a, int hd, int sms, cudaStream_t st, bool* taken);
cudaError_t prepare_attend_shared();
cudaError_t prepare_attend_own();
cudaError_t launch_attend_own(const AttendArgs& a, int hd, cudaStream_t st);
// *taken false: strides that a tensor map cannot hold, nothing launched
cudaError_t launch_attend_shared(const AttendArgs& a, const int32_t* group, const int32_t* shared, int n_groups, int hd, int sms,
                                 cudaStream_t st, int64_t worth, bool* taken);
cudaError_t launch_attend_split(const AttendArgs& a, int hd, int sms, cudaStream_t st);

// ---- device side

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr long long kWaitClocks = 4000000000ll;                   // about two seconds

// a / b for a >= 0, b > 0: in 32 bits where both fit (a 64-bit division costs a few hundred cycles)
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// Where the records of a part of an item lie, as 4-column pieces [piece][row] and behind them (maximum, sum) of each row: the
// part that begins the item has the place of its rows among all (request, head) rows, the others their block's.
__device__ __forceinline__ float* shared_records(const AttendArgs& a, bool begins, int64_t first_row, int block) {
    return a.recs + (begins ? first_row : (int64_t)a.B * a.H + (int64_t)block * kSharedBlock) * kSharedRecord;
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mb_init(uint32_t mb, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(mb), "r"(n) : "memory");
}
__device__ __forceinline__ void mb_expect(uint32_t mb, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mb), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mb_expect_more(uint32_t mb, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(mb), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mb_arrive(uint32_t mb) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(mb) : "memory");
}
__device__ __forceinline__ bool mb_try(uint32_t mb, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(mb), "r"(parity) : "memory");
    return ok != 0;
}
// The same, asleep until the phase completes or about 20 us have passed: a polling warp takes issue slots from the
// others of its scheduler
__device__ __forceinline__ bool mb_sleep(uint32_t mb, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(mb), "r"(parity), "r"(20000u) : "memory");
    return ok != 0;
}
// Bounded; gives up early once another warp of the block has given up.
__device__ __forceinline__ bool mb_wait(uint32_t mb, uint32_t parity, volatile int* bad, long long limit = kWaitClocks) {
    if (mb_sleep(mb, parity)) return true;
    const long long t0 = clock64();
    while (!mb_sleep(mb, parity)) {
        if (*bad) return false;
        if (clock64() - t0 > limit) {
            *bad = 1;
            return false;
        }
    }
    return true;
}
// The same by a whole warp, with one answer: what follows may be an instruction of all its lanes.
__device__ __forceinline__ bool warp_wait(uint32_t mb, uint32_t parity, volatile int* bad, long long limit = kWaitClocks) {
    return __all_sync(0xffffffffu, mb_wait(mb, parity, bad, limit));
}
__device__ __forceinline__ void report_expired(const AttendArgs& a) {
    *a.err = SD_ERR_TIMEOUT;
    *a.dead = 1;
}
// One lane of a converged warp.  (The compiler keeps what such a branch computes in uniform registers, which a
// comparison of lane numbers does not give.)
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void tma4(uint32_t dst, const CUtensorMap* map, int x, int h, int r, int b, uint32_t mb) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(r), "r"(b), "r"(mb) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- tensor maps

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeFn tensor_map_encoder() {
    static EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return (EncodeFn) nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// K or V by strides, as [outer][head][position][hd]: boxes of `box` positions of up to 128 bytes of a row
inline bool map_kv(CUtensorMap* map, int dtype, const void* base, int hd, int positions, int heads, int outer, int64_t pos_stride,
            int64_t head_stride, int64_t outer_stride, int box) {
    EncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    const int bytes = dtype == SD_E4M3 ? 1 : 2, row = hd * bytes;
    const cuuint64_t dims[4] = {(cuuint64_t)hd, (cuuint64_t)positions, (cuuint64_t)heads, (cuuint64_t)outer};
    // the stride of a dimension of one element is not used: any legal value
    const cuuint64_t strides[3] = {(cuuint64_t)(positions > 1 ? pos_stride * bytes : row),
                                   (cuuint64_t)(heads > 1 ? head_stride * bytes : row),
                                   (cuuint64_t)(outer > 1 ? outer_stride * bytes : row)};
    const cuuint32_t boxes[4] = {(cuuint32_t)(row < 128 ? hd : 128 / bytes), (cuuint32_t)box, 1, 1}, one[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = dtype == SD_E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : dtype == SD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return enc(map, type, 4, const_cast<void*>(base), dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               row < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sd
