// Shared by the kernels behind sd_attend_pages and sd_attend_cross.
#pragma once
#include <cuda.h>

#include "pages_dev.cuh"

// Partial results: a record a block of the tensor-core kernel, or two of the split kernel with its arrival counters.
// The counters are zero between calls (the last arriver of a unit clears its own).
struct sd_attn_ws {
    int device = 0, sms = 0;
    float* part = nullptr;
    int* cnt = nullptr;              // the counters, and behind them the word of AttendArgs::dead
    int* err = nullptr;              // pinned: a kernel's expired wait, for the host
    long long test_stall = 0;        // test hook (SD_TEST_STALL_US): cycles for one wait of the first uncaptured call
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
    int* dead;                       // set with err.  A launch that finds it set (a replayed graph: no host call looks at err)
                                     // leaves the counters alone, which are not zero then, and writes NaN
    long long stall;                 // test hook: block 0 waits as many cycles for a barrier that nothing arrives at
};

constexpr int kSplitRows = 8;                                     // query rows of a unit
constexpr int kSplitRecord = kSplitRows * (128 + 2);              // floats of a partial record
constexpr int kTcRecord = 2 * 128 * (128 + 2);                    // of the tensor-core kernel: two tiles of 128 queries

constexpr int kMaxPositions = INT32_MAX - 1023;                   // of a row: tile arithmetic stays within int32

cudaError_t prepare_attend_split();                               // shared-memory limits on the current device
cudaError_t prepare_attend_tc();
cudaError_t launch_attend_tc(const AttendArgs& a, int hd, int sms, cudaStream_t st, bool* taken);
cudaError_t launch_attend_split(const AttendArgs& a, int hd, int sms, cudaStream_t st);

// ---- device side

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr long long kWaitClocks = 4000000000ll;                   // about two seconds

// a / b for a >= 0, b > 0: in 32 bits where both fit (a 64-bit division costs a few hundred cycles)
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
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

}  // namespace sd
