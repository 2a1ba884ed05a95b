// sd_page_plan: block tables, slot maps and positions of a step from the
// requests' lengths, in one launch and without the host.
//
// With old(r) = ceil(len / ps) and all(r) = ceil((len + new) / ps), request r takes
// all(r) - old(r) pages of the free list, behind those of the requests before it,
// and its tokens follow theirs: two prefix sums over the requests.  Nothing is
// computed beyond that; at the sizes of a step (some KB) the call is bound by the
// chain launch -> lengths -> prefix -> table entry -> store.
//
// Split: a block owns kTok consecutive tokens.  Each block forms the prefix sums
// over all requests itself (8 bytes a request out of L2) instead of waiting for a
// first kernel's sums.  A request that begins in the block's tokens marks its
// first token; the token's request is the last mark at or before it, found with
// one bit mask per 32 tokens.  A page taken anew always begins with a new token
// (its first position is at or behind len), so that token's thread puts the page
// into the table, however long the request.
#include "pages_dev.cuh"

namespace sd {
namespace {

constexpr int kThreads = 512, kTok = 512, kWords = kTok / 32;
enum { BIT_ROWS = 1, BIT_FREE = 2, BIT_WIDE = 4, BIT_NEG = 8 };

struct PlanArgs {
    const int32_t *len, *fresh, *free_list;
    int32_t *table, *total, *start, *slot, *pos, *req, *info;
    int32_t R, n_free, width, rows;
    uint32_t ps;
    FastDiv by_ps;
};

struct Request {
    int64_t total;
    int32_t len, fresh, old, take, flags;
};

__device__ __forceinline__ Request request(const PlanArgs& a, int r) {
    Request q;
    int32_t len = a.len[r], fresh = a.fresh[r];
    q.flags = (len < 0 || fresh < 0) ? BIT_NEG : 0;
    q.len = len = max(len, 0);
    q.fresh = fresh = max(fresh, 0);
    q.total = (int64_t)len + fresh;
    // ceil(x / ps) = floor((x - 1) / ps) + 1 for x > 0: stays below 2^31
    q.old = len ? (int32_t)a.by_ps.div((uint32_t)len - 1) + 1 : 0;
    int64_t all = q.total ? (q.total - 1 <= INT32_MAX ? (int64_t)a.by_ps.div((uint32_t)(q.total - 1)) : (q.total - 1) / a.ps) + 1 : 0;
    if (all > a.width) {
        q.flags |= BIT_WIDE;
        all = a.width;
    }
    q.take = all > q.old ? (int32_t)all - q.old : 0;
    return q;
}

__device__ __forceinline__ int32_t clip(int64_t v) { return v > INT32_MAX ? INT32_MAX : (int32_t)v; }

template <int kOwn>
__global__ void __launch_bounds__(kThreads) k_page_plan(const PlanArgs a) {
    pdl_trigger();
    pdl_wait();
    __shared__ int32_t s_req[kTok], s_len[kTok], s_first[kTok], s_off[kTok];
    __shared__ uint32_t s_mark[kWords];
    __shared__ int32_t s_prev[kWords];
    __shared__ int64_t s_tok[kThreads / 32], s_page[kThreads / 32];
    __shared__ int32_t s_flags, s_long;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t lo = (int64_t)blockIdx.x * kTok, hi = lo + kTok;
    if (tid < kWords) s_mark[tid] = 0;
    if (tid == 0) s_flags = s_long = 0;
    __syncthreads();

    int64_t tok0 = 0, page0 = 0;   // tokens and pages of the requests before this round's
    int32_t flags = 0, longest = 0;
    int round = 0;
    for (int64_t r0 = 0; r0 < a.R; r0 += kThreads * kOwn, ++round) {
        // kOwn consecutive requests a thread: one exchange between the threads for all of them
        const int64_t first_r = r0 + tid * kOwn;
        Request q[kOwn] = {};
        int64_t t = 0, p = 0;
#pragma unroll
        for (int k = 0; k < kOwn; ++k)
            if (first_r + k < a.R) q[k] = request(a, (int)(first_r + k));
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            t += q[k].fresh;
            p += q[k].take;
            flags |= q[k].flags;
            longest = max(longest, clip(q[k].total));
        }
        const int64_t own_t = t, own_p = p;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t tt = __shfl_up_sync(0xffffffffu, t, o), pp = __shfl_up_sync(0xffffffffu, p, o);
            if (lane >= o) {
                t += tt;
                p += pp;
            }
        }
        if (lane == 31) {
            s_tok[warp] = t;
            s_page[warp] = p;
        }
        __syncthreads();
        int64_t start = tok0 + t - own_t, first = page0 + p - own_p;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int64_t x = s_tok[w], y = s_page[w];
            if (w < warp) {
                start += x;
                first += y;
            }
            tok0 += x;
            page0 += y;
        }
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const int64_t r = first_r + k;
            if (r >= a.R) break;
            if (round % gridDim.x == blockIdx.x) {
                a.total[r] = clip(q[k].total);
                a.start[r] = clip(start);
            }
            if (q[k].fresh > 0 && start < hi && start + q[k].fresh > lo) {
                const int at = start > lo ? (int)(start - lo) : 0;
                atomicOr(&s_mark[at >> 5], 1u << (at & 31));
                s_req[at] = (int32_t)r;
                s_len[at] = q[k].len;
                s_off[at] = (int32_t)(lo + at - start);          // tokens of the request before this one
                s_first[at] = clip(first);
            }
            start += q[k].fresh;
            first += q[k].take;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0) {
        if (flags) atomicOr(&s_flags, flags);
        atomicMax(&s_long, longest);
    }
    // the last mark before each group of 32 tokens
    if (warp == 0) {
        const uint32_t m = lane < kWords ? s_mark[lane] : 0;
        int32_t last = m ? lane * 32 + 31 - __clz(m) : -1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t x = __shfl_up_sync(0xffffffffu, last, o);
            if (lane >= o) last = max(last, x);
        }
        const int32_t before = __shfl_up_sync(0xffffffffu, last, 1);
        if (lane < kWords) s_prev[lane] = lane ? before : -1;
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        a.start[a.R] = clip(tok0);
        a.info[0] = clip(tok0);
        a.info[1] = clip(page0);
        a.info[2] = s_flags | (tok0 > a.rows ? BIT_ROWS : 0) | (page0 > a.n_free ? BIT_FREE : 0);
        a.info[3] = s_long;
    }
#pragma unroll
    for (int k = 0; k < kTok / kThreads; ++k) {
        const int at = k * kThreads + tid;
        const int64_t i = lo + at;
        if (i >= a.rows) break;
        int32_t slot = -1, pos = 0, req = -1;
        if (i < tok0) {
            const uint32_t m = s_mark[at >> 5] & (0xffffffffu >> (31 - (at & 31)));
            const int h = m ? (at & ~31) + 31 - __clz(m) : s_prev[at >> 5];
            req = s_req[h];
            const int32_t len = s_len[h];
            const int64_t p64 = (int64_t)len + s_off[h] + (at - h);
            pos = clip(p64);
            if (p64 < INT32_MAX) {
                const uint32_t page = a.by_ps.div((uint32_t)pos), in = (uint32_t)pos - page * a.ps;
                if (page < (uint32_t)a.width) {
                    const int32_t old = len ? (int32_t)a.by_ps.div((uint32_t)len - 1) + 1 : 0;
                    int32_t* entry = a.table + (int64_t)req * a.width + page;
                    int32_t id;
                    if ((int32_t)page < old) {
                        id = *entry;
                    } else {
                        const int64_t j = (int64_t)s_first[h] + page - old;
                        id = j < a.n_free ? a.free_list[j] : -1;
                        if (in == 0) *entry = id;
                    }
                    const int64_t s = (int64_t)id * a.ps + in;
                    slot = id >= 0 && s <= INT32_MAX ? (int32_t)s : -1;
                }
            }
        }
        a.slot[i] = slot;
        a.pos[i] = pos;
        a.req[i] = req;
    }
}

}  // namespace
}  // namespace sd

extern "C" int sd_page_plan(const int32_t* len_dev, const int32_t* new_dev, int32_t R, const int32_t* free_dev,
                            int32_t n_free, int32_t page_size, int32_t* table_dev, int32_t table_stride, int32_t rows,
                            int32_t* total_dev, int32_t* start_dev, int32_t* slot_dev, int32_t* pos_dev,
                            int32_t* req_dev, int32_t* info_dev, void* stream) {
    using namespace sd;
    static const char* who = "sd_page_plan";
    if (!len_dev || !new_dev || !table_dev || !total_dev || !start_dev || !info_dev)
        return op_fail(SD_ERR_INVALID_ARG, "%s: NULL argument", who);
    if (R < 1 || n_free < 0 || rows < 0 || table_stride < 1 || page_size < 1 || page_size > 65536)
        return op_fail(SD_ERR_INVALID_ARG, "%s: R %d, n_free %d, rows %d, table_stride %d, page_size %d", who, R, n_free,
                       rows, table_stride, page_size);
    if (n_free > 0 && !free_dev) return op_fail(SD_ERR_INVALID_ARG, "%s: free_dev is NULL", who);
    if (rows > 0 && (!slot_dev || !pos_dev || !req_dev))
        return op_fail(SD_ERR_INVALID_ARG, "%s: slot_dev, pos_dev or req_dev is NULL", who);
    PlanArgs a;
    a.len = len_dev; a.fresh = new_dev; a.free_list = free_dev; a.table = table_dev; a.total = total_dev;
    a.start = start_dev; a.slot = slot_dev; a.pos = pos_dev; a.req = req_dev; a.info = info_dev;
    a.R = R; a.n_free = n_free; a.width = table_stride; a.rows = rows; a.ps = (uint32_t)page_size;
    a.by_ps = FastDiv((uint32_t)page_size);
    const int grid = rows > kTok ? (int)(((int64_t)rows + kTok - 1) / kTok) : 1;
    // Requests of a thread: one where the threads suffice (16 requests: 3.1 us, 4.0 us with four), else four, which
    // saves exchanges between the threads (2000 requests, 61k tokens: 5.0 us, 8.0 us with one and 1024 tokens a block).
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = R <= kThreads ? launch_k(k_page_plan<1>, dim3(grid), dim3(kThreads), 0, st, a)
                                        : launch_k(k_page_plan<4>, dim3(grid), dim3(kThreads), 0, st, a);
    if (e != cudaSuccess) return op_fail(SD_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return SD_OK;
}
