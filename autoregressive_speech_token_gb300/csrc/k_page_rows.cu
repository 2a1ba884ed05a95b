// sd_page_fork and sd_page_compact: tables, reference counts, copy lists and free
// lists when rows of a paged cache are forked, ended or moved together.
//
// Fork.  New row i continues row p = parent[i]; of n = len[p] positions the full
// pages are shared, and the partly filled one belongs to the lowest i of its parent.
// Any other i takes the free page whose place in the list is its rank,
//   rank(i) = #{k < i : k needs a page},   k needs one <=> n % ps > 0 and first[parent[k]] != k,
// first[p] = the lowest row with parent p (an atomic minimum).  A page goes back to the free list if an
// old row names it and no new row does: two bit maps, and a prefix sum of bits for its place.
//
// Compact.  With L pages in use, the k-th page in use with an id from L on moves to the k-th
// id below L that is not in use: ranks in one bit map.
//
// Counts and bits are order-independent, places are prefix sums: the outputs do not depend on which
// atomic came first.  Little is computed; what bounds the calls is the chain of
// passes (clear, mark, fill, list), each of which needs all of the one before.
// Small calls run it in one block, others a launch for each pass: 16 rollouts of a prompt forked 4.3 us in one
// block, 10.0 in four launches; compacted 3.5 and 14.3; 2000 rows forked 16 us, compacted 13.
#include <algorithm>

#include "pages_dev.cuh"

namespace sd {
namespace {

enum { BIT_FREE = 2, BIT_WIDE = 4, BIT_NEG = 8, BIT_ID = 16 };
enum { W_FLAGS = 0, W_LONGEST = 1, W_WORDS = 32 };        // words of the work area before its arrays

struct RowArgs {
    const int32_t *table, *len, *parent, *free_list;
    int32_t *out, *len_out, *copies, *ref, *free_out, *info;
    int32_t *word, *first, *place;                         // place: compact's rank of a page that moves
    uint32_t *old_bits, *new_bits;
    int32_t R, N, n_free, width, n_pages, words;           // words of a bit map
    uint32_t ps;
    FastDiv by_ps;
};

// A row's positions, limited to what its table row holds, and its pages
struct Row {
    int32_t len, full, rest, used;
    int32_t flags;
};
__device__ __forceinline__ Row row_of(const RowArgs& a, int32_t len) {
    Row r;
    r.flags = len < 0 ? BIT_NEG : 0;
    len = max(len, 0);
    r.full = (int32_t)a.by_ps.div((uint32_t)len);
    r.rest = len - r.full * (int32_t)a.ps;
    if (r.full >= a.width && (r.full > a.width || r.rest)) {
        r.flags |= BIT_WIDE;
        r.full = a.width;
        r.rest = 0;
        len = (int32_t)((int64_t)a.width * a.ps);          // below the row's own length: fits
    }
    r.len = len;
    r.used = r.full + (r.rest > 0);
    return r;
}
// Old row of new row i, -1 without one
__device__ __forceinline__ int32_t parent_of(const RowArgs& a, int64_t i) {
    const int32_t p = a.parent[i];
    return (uint32_t)p < (uint32_t)a.R ? p : -1;
}
__device__ __forceinline__ bool needs_page(const RowArgs& a, int64_t i) {
    const int32_t p = parent_of(a, i);
    if (p < 0) return false;
    const int32_t first = __ldcg(a.first + p);
    return row_of(a, a.len[p]).rest > 0 && first != i;
}
__device__ __forceinline__ void raise(const RowArgs& a, int32_t flags) {
    if (flags) atomicOr(a.word + W_FLAGS, flags);
}

// This thread's place among the threads that run a pass: of one block or of the grid
struct Team {
    int64_t thread, threads;
    __device__ __forceinline__ int64_t warp() const { return thread >> 5; }
    __device__ __forceinline__ int64_t warps() const { return threads >> 5; }
};

__device__ __forceinline__ void pass_clear(const RowArgs& a, Team t) {
    for (int64_t i = t.thread; i < a.n_pages; i += t.threads) a.ref[i] = 0;
    for (int64_t i = t.thread; i < a.words; i += t.threads) a.old_bits[i] = a.new_bits[i] = 0;
    if (a.parent)
        for (int64_t i = t.thread; i < a.R; i += t.threads) a.first[i] = INT32_MAX;
    if (t.thread < W_WORDS) a.word[t.thread] = 0;
}

constexpr int kEntries = 8, kChunk = 32 * kEntries;       // table entries of a lane and of a warp at a time

// Bits of the pages that the old rows name; the lowest new row of each old one
__device__ __forceinline__ void pass_mark(const RowArgs& a, Team t) {
    const int lane = threadIdx.x & 31;
    if (a.parent)
        for (int64_t i = t.thread; i < a.N; i += t.threads) {
            const int32_t p = parent_of(a, i);
            if (p >= 0) atomicMin(a.first + p, (int32_t)i);
        }
    const int64_t chunks = (a.width + kChunk - 1) / kChunk;
    for (int64_t w = t.warp(); w < a.R * chunks; w += t.warps()) {
        const int64_t r = w / chunks;
        const int c = (int)(w - r * chunks) * kChunk;
        const Row row = row_of(a, a.len[r]);
        int32_t flags = c == 0 ? row.flags : 0, id[kEntries];
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int j = c + e * 32 + lane;
            id[e] = j < row.used ? a.table[r * a.width + j] : INT32_MIN;
        }
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            if (id[e] == INT32_MIN && c + e * 32 + lane >= row.used) continue;
            if ((uint32_t)id[e] < (uint32_t)a.n_pages) atomicOr(a.old_bits + (id[e] >> 5), 1u << (id[e] & 31));
            else flags |= BIT_ID;
        }
        raise(a, flags);
    }
}

// Inclusive sum over a block's threads; *total of all.  s_sum has a word for each warp.
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* s_sum, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) x += s_sum[w];
        all += s_sum[w];
    }
    *total = all;
    return x;
}

// ---- fork

// The new rows but for the pages that are taken anew
__device__ __forceinline__ void pass_fill(const RowArgs& a, Team t) {
    const int lane = threadIdx.x & 31;
    const int64_t chunks = (a.width + kChunk - 1) / kChunk;
    for (int64_t w = t.warp(); w < a.N * chunks; w += t.warps()) {
        const int64_t i = w / chunks;
        const int c = (int)(w - i * chunks) * kChunk;
        const int32_t p = parent_of(a, i);
        Row row = {};
        bool fresh = false;
        if (p >= 0) {
            const int32_t first = __ldcg(a.first + p);
            row = row_of(a, a.len[p]);
            fresh = row.rest > 0 && first != i;
        }
        int32_t id[kEntries];
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int j = c + e * 32 + lane;
            id[e] = j < row.used ? a.table[(int64_t)p * a.width + j] : -1;
        }
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int j = c + e * 32 + lane;
            if (j >= a.width || (fresh && j == row.full)) continue;
            const bool live = (uint32_t)id[e] < (uint32_t)a.n_pages;
            a.out[i * a.width + j] = live ? id[e] : -1;
            if (live && atomicAdd(a.ref + id[e], 1) == 0) atomicOr(a.new_bits + (id[e] >> 5), 1u << (id[e] & 31));
        }
    }
}

// Lengths, and the pages taken anew, of rows [lo, hi): one block's.  Returns how many rows below hi need a page.
__device__ __forceinline__ int64_t pass_take(const RowArgs& a, int64_t lo, int64_t hi, int64_t* s_sum) {
    int64_t mine = 0, before;
    for (int64_t i = threadIdx.x; i < lo; i += blockDim.x) mine += needs_page(a, i);
    block_sum(mine, s_sum, &before);
    int32_t longest = 0;
    for (int64_t i0 = lo; i0 < hi; i0 += blockDim.x) {
        const int64_t i = i0 + threadIdx.x;
        const bool need = i < hi && needs_page(a, i);
        int64_t all;
        const int64_t k = before + block_sum(need, s_sum, &all) - need;
        before += all;
        if (i >= hi) continue;
        const int32_t p = parent_of(a, i);
        Row row = {};
        if (p >= 0) row = row_of(a, a.len[p]);
        if (need) {
            const bool have = k < a.n_free;
            int32_t page = have ? a.free_list[k] : -1, from = a.table[(int64_t)p * a.width + row.full];
            if (have && (uint32_t)page >= (uint32_t)a.n_pages) {
                page = -1;
                raise(a, BIT_ID);
            }
            if ((uint32_t)from >= (uint32_t)a.n_pages) from = -1;
            a.out[i * a.width + row.full] = page;
            if (page >= 0 && atomicAdd(a.ref + page, 1) == 0) atomicOr(a.new_bits + (page >> 5), 1u << (page & 31));
            if (page < 0) row.len -= row.rest;
            if (have) {
                a.copies[3 * k] = from;
                a.copies[3 * k + 1] = page;
                a.copies[3 * k + 2] = row.rest;
            }
        }
        a.len_out[i] = row.len;
        longest = max(longest, row.len);
    }
    if (longest) atomicMax(a.word + W_LONGEST, longest);
    return before;
}

// ---- places in bit maps.  A block has kWords words of a map, a thread four of their pages; how many bits lie before them,
// every block counts for itself.

constexpr int kThreads = 256, kWords = 32;                // threads of a block of a pass
struct Words {
    uint32_t word[kWords];
    int64_t before[kWords];                                // bits before the word
};
// The block's words, `x` those of thread < kWords, with `at` bits before the first
__device__ __forceinline__ void lay_words(Words& s, uint32_t x, int64_t at) {
    if (threadIdx.x < kWords) {
        int n = __popc(x);
        const int own = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, n, o);
            if ((int)threadIdx.x >= o) n += y;
        }
        s.word[threadIdx.x] = x;
        s.before[threadIdx.x] = at + n - own;
    }
    __syncthreads();
}

// The free list: what is left of the old one, then the pages of old rows that no new row names.
__device__ __forceinline__ void pass_release(const RowArgs& a, int64_t need, Team t, Words& s, int64_t* s_sum) {
    const int64_t taken = min(need, (int64_t)a.n_free), left = a.n_free - taken;
    for (int64_t i = t.thread; i < left; i += t.threads)
        if (i < a.n_pages) a.free_out[i] = a.free_list[taken + i];
    auto word = [&](int64_t w) { return w < a.words ? __ldcg(a.old_bits + w) & ~__ldcg(a.new_bits + w) : 0u; };
    const int64_t lo = (int64_t)blockIdx.x * kWords;
    const uint32_t x = threadIdx.x < kWords ? word(lo + threadIdx.x) : 0;
    int64_t mine = 0, at;
    for (int64_t w = threadIdx.x; w < lo; w += kThreads) mine += __popc(word(w));
    block_sum(mine, s_sum, &at);
    at += left;
    lay_words(s, x, at);
    for (int i = threadIdx.x; i < kWords * 32; i += kThreads) {
        const uint32_t bits = s.word[i >> 5];
        const int64_t k = s.before[i >> 5] + __popc(bits & ((1u << (i & 31)) - 1));
        if (((bits >> (i & 31)) & 1) && k < a.n_pages) a.free_out[k] = (int32_t)(lo * 32 + i);
    }
    if (lo + kWords >= a.words && threadIdx.x == 0) {
        at = s.before[kWords - 1] + __popc(s.word[kWords - 1]);
        a.info[0] = (int32_t)taken;
        a.info[1] = (int32_t)min(at, (int64_t)a.n_pages);
        a.info[2] = __ldcg(a.word + W_FLAGS) | (need > a.n_free ? BIT_FREE : 0);
        a.info[3] = __ldcg(a.word + W_LONGEST);
    }
}

// Where pages move
__device__ __forceinline__ void pass_places(const RowArgs& a, Team t, Words& s, int64_t* s_sum) {
    const int64_t lo = (int64_t)blockIdx.x * kWords;
    const uint32_t x = threadIdx.x < kWords && lo + threadIdx.x < a.words ? __ldcg(a.old_bits + lo + threadIdx.x) : 0;
    int64_t all = 0, low = 0, live, at;
    for (int64_t w = threadIdx.x; w < a.words; w += kThreads) {
        const int n = __popc(__ldcg(a.old_bits + w));
        all += n;
        if (w < lo) low += n;
    }
    block_sum(all, s_sum, &live);
    block_sum(low, s_sum, &at);
    // pages in use below `live`, which stay
    int64_t mine = 0, stay;
    for (int64_t w = threadIdx.x; w <= live >> 5 && w < a.words; w += kThreads)
        mine += __popc(__ldcg(a.old_bits + w) & (w < live >> 5 ? 0xffffffffu : (1u << (live & 31)) - 1));
    block_sum(mine, s_sum, &stay);
    lay_words(s, x, at);
    for (int i = threadIdx.x; i < kWords * 32; i += kThreads) {
        const int64_t id = lo * 32 + i;
        if (id >= a.n_pages) break;
        const uint32_t bits = s.word[i >> 5];
        const int64_t k = s.before[i >> 5] + __popc(bits & ((1u << (i & 31)) - 1));
        if ((bits >> (i & 31)) & 1) {
            if (id >= live) {                              // the (k - stay)-th that moves
                a.place[id] = (int32_t)(k - stay);
                a.copies[3 * (k - stay)] = (int32_t)id;
                a.copies[3 * (k - stay) + 2] = (int32_t)a.ps;
            }
        } else if (id < live) {
            a.copies[3 * (id - k) + 1] = (int32_t)id;      // the (id - k)-th that is free
        }
        if (id >= live) a.free_out[id - live] = (int32_t)id;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.info[0] = (int32_t)(live - stay);
        a.info[1] = (int32_t)(a.n_pages - live);
        a.info[2] = __ldcg(a.word + W_FLAGS);
        a.info[3] = (int32_t)live;
    }
}

// The rows with the pages' new ids
__device__ __forceinline__ void pass_rename(const RowArgs& a, Team t, int64_t live) {
    const int lane = threadIdx.x & 31;
    const int64_t chunks = (a.width + kChunk - 1) / kChunk;
    for (int64_t w = t.warp(); w < a.R * chunks; w += t.warps()) {
        const int64_t r = w / chunks;
        const int c = (int)(w - r * chunks) * kChunk;
        const Row row = row_of(a, a.len[r]);
        int32_t id[kEntries];
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int j = c + e * 32 + lane;
            id[e] = j < row.used ? a.table[r * a.width + j] : -1;
            if ((uint32_t)id[e] >= (uint32_t)a.n_pages) id[e] = -1;
        }
#pragma unroll
        for (int e = 0; e < kEntries; ++e)
            if (id[e] >= live) id[e] = __ldcg(a.copies + 3 * (int64_t)__ldcg(a.place + id[e]) + 1);
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int j = c + e * 32 + lane;
            if (j < a.width) a.out[r * a.width + j] = id[e];
            if (id[e] >= 0) atomicAdd(a.ref + id[e], 1);
        }
    }
}

// ---- kernels

constexpr int kOne = 1024;                                 // threads of the block that does all passes

__device__ __forceinline__ Team grid_team() {
    return {blockIdx.x * (int64_t)blockDim.x + threadIdx.x, gridDim.x * (int64_t)blockDim.x};
}

__global__ void __launch_bounds__(kThreads) k_rows_clear(const RowArgs a) {
    pdl_trigger();
    pdl_wait();
    pass_clear(a, grid_team());
}
__global__ void __launch_bounds__(kThreads) k_rows_mark(const RowArgs a) {
    pdl_trigger();
    pdl_wait();
    pass_mark(a, grid_team());
}
// The first `takers` blocks: lengths and new pages of kThreads rows each; the others: the rows
__global__ void __launch_bounds__(kThreads) k_fork_fill(const RowArgs a, int takers) {
    __shared__ int64_t s_sum[kThreads / 32];
    pdl_trigger();
    pdl_wait();
    if ((int)blockIdx.x < takers) {
        const int64_t lo = (int64_t)blockIdx.x * kThreads, hi = min(lo + kThreads, (int64_t)a.N);
        const int64_t need = pass_take(a, lo, hi, s_sum);
        if ((int)blockIdx.x == takers - 1 && threadIdx.x == 0) *reinterpret_cast<int64_t*>(a.word + 2) = need;
        return;
    }
    pass_fill(a, {((int64_t)blockIdx.x - takers) * kThreads + threadIdx.x, ((int64_t)gridDim.x - takers) * kThreads});
}
__global__ void __launch_bounds__(kThreads) k_fork_release(const RowArgs a) {
    __shared__ int64_t s_sum[kThreads / 32];
    __shared__ Words s;
    pdl_trigger();
    pdl_wait();
    pass_release(a, __ldcg(reinterpret_cast<const long long*>(a.word + 2)), grid_team(), s, s_sum);
}
__global__ void __launch_bounds__(kThreads) k_compact_places(const RowArgs a) {
    __shared__ int64_t s_sum[kThreads / 32];
    __shared__ Words s;
    pdl_trigger();
    pdl_wait();
    pass_places(a, grid_team(), s, s_sum);
}
__global__ void __launch_bounds__(kThreads) k_compact_rename(const RowArgs a) {
    pdl_trigger();
    pdl_wait();
    pass_rename(a, grid_team(), __ldcg(a.info + 3));
}
// ---- all passes in one block: counts, bits and lowest rows in shared memory, so that the only things waited for in turn are
// lengths and parents, table entries, and the free list

constexpr int kOneRows = 2048, kOnePages = 4096;           // old and new rows; pages
struct One {
    uint32_t old_bits[kOnePages / 32], new_bits[kOnePages / 32];
    int32_t ref[kOnePages], sum[kOne / 32], flags, longest;
};

// Inclusive sum over the block's threads; *total of all
__device__ __forceinline__ int32_t one_sum(int32_t x, int32_t* s_sum, int32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    int32_t y = s_sum[lane];                               // as many warps as lanes
    const int32_t own = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    *total = __shfl_sync(0xffffffffu, y, 31);
    return x + __shfl_sync(0xffffffffu, y - own, warp);
}
static_assert(kOne == 1024, "as many warps as lanes");

// Bits of the pages that the rows name, from a warp for each 256 entries
__device__ __forceinline__ void one_mark(const RowArgs& a, One& s, const int32_t* s_len) {
    const int lane = threadIdx.x & 31;
    const int chunks = (a.width + kChunk - 1) / kChunk;
    for (int w = threadIdx.x >> 5; w < a.R * chunks; w += kOne / 32) {
        const int r = w / chunks, c = (w - r * chunks) * kChunk;
        const Row row = row_of(a, s_len[r]);
        int32_t flags = c == 0 ? row.flags : 0;
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int j = c + e * 32 + lane;
            if (j >= row.used) break;
            const int32_t id = a.table[(int64_t)r * a.width + j];
            if ((uint32_t)id < (uint32_t)a.n_pages) atomicOr(s.old_bits + (id >> 5), 1u << (id & 31));
            else flags |= BIT_ID;
        }
        if (flags) atomicOr(&s.flags, flags);
    }
}
__device__ __forceinline__ void one_clear(const RowArgs& a, One& s) {
    for (int i = threadIdx.x; i < a.n_pages; i += kOne) s.ref[i] = 0;
    for (int i = threadIdx.x; i < kOnePages / 32; i += kOne) s.old_bits[i] = s.new_bits[i] = 0;
    if (threadIdx.x == 0) s.flags = s.longest = 0;
}

__global__ void __launch_bounds__(kOne) k_fork_one(const RowArgs a) {
    __shared__ One s;
    extern __shared__ int32_t s_rows[];                    // [R] lengths, [R] lowest new rows
    int32_t *s_len = s_rows, *s_first = s_rows + a.R;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    int32_t parent[kOneRows / kOne];
#pragma unroll
    for (int x = 0; x < kOneRows / kOne; ++x) parent[x] = tid + x * kOne < a.N ? parent_of(a, tid + x * kOne) : -1;
    for (int i = tid; i < a.R; i += kOne) {
        s_len[i] = a.len[i];
        s_first[i] = INT32_MAX;
    }
    one_clear(a, s);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kOneRows / kOne; ++x)
        if (parent[x] >= 0) atomicMin(s_first + parent[x], tid + x * kOne);
    one_mark(a, s, s_len);
    __syncthreads();
    // ---- lengths, and the pages taken anew
    int32_t need_all = 0;
#pragma unroll
    for (int x = 0; x < kOneRows / kOne; ++x) {
        if (x * kOne >= a.N) break;
        const int i = tid + x * kOne, p = parent[x];
        Row row = {};
        if (p >= 0) row = row_of(a, s_len[p]);
        const bool need = row.rest > 0 && s_first[p] != i;
        int32_t all;
        const int32_t k = need_all + one_sum(need, s.sum, &all) - need;
        need_all += all;
        if (need) {
            const bool have = k < a.n_free;
            int32_t page = have ? a.free_list[k] : -1, from = a.table[(int64_t)p * a.width + row.full];
            if (have && (uint32_t)page >= (uint32_t)a.n_pages) {
                page = -1;
                atomicOr(&s.flags, BIT_ID);
            }
            if ((uint32_t)from >= (uint32_t)a.n_pages) from = -1;
            a.out[(int64_t)i * a.width + row.full] = page;
            if (page >= 0) {
                atomicAdd(s.ref + page, 1);
                atomicOr(s.new_bits + (page >> 5), 1u << (page & 31));
            } else {
                row.len -= row.rest;
            }
            if (have) {
                a.copies[3 * k] = from;
                a.copies[3 * k + 1] = page;
                a.copies[3 * k + 2] = row.rest;
            }
        }
        if (i < a.N) a.len_out[i] = row.len;
        if (row.len) atomicMax(&s.longest, row.len);
    }
    // ---- the new rows but for those pages
    const int chunks = (a.width + kChunk - 1) / kChunk;
    for (int w = tid >> 5; w < a.N * chunks; w += kOne / 32) {
        const int i = w / chunks, c = (w - i * chunks) * kChunk;
        const int32_t p = parent_of(a, i);
        Row row = {};
        bool fresh = false;
        if (p >= 0) {
            row = row_of(a, s_len[p]);
            fresh = row.rest > 0 && s_first[p] != i;
        }
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int j = c + e * 32 + lane;
            if (j >= a.width) break;
            if (fresh && j == row.full) continue;
            int32_t id = j < row.used ? a.table[(int64_t)p * a.width + j] : -1;
            if ((uint32_t)id >= (uint32_t)a.n_pages) id = -1;
            a.out[(int64_t)i * a.width + j] = id;
            if (id >= 0) {
                atomicAdd(s.ref + id, 1);
                atomicOr(s.new_bits + (id >> 5), 1u << (id & 31));
            }
        }
    }
    __syncthreads();
    // ---- counts and the free list
    const int taken = min(need_all, a.n_free), left = a.n_free - taken;
    for (int i = tid; i < a.n_pages; i += kOne) a.ref[i] = s.ref[i];
    for (int i = tid; i < min(left, a.n_pages); i += kOne) a.free_out[i] = a.free_list[taken + i];
    const uint32_t back = tid < kOnePages / 32 ? s.old_bits[tid] & ~s.new_bits[tid] : 0;
    int32_t all;
    int32_t k = left + one_sum(__popc(back), s.sum, &all) - __popc(back);
    for (uint32_t x = back; x; x &= x - 1, ++k)
        if (k < a.n_pages) a.free_out[k] = tid * 32 + __ffs(x) - 1;
    if (tid == 0) {
        a.info[0] = taken;
        a.info[1] = min(left + all, a.n_pages);
        a.info[2] = s.flags | (need_all > a.n_free ? BIT_FREE : 0);
        a.info[3] = s.longest;
    }
}

__global__ void __launch_bounds__(kOne) k_compact_one(const RowArgs a) {
    __shared__ One s;
    __shared__ int32_t s_before[kOnePages / 32];           // pages in use before a word
    extern __shared__ int32_t s_rows[];                    // [R] lengths, [n_pages / 2] where pages move
    int32_t *s_len = s_rows, *s_to = s_rows + a.R;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < a.R; i += kOne) s_len[i] = a.len[i];
    one_clear(a, s);
    __syncthreads();
    one_mark(a, s, s_len);
    __syncthreads();
    const uint32_t word = tid < kOnePages / 32 ? s.old_bits[tid] : 0;
    int32_t live;
    const int32_t before = one_sum(__popc(word), s.sum, &live) - __popc(word);
    if (tid < kOnePages / 32) s_before[tid] = before;
    __syncthreads();
    // pages in use below id
    auto rank = [&](int id) { return s_before[id >> 5] + __popc(s.old_bits[id >> 5] & ((1u << (id & 31)) - 1)); };
    const int32_t stay = live < kOnePages ? rank(live) : live;             // in use below `live`
    for (int id = tid; id < a.n_pages; id += kOne) {
        const bool used = (s.old_bits[id >> 5] >> (id & 31)) & 1;
        if (used && id >= live) {                          // the k-th that moves
            const int k = rank(id) - stay;
            a.copies[3 * k] = id;
            a.copies[3 * k + 2] = (int32_t)a.ps;
        } else if (!used && id < live) {                   // the k-th that is free
            const int k = id - rank(id);
            a.copies[3 * k + 1] = id;
            s_to[k] = id;
        }
        if (id >= live) a.free_out[id - live] = id;
    }
    __syncthreads();
    const int chunks = (a.width + kChunk - 1) / kChunk;
    for (int w = tid >> 5; w < a.R * chunks; w += kOne / 32) {
        const int r = w / chunks, c = (w - r * chunks) * kChunk;
        const Row row = row_of(a, s_len[r]);
#pragma unroll
        for (int e = 0; e < kEntries; ++e) {
            const int j = c + e * 32 + lane;
            if (j >= a.width) break;
            int32_t id = j < row.used ? a.table[(int64_t)r * a.width + j] : -1;
            if ((uint32_t)id >= (uint32_t)a.n_pages) id = -1;
            if (id >= live) id = s_to[rank(id) - stay];
            a.out[(int64_t)r * a.width + j] = id;
            if (id >= 0) atomicAdd(s.ref + id, 1);
        }
    }
    __syncthreads();
    for (int i = tid; i < a.n_pages; i += kOne) a.ref[i] = s.ref[i];
    if (tid == 0) {
        a.info[0] = live - stay;
        a.info[1] = a.n_pages - live;
        a.info[2] = s.flags;
        a.info[3] = live;
    }
}

// One block does all passes where each of its threads has a few entries.
bool one_block(const RowArgs& a) {
    return ((int64_t)a.R + a.N) * a.width <= 8 * kOne && a.n_pages <= kOnePages && a.n_free <= kOnePages && a.N <= kOneRows && a.R <= kOneRows;
}
int blocks_for(int64_t items, int64_t each) { return (int)std::min<int64_t>(std::max<int64_t>((items + each - 1) / each, 1), 2048); }

void lay_out_work(RowArgs& a, int32_t* work, int32_t R) {
    a.words = (a.n_pages + 31) / 32;
    a.word = work;
    a.old_bits = reinterpret_cast<uint32_t*>(work + W_WORDS);
    a.new_bits = a.old_bits + a.words;
    a.first = work + W_WORDS + 2 * (int64_t)a.words;
    a.place = a.first + R;
}

// Every block of a pass counts for itself what lies before its part, so that work grows with the square of the new rows and of the
// bit map's words: 2^20 rows and 2^26 pages are tenths of a second.  Entries of a row are counted in 32 bits, 256 at a time.
constexpr int kMaxNew = 1 << 20, kMaxPages = 1 << 26, kMaxWidth = 1 << 30;

int check_rows(const char* who, const void* table, int table_stride, const void* len, int R, int page_size, int n_pages) {
    if (R < 0 || table_stride < 1 || page_size < 1 || page_size > 65536 || n_pages < 1 ||
        (int64_t)n_pages * page_size > INT32_MAX)
        return op_fail(SD_ERR_INVALID_ARG, "%s: R %d, table_stride %d, page_size %d, n_pages %d", who, R, table_stride,
                       page_size, n_pages);
    if (table_stride > kMaxWidth || n_pages > kMaxPages)
        return op_fail(SD_ERR_UNSUPPORTED, "%s: table_stride %d (up to 2^30), n_pages %d (up to 2^26)", who, table_stride, n_pages);
    if (R > 0 && (!table || !len)) return op_fail(SD_ERR_INVALID_ARG, "%s: table_dev or len_dev is NULL", who);
    return SD_OK;
}

}  // namespace
}  // namespace sd

extern "C" {

int64_t sd_page_work(int32_t R, int32_t N, int32_t n_pages) {
    if (R < 0 || N < 0 || n_pages < 1) return 0;
    return sd::W_WORDS + 2 * (((int64_t)n_pages + 31) / 32) + R + n_pages;
}

int sd_page_fork(const int32_t* table_dev, int32_t table_stride, const int32_t* len_dev, int32_t R,
                 const int32_t* parent_dev, int32_t N, const int32_t* free_dev, int32_t n_free, int32_t page_size,
                 int32_t n_pages, int32_t* table_out_dev, int32_t* len_out_dev, int32_t* copy_dev, int32_t* ref_dev,
                 int32_t* free_out_dev, int32_t* info_dev, int32_t* work_dev, void* stream) {
    using namespace sd;
    static const char* who = "sd_page_fork";
    if (int rc = check_rows(who, table_dev, table_stride, len_dev, R, page_size, n_pages)) return rc;
    if (N < 0 || n_free < 0) return op_fail(SD_ERR_INVALID_ARG, "%s: N %d, n_free %d", who, N, n_free);
    if (N > kMaxNew) return op_fail(SD_ERR_UNSUPPORTED, "%s: N %d (up to 2^20)", who, N);
    if (N > 0 && (!parent_dev || !table_out_dev || !len_out_dev || !copy_dev))
        return op_fail(SD_ERR_INVALID_ARG, "%s: parent_dev, table_out_dev, len_out_dev or copy_dev is NULL", who);
    if (n_free > 0 && !free_dev) return op_fail(SD_ERR_INVALID_ARG, "%s: free_dev is NULL", who);
    if (!ref_dev || !free_out_dev || !info_dev || !work_dev)
        return op_fail(SD_ERR_INVALID_ARG, "%s: ref_dev, free_out_dev, info_dev or work_dev is NULL", who);
    if (reinterpret_cast<uintptr_t>(work_dev) & 7)
        return op_fail(SD_ERR_INVALID_ARG, "%s: work_dev is not 8-byte aligned", who);
    if (R > 0 && N > 0 && table_out_dev == table_dev)
        return op_fail(SD_ERR_INVALID_ARG, "%s: table_out_dev is table_dev", who);
    RowArgs a = {};
    a.table = table_dev; a.len = len_dev; a.parent = parent_dev; a.free_list = free_dev; a.out = table_out_dev;
    a.len_out = len_out_dev; a.copies = copy_dev; a.ref = ref_dev; a.free_out = free_out_dev; a.info = info_dev;
    a.R = R; a.N = N; a.n_free = n_free; a.width = table_stride; a.n_pages = n_pages; a.ps = (uint32_t)page_size;
    a.by_ps = FastDiv((uint32_t)page_size);
    lay_out_work(a, work_dev, R);
    // without new rows there is no parent to look at, but the old ones' lowest rows are still to be cleared
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (one_block(a)) {
        e = launch_k(k_fork_one, dim3(1), dim3(kOne), sizeof(int32_t) * 2 * a.R, st, a);
    } else {
        const int64_t chunks = ((int64_t)a.width + kChunk - 1) / kChunk;
        const int takers = std::max((N + kThreads - 1) / kThreads, 1);
        e = launch_k(k_rows_clear, dim3(blocks_for(std::max(a.n_pages, R), 4 * kThreads)), dim3(kThreads), 0, st, a);
        if (e == cudaSuccess)
            e = launch_k(k_rows_mark, dim3(blocks_for(std::max<int64_t>(R * chunks, (N + 31) / 32), kThreads / 32)), dim3(kThreads), 0, st, a);
        if (e == cudaSuccess)
            e = launch_k(k_fork_fill, dim3(takers + blocks_for(N * chunks, kThreads / 32)), dim3(kThreads), 0, st, a, takers);
        if (e == cudaSuccess)
            e = launch_k(k_fork_release, dim3((a.words + kWords - 1) / kWords), dim3(kThreads), 0, st, a);
    }
    if (e != cudaSuccess) return op_fail(SD_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return SD_OK;
}

int sd_page_compact(const int32_t* table_dev, int32_t table_stride, const int32_t* len_dev, int32_t R,
                    int32_t page_size, int32_t n_pages, int32_t* table_out_dev, int32_t* copy_dev, int32_t* ref_dev,
                    int32_t* free_out_dev, int32_t* info_dev, int32_t* work_dev, void* stream) {
    using namespace sd;
    static const char* who = "sd_page_compact";
    if (int rc = check_rows(who, table_dev, table_stride, len_dev, R, page_size, n_pages)) return rc;
    if (R > 0 && !table_out_dev) return op_fail(SD_ERR_INVALID_ARG, "%s: table_out_dev is NULL", who);
    if ((n_pages > 1 && !copy_dev) || !ref_dev || !free_out_dev || !info_dev || !work_dev)
        return op_fail(SD_ERR_INVALID_ARG, "%s: copy_dev, ref_dev, free_out_dev, info_dev or work_dev is NULL", who);
    if (reinterpret_cast<uintptr_t>(work_dev) & 7)
        return op_fail(SD_ERR_INVALID_ARG, "%s: work_dev is not 8-byte aligned", who);
    RowArgs a = {};
    a.table = table_dev; a.len = len_dev; a.out = table_out_dev; a.copies = copy_dev; a.ref = ref_dev;
    a.free_out = free_out_dev; a.info = info_dev; a.R = R; a.width = table_stride; a.n_pages = n_pages;
    a.ps = (uint32_t)page_size; a.by_ps = FastDiv((uint32_t)page_size);
    lay_out_work(a, work_dev, R);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (one_block(a)) {
        e = launch_k(k_compact_one, dim3(1), dim3(kOne), sizeof(int32_t) * (a.R + a.n_pages / 2), st, a);
    } else {
        const int64_t chunks = ((int64_t)a.width + kChunk - 1) / kChunk;
        e = launch_k(k_rows_clear, dim3(blocks_for(a.n_pages, 4 * kThreads)), dim3(kThreads), 0, st, a);
        if (e == cudaSuccess) e = launch_k(k_rows_mark, dim3(blocks_for(R * chunks, kThreads / 32)), dim3(kThreads), 0, st, a);
        if (e == cudaSuccess)
            e = launch_k(k_compact_places, dim3((a.words + kWords - 1) / kWords), dim3(kThreads), 0, st, a);
        if (e == cudaSuccess) e = launch_k(k_compact_rename, dim3(blocks_for(R * chunks, kThreads / 32)), dim3(kThreads), 0, st, a);
    }
    if (e != cudaSuccess) return op_fail(SD_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return SD_OK;
}

}  // extern "C"
