// The common part of attention for groups of requests that share their first pages: one pass over a group's
// common keys and values for the queries of all its requests, on the 5th-generation tensor cores.
//
// An item is (group, kv head, up to 256 query rows), a row being (request, head of the kv head's group), against all
// of the group's common positions in tiles of 128.  The tiles of all items, laid end to end, are dealt
// evenly to one block per SM; a block writes, for each of its parts of an item, every row's partial
// result (unnormalised output, maximum, sum).  The next kernel (k_attend_own.cu) joins them with the requests' own positions.
//
//   S_i = Q_i K_j^T     P_i = exp2(S_i scale log2(e) - m_i), over S_i's columns     O_i += P_i V_j
//
// Two warpgroups hold a thread per row.  Above 128 rows each has 128 of them, against every tile; up to
// 128 rows both have the same rows and take the tiles in turn, one forming P while the tensor cores work
// on the other's, and the first joins the two halves at the end.
//
// Queries are written to shared memory by the warpgroups themselves, whatever their type and stride.  Where the
// keys' type does not hold them (fp32, or the other 16-bit type) they enter as two parts, rows scaled by
// a power of two, and so do the probabilities: three to four times the products, with 128 rows to an item.
//
// Measured: 8 groups of 2 to 32 requests behind 1000 to 16000 positions, 64 query and 8 kv heads of 128, bf16, 193 MB
// read: 48 us of the call's 79, 4.0 TB/s and 27 % of the tensor pipe (the requests each by itself 105 us, mostly from L2).  64 rollouts
// behind 2000 positions, 16 heads of 64, fp32: 20 of 29 us (66 each by itself).  What bounds it: the first 9000 cycles, until
// a block knows its piece and the first keys are there, and the last block's record; in between a tile passes in
// 1500 to 2000 cycles, the time from scores to exponentials to products.
#include <algorithm>

#include "tc_dev.cuh"

namespace sd {
namespace {

constexpr int kM = 128, kN = 128;                     // rows and positions of a tile
constexpr int kSoftWarps = 8, kThreads = 32 * (kSoftWarps + 4);    // 2 softmax warpgroups; products, two loaders, pieces
constexpr int kMmaWarp = kSoftWarps, kKeyWarp = kSoftWarps + 1, kValueWarp = kSoftWarps + 2, kItemWarp = kSoftWarps + 3;
constexpr int kSoftRegs = 216, kOtherRegs = 72;
static_assert(256 * kSoftRegs + 128 * kOtherRegs <= 384 * 168, "the shares exceed what the block was launched with");
constexpr float kSlack = 8.f;                         // log2 of the growth that moves the reference
constexpr float kFar = 0x1p20f;                       // exponents from which the reference is subtracted before scaling
constexpr int kMasks = 8;                             // tiles whose masks are kept: more than the ring holds

struct alignas(128) SharedArgs {
    CUtensorMap k, v;
    AttendArgs a;
    const int32_t *group, *shared;
    int32_t n_groups, box;
    int64_t worth;                                    // key and value rows that sharing has to save
};

template <int HD>
struct Cfg {
    static constexpr int kPanel = kN * 128;                       // 128 rows of 64 elements, 128-byte swizzle
    static constexpr int kTileBytes = kPanel * (HD / 64);         // a Q, K or V tile
    static constexpr int kStages = HD == 128 ? 5 : 9;             // K and V tiles in flight (odd: K and V take turns)
    static constexpr int kSmem = (2 + kStages) * kTileBytes + 1024;
    static constexpr uint32_t kO = 256;                           // tensor memory: S0, S1, O0, O1
};

// A group as the kernels see it
struct Group {
    int r0, size, pages, tiles, items;                            // tiles 0: nothing is shared
};
__device__ __forceinline__ Group group_of(const SharedArgs& t, int x, int rows) {
    const AttendArgs& a = t.a;
    const int G = a.H / a.Hkv;
    const int r0 = __ldcg(t.group + x), end = __ldcg(t.group + x + 1), pages = __ldcg(t.shared + x);
    Group p;
    p.r0 = min(max(r0, 0), a.B);
    p.size = max(min(max(end, 0), a.B) - p.r0, 0);
    p.pages = min(max(pages, 0), a.table_stride);
    const int64_t pos = min((int64_t)p.pages * a.by_ps.d, (int64_t)a.max_len);
    p.tiles = p.size > 1 ? (int)((pos + kN - 1) / kN) : 0;
    p.items = a.Hkv * ((p.size * G + rows - 1) / rows);           // the query rows of all requests are at most kSharedRows
    return p;
}
// All groups, as a warp sees them: up to 32 a lane each, more by their number from memory.
struct Groups32 {
    Group mine;
    bool few;
    int64_t first, T;                                             // tiles before the lane's group; of all (0: sharing does not pay)
};
// A group's tiles, with the empty ones before each item
__device__ __forceinline__ int64_t span(const Group& p) { return p.tiles ? (int64_t)(p.tiles + kShareLead) * p.items : 0; }
// By the kOthers threads behind the softmax warps; s_sum has two words for each warp.
//
// Sharing pays if it saves `worth` rows of keys and values, and if no request has so many positions of its own that the
// one block that takes them (some 40 GB/s) ends behind the time that all others need for what is saved (some 5 TB/s).
constexpr int kOthers = kThreads - 32 * kSoftWarps;
__device__ __forceinline__ void others_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kOthers) : "memory"); }
__device__ __forceinline__ Groups32 groups_of(const SharedArgs& t, int rows, int64_t* s_sum) {
    constexpr int threads = kOthers;
    const int tid = threadIdx.x - 32 * kSoftWarps, lane = tid & 31, warp = tid >> 5;
    int len0 = tid < t.a.B ? __ldcg(t.a.len + tid) : 0;           // asked for beside the groups
    Groups32 g = {};
    g.few = t.n_groups <= 32;
    int64_t tiles = 0, saved = 0;
    auto saves = [&](const Group& p) { return p.tiles ? (int64_t)(p.size - 1) * p.pages * t.a.by_ps.d * t.a.Hkv : 0; };
    if (g.few) {
        if (lane < t.n_groups) g.mine = group_of(t, lane, rows);
        tiles = span(g.mine);
        saved = saves(g.mine);
        int64_t at = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += y;
            saved += __shfl_xor_sync(0xffffffffu, saved, o);
        }
        g.first = at - tiles;
        g.T = __shfl_sync(0xffffffffu, at, 31);
        // the most positions that a request has of its own: a thread for each request
        int most = 0;
        for (int b = tid; b - lane < t.a.B; b += threads) {
            const int len = b < t.a.B ? min(max(b == tid ? len0 : __ldcg(t.a.len + b), 0), t.a.max_len) : 0;
            int64_t skip = 0;
            for (int x = 0; x < t.n_groups; ++x) {
                const int r0 = __shfl_sync(0xffffffffu, g.mine.r0, x), size = __shfl_sync(0xffffffffu, g.mine.size, x);
                const int pages = __shfl_sync(0xffffffffu, g.mine.tiles ? g.mine.pages : 0, x);
                if (b >= r0 && b < r0 + size) skip = (int64_t)pages * t.a.by_ps.d;
            }
            most = max(most, (int)max(len - skip, (int64_t)0));
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) s_sum[warp] = most;
        others_sync();
        for (int w = 0; w < threads / 32; ++w) most = max(most, (int)s_sum[w]);
        if (t.worth > 0 && saved < 128 * (int64_t)most) g.T = 0;
    } else {
        for (int x = tid; x < t.n_groups; x += threads) {
            const Group p = group_of(t, x, rows);
            tiles += span(p);
            saved += saves(p);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
            saved += __shfl_xor_sync(0xffffffffu, saved, o);
        }
        if (lane == 0) {
            s_sum[2 * warp] = tiles;
            s_sum[2 * warp + 1] = saved;
        }
        others_sync();
        saved = 0;
        for (int w = 0; w < threads / 32; ++w) {
            g.T += s_sum[2 * w];
            saved += s_sum[2 * w + 1];
        }
    }
    if (saved < t.worth) g.T = 0;
    return g;
}
__device__ __forceinline__ Group group_at(const SharedArgs& t, const Groups32& g, int x, int rows) {
    if (!g.few) return group_of(t, x, rows);
    Group p;
    p.r0 = __shfl_sync(0xffffffffu, g.mine.r0, x);
    p.size = __shfl_sync(0xffffffffu, g.mine.size, x);
    p.pages = __shfl_sync(0xffffffffu, g.mine.pages, x);
    p.tiles = __shfl_sync(0xffffffffu, g.mine.tiles, x);
    p.items = __shfl_sync(0xffffffffu, g.mine.items, x);
    return p;
}
__device__ __forceinline__ int64_t tiles_of_block(int64_t T, int blocks) { return max(quot(T + blocks - 1, blocks), (int64_t)1); }

// A piece of work of a block: tiles [i0, i0 + tiles) of an item; tiles 0: no more
struct Item {
    int r0, g, i0, tiles, pages, m0, rows, size;
};
constexpr int kItems = 3;                                         // prepared ahead

// O += P V: P of 32 positions lies in the first 16 columns of their scores (its low part in the other 16)
template <int K, int kEnd>
__device__ __forceinline__ void chunk_steps(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (K < kEnd) {
        mma_ts<(K / 2) * 32 + (K % 2) * 8, K * (2048 >> 4)>(d, a, b, idesc, acc);
        chunk_steps<K + 1, kEnd>(d, a, b, idesc, 1);
    }
}

template <int HD, bool BF, bool LOW>
__global__ void __launch_bounds__(kThreads, 1) k_attend_shared(const __grid_constant__ SharedArgs t) {
    using C = Cfg<HD>;
    constexpr int kSt = C::kStages;
    constexpr int kRows = LOW ? kM : 2 * kM;                      // of an item
    constexpr float kShift = BF ? 0.f : 7.f;
    constexpr uint32_t kType = BF ? 1u : 0u;
    constexpr uint32_t kIdescS = (1u << 4) | (kType << 7) | (kType << 10) | ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
    constexpr uint32_t kIdescO = (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
    extern __shared__ unsigned char smraw[];
    __shared__ __align__(8) unsigned long long s_full[kSt], s_empty[kSt], s_qfull, s_qempty, s_sfull[2], s_pfull[2][2], s_ofull[2], s_half, s_joined, s_never, s_dry, s_ifull[kItems], s_iempty[kItems];
    __shared__ Item s_item[kItems];
    __shared__ uint32_t s_mask[kMasks][4], s_tmem;
    __shared__ int2 s_box[2][32];
    __shared__ __align__(8) float s_row[2 * kM];
    // a row's scale, from the first warpgroup to the second, and later its maximum, and its sum, back
    float *s_scale = s_row, *s_top = s_row, *s_sum = s_row + kM;
    int64_t* s_red = reinterpret_cast<int64_t*>(s_box);           // the loaders' from the first piece on, which follows the sums
    __shared__ int s_bad;
    const AttendArgs& a = t.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sm = (smem_u32(smraw) + 1023u) & ~1023u;
    const uint32_t ring = sm + 2 * C::kTileBytes;
    const int G = a.H / a.Hkv, ps = (int)a.by_ps.d;
    volatile int* bad = &s_bad;
    pdl_trigger();

    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int s = 0; s < kSt; ++s) {
            mb_init(smem_u32(&s_full[s]), 1);
            mb_init(smem_u32(&s_empty[s]), 1);
        }
        mb_init(smem_u32(&s_qfull), LOW ? kSoftWarps : 1);
        mb_init(smem_u32(&s_qempty), 1);
        mb_init(smem_u32(&s_half), kM / 32);
        mb_init(smem_u32(&s_joined), kM / 32);
        mb_init(smem_u32(&s_never), 1);
        mb_init(smem_u32(&s_dry), kSoftWarps);
        for (int i = 0; i < kItems; ++i) {
            mb_init(smem_u32(&s_ifull[i]), 1);
            mb_init(smem_u32(&s_iempty[i]), kSoftWarps + 3);
        }
        for (int i = 0; i < 2; ++i) {
            mb_init(smem_u32(&s_sfull[i]), 1);
            mb_init(smem_u32(&s_pfull[i][0]), kM / 32);
            mb_init(smem_u32(&s_pfull[i][1]), kM / 32);
            mb_init(smem_u32(&s_ofull[i]), 1);
        }
        s_bad = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tm_before();
    __syncthreads();
    tm_after();
    const uint32_t tmem = s_tmem;

    // The pieces of this block in turn; by a whole warp, or by the one thread that issues products
    uint32_t n_item = 0;
    auto take = [&](Item& it, bool alone) -> bool {
        const uint32_t slot = n_item % kItems, parity = (n_item / kItems) & 1;
        ++n_item;
        if (!(alone ? mb_wait(smem_u32(&s_ifull[slot]), parity, bad) : warp_wait(smem_u32(&s_ifull[slot]), parity, bad))) return false;
        it = s_item[slot];
        if (!alone) __syncwarp();
        if (alone || lane == 0) mb_arrive(smem_u32(&s_iempty[slot]));
        return it.tiles > 0;
    };
    Item it;

    pdl_wait();
    if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // ---------------------------------------------------- groups, their tiles, and whether it is worth it
        const Groups32 groups = groups_of(t, kRows, s_red);
        const int64_t T = groups.T, per = tiles_of_block(T, gridDim.x);
        const int64_t t_begin = blockIdx.x * per, t_end = min(T, t_begin + per);
        if (warp == kKeyWarp || warp == kValueWarp) {
            // ------------------------------------------------ loads: a tile's keys (entry 2 j of the ring) or values (2 j + 1)
            const int op = warp - kKeyWarp;
            uint32_t n = 0, last = 0;                              // tiles of the items before; entries up to this warp's last
            bool ok = true;
            const int box = t.box, groups = kN / box;
            auto lookup = [&](const Item& it, int j, int k) -> int {   // page of this lane's box, -1 without one
                const int64_t pos = (int64_t)(it.i0 + j) * kN + (k * 32 + lane) * box;
                if (j >= it.tiles || k * 32 + lane >= groups || pos >= min((int64_t)it.pages * ps, (int64_t)a.max_len)) return -1;
                return __ldcg(a.table + (int64_t)it.r0 * a.table_stride + a.by_ps.div((uint32_t)pos));
            };
            Item next;
            bool have_next = take(next, false);
            int next_id = have_next ? lookup(next, 0, 0) : -1;
            while (ok && have_next) {
                it = next;
                int ahead = next_id;
                // the next piece and its first pages: not waited for before this piece's last tile
                have_next = take(next, false);
                next_id = have_next ? lookup(next, 0, 0) : -1;
                for (int j = 0; j < it.tiles && ok; ++j) {
                    const int first = (it.i0 + j) * kN;
                    const int id0 = ahead;
                    ahead = lookup(it, j + 1, 0);                  // a tile ahead: not waited for here
                    const uint32_t e = 2 * (n + j) + op, slot = e % kSt, turn = e / kSt;
                    if (turn > 0) ok = warp_wait(smem_u32(&s_empty[slot]), (turn - 1) & 1, bad);
                    if (!ok) break;
                    if (a.stall && it.i0 == 0 && it.g == 0) ok = warp_wait(smem_u32(&s_never), 0, bad, a.stall);
                    if (!ok) break;
                    last = e + 1;
                    const uint32_t mb = smem_u32(&s_full[slot]), dst = ring + slot * C::kTileBytes;
                    uint32_t* mask = s_mask[(n + j) % kMasks];
                    if (op == 0 && lane < 4) mask[lane] = 0;
                    __syncwarp();
#pragma unroll 1
                    for (int k = 0; k * 32 < groups; ++k) {
                        int id = k == 0 ? id0 : lookup(it, j, k);
                        if ((uint32_t)id >= (uint32_t)a.n_pages) id = -1;
                        const int row = (k * 32 + lane) * box, pos = first + row;
                        const int in = pos - (int)(a.by_ps.div((uint32_t)pos) * a.by_ps.d);
                        if (op == 0 && id >= 0)
                            for (int r = row; r < row + box; r += 32)
                                atomicOr(mask + (r >> 5), box >= 32 ? 0xffffffffu : ((1u << box) - 1) << (r & 31));
                        const uint32_t have = __ballot_sync(0xffffffffu, id >= 0);
                        const int boxes = min(32, groups - k * 32);
                        if (op == 1) {
                            // values that are not there: 0 x anything must be 0
                            for (uint32_t none = ~have & (0xffffffffu >> (32 - boxes)); none; none &= none - 1) {
                                const int r0 = (k * 32 + __ffs(none) - 1) * box;
                                for (int y = lane; y < box * 8 * (HD / 64); y += 32) {
                                    const int part = y / (box * 8), z = y - part * box * 8;
                                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + part * C::kPanel + r0 * 128 + z * 16), "r"(0) : "memory");
                                }
                            }
                            if (have != 0xffffffffu >> (32 - boxes)) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        }
                        s_box[op][lane] = make_int2(id, in);
                        __syncwarp();
                        if (elect_one()) {
                            if (have) mb_expect_more(mb, __popc(have) * box * HD * 2);
                            uint32_t to = dst + k * 32 * box * 128;
                            for (int y = 0; y < boxes; ++y, to += box * 128) {
                                const int2 b = s_box[op][y];
                                if (b.x < 0) continue;
#pragma unroll
                                for (int part = 0; part < HD / 64; ++part)
                                    tma4(to + part * C::kPanel, op ? &t.v : &t.k, part * 64, b.y, it.g, b.x, mb);
                            }
                        }
                        __syncwarp();
                    }
                    if (lane == 0) mb_arrive(mb);
                }
                n += it.tiles;
            }
            if (!ok)                                               // bounded: this warp's own copies
                for (uint32_t e = last > kSt ? last - kSt : 0; e < last; ++e) {
                    if ((int)(e & 1) != op) continue;
                    const long long t0 = clock64();
                    while (!mb_try(smem_u32(&s_full[e % kSt]), (e / kSt) & 1) && clock64() - t0 < kWaitClocks) {}
                }
        } else if (warp == kItemWarp) {
            // ---------------------------------------------------- pieces, ahead of everyone
            int x = 0;
            int64_t at = t_begin, base = 0;
            if (t_begin >= T) {
            } else if (groups.few) {
                const int64_t n = span(groups.mine);
                x = __ffs(__ballot_sync(0xffffffffu, n && groups.first <= at && at < groups.first + n)) - 1;
                base = __shfl_sync(0xffffffffu, groups.first, x & 31);
            } else {
                // 32 groups at a time, up to the one that holds the first tile
                for (int x0 = 0; x0 < t.n_groups; x0 += 32) {
                    const Group p = x0 + lane < t.n_groups ? group_of(t, x0 + lane, kRows) : Group{};
                    const int64_t n = span(p);
                    int64_t sum = n;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
                        if (lane >= o) sum += y;
                    }
                    const uint32_t here = __ballot_sync(0xffffffffu, n && base + sum - n <= at && at < base + sum);
                    if (here) {
                        x = x0 + __ffs(here) - 1;
                        base += __shfl_sync(0xffffffffu, sum - n, __ffs(here) - 1);
                        break;
                    }
                    base += __shfl_sync(0xffffffffu, sum, 31);
                }
            }
            Group p = t_begin < T ? group_at(t, groups, x, kRows) : Group{};
            bool ok = true;
            auto make = [&](Item& it) {
                it.tiles = 0;
                while (at < t_end && it.tiles <= 0) {
                    if (at >= base + span(p)) {
                        if (x + 1 >= t.n_groups) break;
                        base += span(p);
                        p = group_at(t, groups, ++x, kRows);
                        continue;
                    }
                    const int pairs = p.items / a.Hkv, width = p.tiles + kShareLead;
                    const int64_t u = quot(at - base, width), u0 = base + u * width, end = min(u0 + width, t_end);
                    it.r0 = p.r0;
                    it.size = p.size;
                    it.pages = p.pages;
                    it.g = (int)u / pairs;
                    it.m0 = ((int)u - it.g * pairs) * kRows;
                    it.rows = min(kRows, p.size * G - it.m0);
                    it.i0 = (int)max(at - u0 - kShareLead, (int64_t)0);
                    it.tiles = (int)(end - u0) - kShareLead - it.i0;      // none: empty ones alone in this block
                    at = end;
                }
                it.tiles = max(it.tiles, 0);
            };
            auto post = [&](uint32_t n, const Item& it) {
                const uint32_t slot = n % kItems;
                if (n >= kItems) ok = warp_wait(smem_u32(&s_iempty[slot]), (n / kItems - 1) & 1, bad);
                if (ok && lane == 0) {
                    s_item[slot] = it;
                    mb_arrive(smem_u32(&s_ifull[slot]));
                }
                __syncwarp();
            };
            Item later;
            make(it);
            post(0, it);
            // a piece is known one piece before its queries are loaded: its keys need not wait for them
            for (uint32_t n = 0; ok && it.tiles; ++n, it = later) {
                make(later);
                post(n + 1, later);
                if (!ok) break;
                if constexpr (LOW) {
                    // its queries on their way: what is not in L2 waits behind everything that the loaders have asked for
                    for (int r = lane; r < it.rows; r += 32) {
                        const int row = it.m0 + r, b = it.r0 + row / G, bytes = a.dtype == SD_F32 ? 4 : 2;
                        const char* q = static_cast<const char*>(a.q) + (b * a.q_batch + (int64_t)(it.g * G + row % G) * HD) * bytes;
                        for (int x = 0; x < HD * bytes; x += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + x));
                    }
                } else {
                    // its queries to shared memory, as soon as the last scores of the piece before are formed
                    if (n > 0) ok = warp_wait(smem_u32(&s_qempty), (n - 1) & 1, bad);
                    if (!ok) break;
                    // (rows that are not there keep what the memory holds: no other row sees it)
                    constexpr int kStep = 32 / (HD / 8);           // rows of a turn
                    const int col = lane % (HD / 8), r0 = lane / (HD / 8), row = it.m0 + r0;
                    int qi = row / G, hh = row - qi * G;
                    const uint16_t* q = static_cast<const uint16_t*>(a.q) + (int64_t)(it.g * G) * HD + col * 8;
                    const uint32_t dst = sm + (col >> 3) * C::kPanel;
#pragma unroll 4
                    for (int r = r0; r < it.rows; r += kStep) {
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                     ::"r"(dst + (r >> 7) * C::kTileBytes + (r & 127) * 128 + (((col & 7) ^ (r & 7)) << 4)),
                                     "l"(q + (it.r0 + qi) * a.q_batch + hh * HD) : "memory");
                        for (hh += kStep; hh >= G; hh -= G) ++qi;
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mb_arrive(smem_u32(&s_qfull));
                }
            }
            // which kernel follows, and what it needs to know of each request
            if (blockIdx.x == 0 && lane == 0) *a.shared = T > 0;
            for (int b = blockIdx.x; b < a.B && T; b += gridDim.x) {
                SharedRow d = {};
                int64_t start = 0;
                for (int x0 = 0; x0 < t.n_groups; x0 += 32) {
                    Group q = groups.mine;
                    int64_t first = groups.first;
                    if (!groups.few) {
                        q = x0 + lane < t.n_groups ? group_of(t, x0 + lane, kRows) : Group{};
                        int64_t sum = span(q);
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
                            if (lane >= o) sum += y;
                        }
                        first = start + sum - span(q);
                        start += __shfl_sync(0xffffffffu, sum, 31);
                    }
                    const uint32_t here = __ballot_sync(0xffffffffu, q.tiles && b >= q.r0 && b < q.r0 + q.size);
                    if (!here) continue;
                    const int x = __ffs(here) - 1;
                    d.skip = __shfl_sync(0xffffffffu, q.pages, x);
                    d.r0 = __shfl_sync(0xffffffffu, q.r0, x);
                    d.size = __shfl_sync(0xffffffffu, q.size, x);
                    d.tiles = __shfl_sync(0xffffffffu, q.tiles, x);
                    d.base = __shfl_sync(0xffffffffu, first, x);
                    break;
                }
                d.rows = kRows;
                d.per = per;
                if (lane == 0) a.desc[b] = d;
            }
        } else if (warp == kMmaWarp) {
            if (elect_one()) {
                // ------------------------------------------------ products
                const uint64_t qdesc = sdesc(sm, 16), kdesc = sdesc(ring, 16), vdesc = sdesc(ring, C::kPanel);
                constexpr uint32_t kTile16 = C::kTileBytes >> 4;
                uint32_t n = 0, nq = 0, np = 0, no = 0;                // np, no: a bit for each tile's phase
                bool ok = true, any = false;
                auto scores = [&](int i, int q, uint32_t stage) {  // S_i of query tile q
                    const uint64_t kd = kdesc + stage * kTile16;
                    score_steps<HD, C::kPanel>(tmem + i * kN, qdesc + (uint32_t)q * kTile16, kd, kIdescS);
                    if constexpr (LOW) score_steps<HD, C::kPanel>(tmem + i * kN, qdesc + kTile16, kd, kIdescS, 1);
                    commit(smem_u32(&s_sfull[i]));
                    any = true;
                };
                auto results = [&](int i, uint32_t stage, bool first) -> bool {
                    const uint64_t vd = vdesc + stage * kTile16;
                    const uint32_t o = tmem + C::kO + i * HD, pr = tmem + i * kN;
                    // the products of P's first half begin while its second half is formed
                    if (!mb_wait(smem_u32(&s_pfull[i][0]), np >> i & 1, bad)) return false;
                    tm_after();
                    chunk_steps<0, kN / 32>(o, pr, vd, kIdescO, !first);
                    if constexpr (LOW) chunk_steps<0, kN / 32>(o, pr + 16, vd, kIdescO, 1);
                    if (!mb_wait(smem_u32(&s_pfull[i][1]), np >> i & 1, bad)) return false;
                    tm_after();
                    chunk_steps<kN / 32, kN / 16>(o, pr, vd, kIdescO, 1);
                    if constexpr (LOW) chunk_steps<kN / 32, kN / 16>(o, pr + 16, vd, kIdescO, 1);
                    np ^= 1u << i;
                    return true;
                };
                auto loaded = [&](uint32_t e) { return mb_wait(smem_u32(&s_full[e % kSt]), (e / kSt) & 1, bad); };
                auto release = [&](uint32_t e) { commit(smem_u32(&s_empty[e % kSt])); };
                ok = mb_wait(smem_u32(&s_dry), 0, bad);            // the dry turn writes where scores go
                tm_after();
                while (ok && take(it, true)) {
                    ok = mb_wait(smem_u32(&s_qfull), nq & 1, bad);
                    if (!ok) break;
                    ++nq;
                    tm_after();
                    const uint32_t e0 = 2 * n;
                    if (!LOW && it.rows > kM) {
                        ok = loaded(e0);
                        if (!ok) break;
                        tm_after();
                        scores(0, 0, e0 % kSt);
                        scores(1, 1, e0 % kSt);
                        release(e0);
                        if (it.tiles == 1) commit(smem_u32(&s_qempty));
                        for (int j = 0; j < it.tiles && ok; ++j) {
                            const uint32_t ev = e0 + 2 * j + 1, ek = ev + 1;
                            const bool more = j + 1 < it.tiles;
                            ok = loaded(ev);
                            for (int i = 0; i < 2 && ok; ++i) {
                                tm_after();
                                ok = results(i, ev % kSt, j == 0);
                                if (!ok) break;
                                if (more) {
                                    if (i == 0) ok = loaded(ek);
                                    if (!ok) break;
                                    tm_after();
                                    scores(i, i, ek % kSt);
                                } else {
                                    commit(smem_u32(&s_ofull[i]));
                                    no ^= 1u << i;
                                }
                            }
                            if (!ok) break;
                            release(ev);
                            if (more) {
                                release(ek);
                                if (j + 2 == it.tiles) commit(smem_u32(&s_qempty));
                            }
                        }
                    } else {
                        for (int j = 0; j < 2 && j < it.tiles && ok; ++j) {
                            ok = loaded(e0 + 2 * j);
                            if (!ok) break;
                            tm_after();
                            scores(j, 0, (e0 + 2 * j) % kSt);
                            release(e0 + 2 * j);
                            if (j + 1 == it.tiles) commit(smem_u32(&s_qempty));
                        }
                        for (int j = 0; j < it.tiles && ok; ++j) {
                            const uint32_t ev = e0 + 2 * j + 1, ek = e0 + 2 * (j + 2);
                            const int i = j & 1;
                            ok = loaded(ev);
                            if (!ok) break;
                            tm_after();
                            ok = results(i, ev % kSt, j < 2);
                            if (!ok) break;
                            release(ev);
                            if (j + 2 < it.tiles) {
                                ok = loaded(ek);
                                if (!ok) break;
                                tm_after();
                                scores(i, 0, ek % kSt);
                                release(ek);
                                if (j + 3 == it.tiles) commit(smem_u32(&s_qempty));
                            } else {
                                commit(smem_u32(&s_ofull[i]));
                                no ^= 1u << i;
                            }
                        }
                    }
                    n += it.tiles;
                }
                if (!ok && any) {                                  // bounded: products in flight
                    commit(smem_u32(&s_ofull[0]));
                    const long long t0 = clock64();
                    while (!mb_try(smem_u32(&s_ofull[0]), no & 1) && clock64() - t0 < kWaitClocks) {}
                }
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // ---------------------------------------------------- softmax: a thread per row
        const int i = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + i * kN, to = tmem + lanes + C::kO;
        const float s0 = fabsf(a.scale) * kLog2e;
        uint32_t ns = 0, no = 0, nq = 0, n = 0, halves = 0;
        bool ok = true;
        // The first turn is a dry one, over whatever tensor memory holds and before any product is issued, beside the other
        // warps' look at the groups: it brings the loop into the instruction cache.  Once the loads of all blocks are
        // under way a miss waits behind them, and the first tile took 9000 cycles.
        bool dry = true;
        auto row_of = [&](const Item& x) { return x.m0 + (!LOW && x.rows > kM ? i * kM : 0) + r; };
        auto row_in = [&](const Item& x) { return (!LOW && x.rows > kM ? i * kM : 0) + r < x.rows; };
        // the length of this thread's row of a piece
        auto ask = [&](const Item& x) { return row_in(x) ? __ldcg(a.len + x.r0 + row_of(x) / G) : 0; };
        Item next = {};
        int next_len = 0;
        bool have_next = true;
        while (ok) {
            int len = 0;
            if (dry) {
                it = Item{};
                it.tiles = i + 1;
            } else {
                if (!have_next) break;
                it = next;
                len = next_len;
                have_next = take(next, false);
                if (have_next) next_len = ask(next);
            }
            const bool two = !LOW && it.rows > kM;
            // ---- this thread's row: request b, head h, and how many of the common positions it has
            const bool mine = row_in(it);
            const int local = (two ? i * kM : 0) + r, mrow = mine ? row_of(it) : 0, qi = mrow / G, b = it.r0 + qi, h = it.g * G + (mrow - qi * G);
            float sl = s0;
            if (!dry) {
            if constexpr (LOW) {
              // ---- queries to shared memory, in two parts
              if (nq > 0) ok = warp_wait(smem_u32(&s_qempty), (nq - 1) & 1, bad);
              if (!ok) break;
              if (i == 0) {
                const uint32_t dst = sm + r * 128;
                const int64_t src = b * a.q_batch + (int64_t)h * HD;
                {
                    float y[HD];                                   // the row, all loads in flight together
                    if (!mine) {
#pragma unroll
                        for (int e = 0; e < HD; ++e) y[e] = 0.f;
                    } else if (a.dtype == SD_F32) {
#pragma unroll
                        for (int e = 0; e < HD; e += 4) *reinterpret_cast<float4*>(y + e) = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + src + e));
                    } else {
#pragma unroll
                        for (int c = 0; c < HD; c += 8) {
                            const uint4 u = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + src + c));
                            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 f = a.dtype == SD_BF16 ? make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u))
                                                                    : __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
                                y[c + 2 * e] = f.x;
                                y[c + 2 * e + 1] = f.y;
                            }
                        }
                    }
                    // fp16: the row by a power of two to a largest element in [2^14, 2^15), so that what the first part leaves
                    // stays above 2^-39 of it; rows below 2^-112 count as that large
                    float down = a.scale < 0.f ? -1.f : 1.f;
                    if constexpr (!BF) {
                        float mx = 0.f;
#pragma unroll
                        for (int e = 0; e < HD; ++e) mx = fmaxf(mx, fabsf(y[e]));
                        const int e = min(max((int)(__float_as_uint(mx) >> 23), 15), 254);
                        down *= __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
                        sl = fminf(fmaxf(sl * __uint_as_float((uint32_t)(e - 14) << 23), 1e-38f), 3e38f);    // 0 x inf is no score
                    }
#pragma unroll
                    for (int c = 0; c < HD / 8; ++c) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float u = y[8 * c + 2 * e] * down, w = y[8 * c + 2 * e + 1] * down;
                            hi[e] = pack2<BF>(u, w);
                            float2 f;
                            if constexpr (BF) f = make_float2(__uint_as_float(hi[e] << 16), __uint_as_float(hi[e] & 0xffff0000u));
                            else f = __half22float2(*reinterpret_cast<const __half2*>(&hi[e]));
                            // an infinite element has no second part
                            lo[e] = pack2<BF>(f.x - f.x == 0.f ? u - f.x : 0.f, f.y - f.y == 0.f ? w - f.y : 0.f);
                        }
                        const uint32_t at = dst + (c >> 3) * C::kPanel + (((c & 7) ^ (r & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + C::kTileBytes), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
                    }
                    s_scale[r] = sl;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              }
              __syncwarp();
              if (lane == 0) mb_arrive(smem_u32(&s_qfull));
              ok = warp_wait(smem_u32(&s_qfull), nq & 1, bad);     // the other warpgroup's rows
              if (!ok) break;
              sl = s_scale[r];
            }
            ++nq;
            }
            // how many of the common positions the row has, from the piece's first
            const int limit = dry || !mine ? 1 << 30 : (int)min((int64_t)max(len, 0), min((int64_t)it.pages * ps, (int64_t)a.max_len)) - it.i0 * kN;
            const float slack = fminf(kSlack / sl, 3.0e38f);
            // the score that the reference stands at, and the one from which it moves (far rows: they subtract in every
            // tile); P = exp2((s - sub) sl - ref)
            float top = -INFINITY, mark = -INFINITY, sub = 0.f, ref = 0.f, l = 0.f;
            const int step = two ? 1 : 2;
            for (int j = two ? 0 : i; j < it.tiles; j += step) {
                if (!dry) {
                    ok = warp_wait(smem_u32(&s_sfull[i]), ns & 1, bad);
                    if (!ok) break;
                    ++ns;
                }
                tm_after();
                // What is seldom done stays short, in loops over tensor memory: out of an empty instruction cache every 128
                // bytes of code cost some hundred cycles
                const int rest = limit - j * kN;
                {
                    const volatile uint32_t* mask = s_mask[(n + j) % kMasks];
                    const uint32_t full = mask[0] & mask[1] & mask[2] & mask[3];
                    if (__any_sync(0xffffffffu, rest < kN) || (full != 0xffffffffu && !dry)) {
#pragma unroll 1
                        for (int c = 0; c < kN; c += 16) {
                            float x[16];
                            tm_ld16(ts + c, x);
                            uint32_t live = mask[c >> 5] >> (c & 16);
                            const int left = rest - c;
                            if (left < 16) live &= left <= 0 ? 0u : (1u << left) - 1;
                            tm_wait_ld();
                            after_wait(x);
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] = (live >> e) & 1 ? x[e] : -INFINITY;
                            tm_st16(ts + c, reinterpret_cast<uint32_t*>(x));
                        }
                        tm_wait_st();
                    }
                }
                // 64 positions at a time, twice the same code: the scores are read again for the exponentials
                constexpr int kHalf = kN / 2;
                float s[kHalf];
                auto load = [&](int c0) {
#pragma unroll
                    for (int c = 0; c < kHalf; c += 32) tm_ld32(ts + c0 + c, s + c);
                    tm_wait_ld();
#pragma unroll
                    for (int c = 0; c < kHalf; c += 16) after_wait(s + c);
                };
                float mx = -INFINITY;
#pragma unroll 1
                for (int c0 = 0; c0 < kN; c0 += kHalf) {
                    load(c0);
                    float m0 = s[0], m1 = s[1], m2 = s[2], m3 = s[3];
#pragma unroll
                    for (int c = 4; c + 8 <= kHalf; c += 8) {
                        m0 = max3(m0, s[c], s[c + 1]);
                        m1 = max3(m1, s[c + 2], s[c + 3]);
                        m2 = max3(m2, s[c + 4], s[c + 5]);
                        m3 = max3(m3, s[c + 6], s[c + 7]);
                    }
                    m0 = max3(m0, s[kHalf - 4], s[kHalf - 3]);
                    m1 = max3(m1, s[kHalf - 2], s[kHalf - 1]);
                    mx = fmaxf(mx, fmaxf(max3(m0, m1, m2), m3));
                }
                if (__any_sync(0xffffffffu, mx > mark)) {
                    const bool grow = mx > (sub != 0.f ? top : mark);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = !grow ? 1.f : top == -INFINITY ? 0.f : ex2((top - mx) * sl);
                        if (grow) top = mx;
                        l *= f;
                        if (j >= step) {                           // O_i holds something
#pragma unroll 1
                            for (int c = 0; c < HD; c += 16) {
                                float o[16];
                                tm_ld16(to + i * HD + c, o);
                                tm_wait_ld();
                                after_wait(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] *= f;
                                tm_st16(to + i * HD + c, reinterpret_cast<uint32_t*>(o));
                            }
                            tm_wait_st();
                        }
                    }
                    const float m = top == -INFINITY ? top : top * sl;
                    const bool far = fabsf(m) >= kFar && m != -INFINITY;
                    sub = far ? top : 0.f;
                    ref = (far || m == -INFINITY ? 0.f : m) - kShift;
                    mark = far ? -INFINITY : top + slack;
                    if (__any_sync(0xffffffffu, far)) {
#pragma unroll 1
                        for (int c = 0; c < kN; c += 16) {
                            float x[16];
                            tm_ld16(ts + c, x);
                            tm_wait_ld();
                            after_wait(x);
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[e] -= sub;
                            tm_st16(ts + c, reinterpret_cast<uint32_t*>(x));
                        }
                        tm_wait_st();
                    }
                }
                float2 l0 = make_float2(0.f, 0.f), l1 = l0;
                const float2 sl2 = make_float2(sl, sl), ref2 = make_float2(-ref, -ref);
#pragma unroll 1
                for (int c0 = 0; c0 < kN; c0 += kHalf) {
                    load(c0);
#pragma unroll
                    for (int c = 0; c < kHalf; c += 32) {
                        uint32_t pr[16], lo[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 x = fma2(make_float2(s[c + 2 * e], s[c + 2 * e + 1]), sl2, ref2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            if (e & 1) l1 = add2(l1, x); else l0 = add2(l0, x);
                            pr[e] = pack2<BF>(x.x, x.y);
                            if constexpr (LOW) {
                                float2 f;
                                if constexpr (BF) f = make_float2(__uint_as_float(pr[e] << 16), __uint_as_float(pr[e] & 0xffff0000u));
                                else f = __half22float2(*reinterpret_cast<const __half2*>(&pr[e]));
                                lo[e] = pack2<BF>(x.x - f.x, x.y - f.y);
                            }
                        }
                        tm_st16(ts + c0 + c, pr);
                        if constexpr (LOW) tm_st16(ts + c0 + c + 16, lo);
                    }
                    tm_wait_st();
                    tm_before();
                    __syncwarp();
                    if (lane == 0 && !dry) mb_arrive(smem_u32(&s_pfull[i][c0 > 0]));
                }
                l += (l0.x + l0.y) + (l1.x + l1.y);
            }
            if (dry) {
                dry = false;
                tm_before();
                __syncwarp();
                if (lane == 0) mb_arrive(smem_u32(&s_dry));
                have_next = take(next, false);
                if (have_next) next_len = ask(next);
                continue;
            }
            if (!ok) break;
            n += it.tiles;
            // ---- the record: row's output, maximum and sum, as weights 2^(s - maximum)
            float m = top == -INFINITY ? top : top * sl;
            const bool have = two || i < it.tiles;                 // this warpgroup had a tile
            if (have) {
                ok = warp_wait(smem_u32(&s_ofull[i]), no >> i & 1, bad);
                if (!ok) break;
                no ^= 1u << i;
                tm_after();
            }
            const float unit = ex2(-kShift);
            if (!two && i == 1) {
                // the second half of a row: its sums to the first warpgroup, which reads the results where they are
                s_top[r] = m;
                s_sum[r] = l;
                tm_before();
                __syncwarp();
                if (lane == 0) mb_arrive(smem_u32(&s_half));
                ok = warp_wait(smem_u32(&s_joined), halves & 1, bad);
                ++halves;
                tm_after();
                continue;
            }
            float f0 = unit, f1 = 0.f;
            bool other = false;
            if (!two) {
                ok = warp_wait(smem_u32(&s_half), halves & 1, bad);
                ++halves;
                if (!ok) break;
                tm_after();
                other = it.tiles > 1;
                if (other) {
                    ok = warp_wait(smem_u32(&s_ofull[1]), no >> 1 & 1, bad);
                    no ^= 2u;
                    if (!ok) break;
                    tm_after();
                }
                const float m1 = s_top[r], l1 = s_sum[r], mx = fmaxf(m, m1);
                f0 = m == -INFINITY ? unit : ex2(m - mx - kShift);
                f1 = m1 == -INFINITY ? unit : ex2(m1 - mx - kShift);
                l = l * f0 + l1 * f1;
                m = mx;
            } else {
                l *= f0;
            }
            float* rec = shared_records(a, it.i0 == 0, (int64_t)it.r0 * a.H + it.g * (it.size * G) + it.m0, blockIdx.x);
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                float o[16];
                tm_ld16(to + i * HD + c, o);
                tm_wait_ld();
                after_wait(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= f0;
                if (other) {
                    float o1[16];
                    tm_ld16(to + HD + c, o1);
                    tm_wait_ld();
                    after_wait(o1);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = fmaf(o1[e], f1, o[e]);
                }
                if (mine) {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        __stcg(reinterpret_cast<float4*>(rec) + (c / 4 + y) * it.rows + local, make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]));
                }
            }
            if (mine) __stcg(reinterpret_cast<float2*>(rec + (int64_t)HD * it.rows) + local, make_float2(m, l));
            tm_before();
            if (!two) {
                __syncwarp();
                if (lane == 0) mb_arrive(smem_u32(&s_joined));
            }
        }
    }
    tm_before();
    __syncthreads();
    tm_after();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    if (tid == 0 && s_bad) report_expired(a);
}

template <int HD, bool BF, bool LOW>
cudaError_t launch_one(const SharedArgs& t, int blocks, cudaStream_t st) {
    return launch_k(k_attend_shared<HD, BF, LOW>, dim3(blocks), dim3(kThreads), Cfg<HD>::kSmem, st, t);
}
template <int HD, bool BF>
cudaError_t launch_low(const SharedArgs& t, bool low, int blocks, cudaStream_t st) {
    return low ? launch_one<HD, BF, true>(t, blocks, st) : launch_one<HD, BF, false>(t, blocks, st);
}
template <int HD, bool BF>
cudaError_t prepare_one() {
    const cudaError_t e = cudaFuncSetAttribute(k_attend_shared<HD, BF, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<HD>::kSmem);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(k_attend_shared<HD, BF, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<HD>::kSmem);
}

}  // namespace

cudaError_t prepare_attend_shared() {
    cudaError_t e = prepare_one<64, false>();
    if (e == cudaSuccess) e = prepare_one<128, false>();
    if (e == cudaSuccess) e = prepare_one<64, true>();
    if (e == cudaSuccess) e = prepare_one<128, true>();
    return e;
}

cudaError_t launch_attend_shared(const AttendArgs& a, const int32_t* group, const int32_t* shared, int n_groups, int hd, int sms,
                                 cudaStream_t st, int64_t worth, bool* taken) {
    SharedArgs t;
    int box = kN;
    while (a.by_ps.d % box) box >>= 1;
    const bool bf = a.kv_dtype == SD_BF16;
    *taken = map_kv(&t.k, a.kv_dtype, a.k, hd, (int)a.by_ps.d, a.Hkv, a.n_pages, a.pos_stride, a.head_stride, a.page_stride, box) &&
             map_kv(&t.v, a.kv_dtype, a.v, hd, (int)a.by_ps.d, a.Hkv, a.n_pages, a.pos_stride, a.head_stride, a.page_stride, box);
    if (!*taken) return cudaSuccess;
    t.a = a;
    t.group = group; t.shared = shared; t.n_groups = n_groups; t.box = box;
    t.worth = worth;
    const bool low = a.dtype != a.kv_dtype || a.scale < 0.f;
    if (hd == 64) return bf ? launch_low<64, true>(t, low, sms, st) : launch_low<64, false>(t, low, sms, st);
    return bf ? launch_low<128, true>(t, low, sms, st) : launch_low<128, false>(t, low, sms, st);
}

}  // namespace sd
