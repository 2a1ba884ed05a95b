// Split-length attention: few queries over many positions, reached through a
// page table or by strides.
//
// A unit is (row b, kv head g, tile of up to 8 query rows of that head's group);
// a row is (query i, head of the group).  Its positions are cut into tiles of
// 128 or 256, and the tiles of all units, laid end to end, are dealt evenly to the
// resident blocks: every block streams the same number of bytes whatever the
// lengths are, and no host needs to know them.  A unit that ends up in several
// blocks is joined by the last of them to arrive, in block order (results do not
// depend on the order of arrival).
//
// The kernel is bound by the key and value bytes: 48 requests of up to 32768 positions, 8 kv
// heads of 128, bf16, 651 MB take 101 us, 6.5 TB/s, 0.95 of the copy rate (e4m3, 64 requests of
// 2000 to 4100, 64 heads to 8: 71 us, 0.83).  Three warps walk the block's share
// and load by TMA, in turn, a tile's keys or its values (32 KB) into a ring, running
// ahead across the ends of units; a fourth prepares the units (where they lie, their queries).
// Eight warps work on a tile, 16 or 32 positions each, with a running maximum and sum of
// their own; four more merge and write a unit's result while the eight are at the next
// one (merging in their place cost about 3 us a unit).  Positions behind a length or in a page
// that is not there are masked; their values are set to 0 in shared memory, so that
// what they hold does not matter.
//
// Scores and results are mma.sync products (m16n8k16) in transposed form, S^T = K q^T and
// O^T = V^T P^T: positions and dimensions fill the 16 rows and the 8 query rows the 8
// columns, so that no part of an instruction is empty and a warp's results take 32 to 64
// registers.  Where fp16 or bf16 does not hold q (fp32) or the probabilities (fp32 results, bf16
// caches), a second product adds what the rounding left.  (tcgen05 needs 64 or 128 query
// rows, of which 1 to 8 would hold work.)
#include "attend_dev.cuh"

namespace sd {
namespace {

constexpr int kWarps = 8, kLoaders = 3, kMergers = kSplitRows / 2, kConsumers = 32 * kWarps;
constexpr int kThreads = kConsumers + 32 * (kLoaders + 1 + kMergers);
// Registers of a thread: 512 x 128 at launch = 256 x 176 + 256 x 80
constexpr int kConsumerRegs = 176, kOtherRegs = 80;
static_assert(kLoaders + 1 == 4 && kMergers == 4 && kWarps % 4 == 0, "warpgroups");
static_assert(kConsumers * kConsumerRegs + (kThreads - kConsumers) * kOtherRegs <= kThreads * 128, "the shares exceed what the block was launched with");

struct alignas(128) SplitArgs {
    CUtensorMap k, v;
    AttendArgs a;
    int32_t box, groups;      // positions of a box (all of one page), boxes of a tile's keys or values and column part
};

__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two e4m3 values (a 16-bit half of w) as fp16x2: exact
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t w) {
    uint32_t d;
    asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(d) : "r"(w));
    return d;
}
// What the rounding of q to fp16 left is kept 2^12 times as large (below 2): from 2^-25 on it would be subnormal
constexpr float kLow = 4096.f;

// x, y rounded to the product's type, and what the rounding left, times `up`
template <bool BF>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo, float up = 1.f) {
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const float2 f = __bfloat1622float2(h);
        const __nv_bfloat162 l = __floats2bfloat162_rn((x - f.x) * up, (y - f.y) * up);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = *reinterpret_cast<const uint32_t*>(&l);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn((x - f.x) * up, (y - f.y) * up);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = *reinterpret_cast<const uint32_t*>(&l);
    }
}
template <bool BF>
__device__ __forceinline__ uint32_t round2(float x, float y) {
    uint32_t hi, lo;
    split2<BF>(x, y, hi, lo);
    return hi;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// high and low product; an infinite high product has no low one (0 * inf)
__device__ __forceinline__ float add_low(float hi, float lo) { return hi - hi == 0.f ? fmaf(lo, 1.f / kLow, hi) : hi; }

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t lds1(uint32_t at) {
    uint32_t x;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ float2 lds2(uint32_t at) {
    float2 x;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(at) : "memory");
    return x;
}
// N (2 or 4) consecutive elements
template <int N>
__device__ __forceinline__ void storev(void* p, int64_t i, int dt, const float* v) {
    if (dt == SD_F32) {
#pragma unroll
        for (int x = 0; x < N; x += 2) *reinterpret_cast<float2*>(static_cast<float*>(p) + i + x) = make_float2(v[x], v[x + 1]);
    } else {
        uint32_t w[N / 2];
#pragma unroll
        for (int x = 0; x < N; x += 2) w[x / 2] = dt == SD_F16 ? round2<false>(v[x], v[x + 1]) : round2<true>(v[x], v[x + 1]);
        uint16_t* q = static_cast<uint16_t*>(p) + i;
        if constexpr (N == 4) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(q) = w[0];
    }
}

constexpr int kUnits = 4;                             // units prepared ahead
constexpr int kMinTiles = 2;                          // of a part of a unit, where blocks are not short

template <int HD, int KV>
struct Shape {
    static constexpr bool kBf = KV == SD_BF16, kE4 = KV == SD_E4M3;
    static constexpr int kRow = HD * (kE4 ? 1 : 2);             // bytes of a position's row
    static constexpr int kCols = kRow / 16;                     // 16-byte columns
    static constexpr int kPart = kRow < 128 ? kRow : 128;       // bytes of a row in a box
    static constexpr int kParts = kRow / kPart;                 // 2 for 256-byte rows
    static constexpr int kChunk = kRow >= 256 ? 16 : 32;        // positions of a warp
    static constexpr int kTile = kChunk * kWarps;
    static constexpr int kStage = kTile * kRow;                 // the keys, or the values, of a tile
    static constexpr int kPitch = HD + 4;                       // floats of a row of results: no bank conflicts between heads
    static constexpr int kMerge = kWarps * kSplitRows * (kPitch + 2) * 4;
    static constexpr int kQueries = kSplitRows * HD * 4;        // a unit's queries, in their own type
    static constexpr int kStages = kStage >= 32768 ? 5 : 10;
    // A loader waits for the stage `kStages` before its own by parity, so the one 2 kStages before must be known to be
    // free: it is, as every warp takes the stages in order and the loader has waited for one at most kLoaders earlier.
    static_assert(kStages >= kLoaders, "a loader could mistake the phase of a stage");
    static constexpr int kRing = kStages * kStage;
    static constexpr int kSmem = kRing + kMerge + kUnits * kQueries + 1024;
    // What beginning and ending a unit costs, in tiles: the share of a block counts it
    static constexpr int kLead = 1;
    // fp16 probabilities are kept as 2^15 p: the smallest ones stay above fp16's subnormal step
    static constexpr float kShift = kBf ? 0.f : 15.f;
    // byte of a 16-byte column of a row: the boxes' swizzle puts the 8 rows of a matrix into 8 different bank groups
    static __device__ __forceinline__ uint32_t at(int row, int col) {
        if constexpr (kRow == 64) return row * 64 + ((col ^ ((row >> 1) & 3)) << 4);
        return (col >> 3) * (kTile * 128) + row * 128 + (((col & 7) ^ (row & 7)) << 4);
    }
};

// What the warps on a unit need to know: m0 its first query row, tiles [i0, i0 + tiles) its part in this block
struct Unit {
    int64_t m0;
    int b, g, len, rows, i0, tiles, c_lo, c_hi, begins;
};

template <int HD, int KV>
__global__ void __launch_bounds__(kThreads, 1) k_attend_split(const __grid_constant__ SplitArgs args) {
    using S = Shape<HD, KV>;
    constexpr int kSteps = HD / 16, kOut = HD / 16, kChunk = S::kChunk, kTile = S::kTile, kSt = S::kStages;
    const AttendArgs& a = args.a;
    extern __shared__ unsigned char smraw[];
    __shared__ __align__(8) unsigned long long s_full[kSt], s_empty[kSt];
    __shared__ __align__(8) unsigned long long s_ufull[kUnits], s_uempty[kUnits], s_done, s_free, s_never;
    __shared__ uint32_t s_live[kSt][kWarps];
    __shared__ Unit s_unit[kUnits];
    __shared__ int2 s_box[kLoaders][32];
    __shared__ int64_t s_sum[kThreads / 32];
    __shared__ int64_t s_base;
    __shared__ int s_len[kThreads];
    __shared__ int s_b, s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned char* smem = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    const uint32_t ring = smem_u32(smem);
    const int G = a.H / a.Hkv;
    const int64_t M = (int64_t)a.Lq * G;                                  // query rows of a (b, kv head)
    const int64_t RT = (M + kSplitRows - 1) / kSplitRows;
    const int64_t U = RT * a.Hkv;                                         // units of a row b
    volatile int* bad = &s_bad;

    if (tid == kConsumers) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&args.k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&args.v)) : "memory");
        for (int s = 0; s < kSt; ++s) {
            mb_init(smem_u32(&s_full[s]), 1);
            mb_init(smem_u32(&s_empty[s]), kWarps);
        }
        mb_init(smem_u32(&s_done), kWarps);
        mb_init(smem_u32(&s_free), kMergers);
        mb_init(smem_u32(&s_never), 1);
        for (int s = 0; s < kUnits; ++s) {
            mb_init(smem_u32(&s_ufull[s]), 1);
            mb_init(smem_u32(&s_uempty[s]), kWarps + kMergers);
        }
        s_bad = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_trigger();
    pdl_wait();

    const bool few = a.B <= 32;                                           // a lane for each row, in every warp
    auto length = [&](int b) { return min(max(a.len ? __ldcg(a.len + b) : a.max_len, 0), a.max_len); };
    auto tiles = [&](int len) { return (len + kTile - 1) / kTile; };

    // ---- this block's share.  Where every unit can have a block of its own, units are cut into parts of `per` tiles
    // with a block each, per = (all tiles) / (blocks left over by whole units): no unit is cut without need, since
    // joining costs about 3 us.  Otherwise all tiles, kLead empty ones before each unit, are dealt out evenly.
    const int64_t grid = gridDim.x;
    const int len0 = few && lane < a.B ? length(lane) : 0;
    const bool whole = few && a.B * U <= grid;
    const int lead = whole ? 0 : S::kLead;
    int64_t per = 1;
    // tiles of a unit with the empty ones before it, or behind it to a multiple of `per`
    auto padded = [&](int n) -> int { return whole ? (int)(quot(max(n, 1) + per - 1, per) * per) : n + S::kLead; };
    int64_t t, base, T;                                                   // next tile; first tile of row b_at
    int b_at;
    if (few) {
        const int n = tiles(len0);
        if (whole) {
            const int64_t all = (int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)n) * U, left = grid - a.B * U;
            per = max(__reduce_max_sync(0xffffffffu, n), 1);
            if (left > 0) per = min(per, max(quot(all + left - 1, left), (int64_t)kMinTiles));
        }
        const int64_t mine = lane < a.B ? padded(n) : 0;
        int64_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        T = __shfl_sync(0xffffffffu, sum, 31) * U;
        if (!whole) per = max(quot(T + grid - 1, grid), (int64_t)1);
        t = blockIdx.x * per;
        const uint32_t here = __ballot_sync(0xffffffffu, (sum - mine) * U <= t && t < sum * U);
        b_at = __ffs(here) - 1;
        base = __shfl_sync(0xffffffffu, (sum - mine) * U, b_at & 31);
    } else {
        // inclusive sums over the threads: of a row each where there are no more rows than threads
        int64_t mine = 0;
        for (int b = tid; b < a.B; b += kThreads) {
            const int len = length(b);
            if (b < kThreads) s_len[b] = len;
            mine += padded(tiles(len));
        }
        int64_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) s_sum[warp] = sum;
        __syncthreads();
        T = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) sum += s_sum[w];
            T += s_sum[w];
        }
        T *= U;
        per = max(quot(T + grid - 1, grid), (int64_t)1);
        t = blockIdx.x * per;
        if (t >= T) return;
        // the row that holds tile t, and its first tile
        if (a.B <= kThreads) {
            if ((sum - mine) * U <= t && t < sum * U) {
                s_b = tid;
                s_base = (sum - mine) * U;
            }
        } else {
            for (int64_t b0 = 0, before = 0; b0 < a.B; b0 += kThreads) {
                const int64_t b = b0 + tid;
                const int64_t n = b < a.B ? padded(tiles(length((int)b))) * U : 0;
                int64_t x = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                __syncthreads();
                if (lane == 31) s_sum[warp] = x;
                __syncthreads();
                int64_t at = before;
                for (int w = 0; w < kThreads / 32; ++w) {
                    if (w < warp) at += s_sum[w];
                    before += s_sum[w];
                }
                if (n && at + x - n <= t && t < at + x) {
                    s_b = (int)b;
                    s_base = at + x - n;
                }
                if (before > t) break;
            }
        }
        __syncthreads();
        b_at = s_b;
        base = s_base;
    }
    if (t >= T) return;
    const int64_t t_begin = t, t_end = min(T, t + per);
    __syncthreads();                                                      // the barriers are initialised

    // The units of this block in turn.
    auto next_unit = [&](Unit& p) -> bool {
        if (t >= t_end) return false;
        p.b = b_at;
        p.len = few ? __shfl_sync(0xffffffffu, len0, b_at) : b_at < kThreads ? s_len[b_at] : length(b_at);
        const int real_tiles = tiles(p.len), nt = padded(real_tiles);
        const int64_t u = quot(t - base, nt), u0 = base + u * nt;        // the unit's tiles [u0, u0 + nt)
        const int64_t next = min(u0 + nt, t_end);
        // blocks with a part of its tiles (an empty unit: the block with its last empty tile)
        const int64_t real = min(u0 + lead, u0 + nt - 1);
        if (next <= real) return false;                                   // only empty tiles left in this block
        p.c_lo = (int)quot(real, per);
        p.c_hi = (int)quot(u0 + nt - 1, per);
        p.begins = real >= t_begin;
        p.i0 = (int)max(t - u0 - lead, (int64_t)0);
        p.tiles = min(real_tiles, (int)(next - u0) - lead) - p.i0;
        p.g = (int)quot(u, RT);
        p.m0 = (u - p.g * RT) * kSplitRows;
        p.rows = (int)min((int64_t)kSplitRows, M - p.m0);
        t = next;
        if (next - base == nt * U) {
            base = next;
            ++b_at;
        }
        return true;
    };

    float* s_o = reinterpret_cast<float*>(smem + S::kRing);              // [warp][row][HD]
    float* s_m = s_o + kWarps * kSplitRows * S::kPitch;                   // [warp][row]
    float* s_l = s_m + kWarps * kSplitRows;
    unsigned char* s_q = smem + S::kRing + S::kMerge;                      // [unit][row][HD] of the queries' type
    const int qbytes = a.dtype == SD_F32 ? 4 : 2;
    if (warp >= kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        bool ok = true;
        if (warp > kWarps + kLoaders) {
            // ============================================ mergers: two rows of every unit each, beside the next unit's tiles
            const int mw = warp - kWarps - kLoaders - 1;
            constexpr int kVec = HD / 32;                                 // columns of a lane
            const bool dead = __ldcg(a.dead) != 0;                        // asked for here, needed behind the first unit's tiles
            for (uint32_t nu = 0;; ++nu) {
                if (!warp_wait(smem_u32(&s_ufull[nu % kUnits]), (nu / kUnits) & 1, bad)) break;
                const Unit u = s_unit[nu % kUnits];
                __syncwarp();
                if (lane == 0) mb_arrive(smem_u32(&s_uempty[nu % kUnits]));
                if (!u.rows) break;
                if (!warp_wait(smem_u32(&s_done), nu & 1, bad)) break;
                float val[2][kVec], mm[2], ll[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = mw + kMergers * e;
                    float mw_[kWarps];
                    mm[e] = -INFINITY;
                    ll[e] = 0.f;
#pragma unroll
                    for (int x = 0; x < kVec; ++x) val[e][x] = 0.f;
                    if (r >= u.rows) continue;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        mw_[w] = s_m[w * kSplitRows + r];
                        mm[e] = fmaxf(mm[e], mw_[w]);
                    }
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        if (mw_[w] == -INFINITY) continue;
                        const float f = ex2(mw_[w] - mm[e]);
                        ll[e] = fmaf(f, s_l[w * kSplitRows + r], ll[e]);
                        const float* so = s_o + (w * kSplitRows + r) * S::kPitch + lane * kVec;
#pragma unroll
                        for (int x = 0; x < kVec; ++x) val[e][x] = fmaf(f, so[x], val[e][x]);
                    }
                }
                __syncwarp();
                if (lane == 0) mb_arrive(smem_u32(&s_free));
                if (mw >= u.rows) continue;
                const int n_rows = mw + kMergers < u.rows ? 2 : 1;
                bool last = true;
                if (u.c_lo != u.c_hi && !dead) {
                    // ---- the last block of the unit to arrive joins the records in block order
                    float* rec = a.part + (int64_t)(2 * blockIdx.x + u.begins) * kSplitRecord;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (e >= n_rows) break;
                        const int r = mw + kMergers * e;
#pragma unroll
                        for (int x = 0; x < kVec; ++x) __stcg(rec + r * HD + lane * kVec + x, val[e][x]);
                        if (lane == 0) __stcg(reinterpret_cast<float2*>(rec + kSplitRows * 128) + r, make_float2(mm[e], ll[e]));
                    }
                    __syncwarp();
                    int before = 0;
                    if (lane == 0) {
                        __threadfence();
                        before = atomicAdd(a.cnt + u.c_lo * kMergers + mw, 1);
                        __threadfence();
                    }
                    last = __shfl_sync(0xffffffffu, before, 0) == u.c_hi - u.c_lo;
                    __syncwarp();                                         // orders the other lanes' reads of records behind lane 0's fence
                    if (last) {
                        if (lane == 0) a.cnt[u.c_lo * kMergers + mw] = 0;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (e >= n_rows) break;
                            const int r = mw + kMergers * e;
                            mm[e] = -INFINITY;
                            ll[e] = 0.f;
#pragma unroll
                            for (int x = 0; x < kVec; ++x) val[e][x] = 0.f;
#pragma unroll 4
                            for (int c = u.c_lo; c <= u.c_hi; ++c) {
                                const float* p = a.part + (int64_t)(2 * c + (c == u.c_lo ? 1 : 0)) * kSplitRecord;
                                const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + kSplitRows * 128) + r);
                                float oc[kVec];
#pragma unroll
                                for (int x = 0; x < kVec; ++x) oc[x] = __ldcg(p + r * HD + lane * kVec + x);
                                const bool have = ml.x != -INFINITY;
                                const float mx = fmaxf(mm[e], ml.x);
                                const float f0 = mm[e] == -INFINITY ? 0.f : ex2(mm[e] - mx), f1 = have ? ex2(ml.x - mx) : 0.f;
                                ll[e] = ll[e] * f0 + ml.y * f1;
#pragma unroll
                                for (int x = 0; x < kVec; ++x) val[e][x] = val[e][x] * f0 + (have ? oc[x] * f1 : 0.f);
                                mm[e] = mx;
                            }
                        }
                    }
                }
                if (!last) continue;
                if (dead) ll[0] = ll[1] = NAN;
                const float vs = a.v_scale ? __ldcg(a.v_scale + u.g) : 1.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (e >= n_rows) break;
                    const int64_t m = u.m0 + mw + kMergers * e, qi = a.Lq == 1 ? 0 : quot(m, G), h = (int64_t)u.g * G + (m - qi * G);
                    const int64_t at = u.b * a.o_batch + qi * a.o_stride + h * HD + lane * kVec;
                    const float inv = ll[e] == 0.f ? 0.f : vs / ll[e];
#pragma unroll
                    for (int x = 0; x < kVec; ++x) val[e][x] = ll[e] == 0.f ? 0.f : val[e][x] * inv;
                    storev<kVec>(a.out, at, a.dtype, val[e]);
                    if (lane == 0 && a.lse)
                        a.lse[((int64_t)u.b * a.Lq + qi) * a.H + h] = ll[e] == 0.f ? -INFINITY : (mm[e] + log2f(ll[e]) - S::kShift) * kLn2;
                }
            }
            if (lane == 0 && *bad) report_expired(a);
            return;
        }
        Unit p;
        if (warp == kWarps + kLoaders) {
            // ============================================ units and their queries
            uint32_t n = 0;
            if (a.stall && blockIdx.x == 0) ok = warp_wait(smem_u32(&s_never), 0, bad, a.stall);
            for (; ok && next_unit(p); ++n) {
                const uint32_t slot = n % kUnits;
                if (n >= kUnits) ok = warp_wait(smem_u32(&s_uempty[slot]), (n / kUnits - 1) & 1, bad);
                if (!ok) break;
                // rows of cols 16-byte pieces; four loads of a lane in flight together
                const int cols = HD * qbytes / 16;
                for (int x0 = lane; x0 < kSplitRows * cols; x0 += 128) {
                    uint4 v[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int x = x0 + y * 32, r = x / cols, c = x - r * cols;
                        v[y] = make_uint4(0, 0, 0, 0);
                        if (r < p.rows) {
                            const int64_t m = p.m0 + r, qi = a.Lq == 1 ? 0 : quot(m, G);
                            const int64_t at = p.b * a.q_batch + qi * a.q_stride + ((int64_t)p.g * G + (m - qi * G)) * HD;
                            v[y] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.q) + at * qbytes + c * 16);
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int x = x0 + y * 32;
                        if (x < kSplitRows * cols) *reinterpret_cast<uint4*>(s_q + slot * S::kQueries + x * 16) = v[y];
                    }
                }
                if (lane == 0) s_unit[slot] = p;
                __syncwarp();
                if (lane == 0) mb_arrive(smem_u32(&s_ufull[slot]));
            }
            // behind the last unit: one without rows
            const uint32_t slot = n % kUnits;
            if (ok && n >= kUnits) ok = warp_wait(smem_u32(&s_uempty[slot]), (n / kUnits - 1) & 1, bad);
            if (lane == 0) {
                s_unit[slot].rows = 0;
                mb_arrive(smem_u32(&s_ufull[slot]));
            }
            return;
        }
        // ================================================ loads: a stage is a tile's keys, the next one its values
        const uint32_t turn_of = warp - kWarps;
        uint32_t n = 0, last = 0;                                         // stages of all loaders so far; up to this one's last
        const int groups = args.groups, box = args.box;
        while (ok && next_unit(p)) {
            // of a lane's box (k * 32 + lane) of tile i: its page, -1 without one
            auto lookup = [&](int i, int k) -> int {
                const int pos = (p.i0 + i) * kTile + (k * 32 + lane) * box;
                if (i >= p.tiles || k * 32 + lane >= groups || pos >= p.len) return -1;
                return a.table ? __ldcg(a.table + (int64_t)p.b * a.table_stride + a.by_ps.div((uint32_t)pos)) : p.b;
            };
            const int outer = a.table ? a.n_pages : a.B;
            int x = (int)((turn_of + kLoaders - n % kLoaders) % kLoaders), ahead = lookup(x >> 1, 0);
            for (; x < 2 * p.tiles && ok; x += kLoaders) {
                const int i = x >> 1, op = x & 1;
                const int first = (p.i0 + i) * kTile, rest = p.len - first;
                // of a box: its position within its page (or row)
                auto inside = [&](int k) -> int {
                    const int pos = first + (k * 32 + lane) * box;
                    return a.table ? pos - (int)(a.by_ps.div((uint32_t)pos) * a.by_ps.d) : pos;
                };
                const int id0 = (uint32_t)ahead < (uint32_t)outer ? ahead : -1, in0 = inside(0);
                ahead = lookup((x + kLoaders) >> 1, 0);                   // a stage ahead: not waited for here
                const uint32_t st = n + x, slot = st % kSt, turn = st / kSt;
                if (turn > 0) ok = warp_wait(smem_u32(&s_empty[slot]), (turn - 1) & 1, bad);
                if (!ok) break;
                last = st + 1;
                const uint32_t mb = smem_u32(&s_full[slot]), dst = ring + slot * S::kStage;
                if (op == 0 && lane < kWarps) s_live[slot][lane] = 0;
                __syncwarp();
#pragma unroll 1
                for (int k = 0; k * 32 < groups; ++k) {
                    int id = id0, in = in0;
                    if (k > 0) {
                        id = lookup(i, k);
                        if ((uint32_t)id >= (uint32_t)outer) id = -1;
                        in = inside(k);
                    }
                    if (op == 0 && id >= 0) {
                        // live positions of each warp's part of the tile
                        const int at = (k * 32 + lane) * box, end = min(at + box, rest);
                        for (int r = at; r < end;) {
                            const int c = r / kChunk, stop = min(end, (c + 1) * kChunk), count = stop - r;
                            atomicOr(&s_live[slot][c], (0xffffffffu >> (32 - count)) << (r - c * kChunk));
                            r = stop;
                        }
                    }
                    const uint32_t have = __ballot_sync(0xffffffffu, id >= 0);
                    if (k > 0) __syncwarp();
                    s_box[turn_of][lane] = make_int2(id, in);
                    __syncwarp();
                    // box by box from the elected lane (by several lanes of a warp at once: 250 cycles each)
                    if (elect_one()) {
                        if (have) mb_expect_more(mb, __popc(have) * box * S::kRow);
                        const int boxes = min(32, groups - k * 32);
                        uint32_t to = dst + k * 32 * box * S::kPart;
                        for (int y = 0; y < boxes; ++y, to += box * S::kPart) {
                            const int2 v = s_box[turn_of][y];
                            if (v.x < 0) continue;
#pragma unroll
                            for (int part = 0; part < S::kParts; ++part)
                                tma4(to + part * (kTile * 128), op ? &args.v : &args.k, part * 64, v.y, p.g, v.x, mb);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mb_arrive(mb);
            }
            n += 2 * max(p.tiles, 0);
        }
        if (!ok)                                                          // bounded: this warp's own copies
            for (uint32_t x = last > kSt ? last - kSt : 0; x < last; ++x) {
                if (x % kLoaders != turn_of) continue;
                const long long t0 = clock64();
                while (!mb_try(smem_u32(&s_full[x % kSt]), (x / kSt) & 1) && clock64() - t0 < kWaitClocks) {}
            }
        return;
    }

    // ==================================================== scores and sums
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
    const int row = lane >> 2, quad = lane & 3, mi = lane >> 3, mr = lane & 7;
    // Low-order parts: of q where the products' type does not hold it (a 16-bit q scaled into fp16 loses only what is
    // 2^-24 of its row's largest element); of the probabilities for fp32 results and where bf16 is all they have
    const bool q_low = a.dtype == SD_F32 || (S::kBf && a.dtype == SD_F16), p_low = a.dtype == SD_F32 || S::kBf;
    uint32_t n = 0;                                                       // tiles of the units before
    for (uint32_t nu = 0;; ++nu) {
        // a failed wait (flagged) ends the waiting, and with it the walk
        bool ok = warp_wait(smem_u32(&s_ufull[nu % kUnits]), (nu / kUnits) & 1, bad);
        const Unit pc = s_unit[nu % kUnits];
        if (!ok || !pc.rows) break;
        const int g = pc.g, rows = pc.rows;
        // ---- the B operand: head `row` of the unit, 4 elements of each 16 a lane
        uint32_t qh[kSteps][2], ql[kSteps][2];
        float scale[2];                                                   // of this lane's two columns of the scores
        {
            float2 x[kSteps][2];
            const uint32_t at = smem_u32(s_q) + nu % kUnits * S::kQueries;
            if (a.dtype == SD_F32) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) x[k][e] = lds2(at + 4 * (row * HD + 16 * k + (S::kE4 ? 4 * quad + 2 * e : 2 * quad + 8 * e)));
            } else {
                uint32_t w[kSteps][2];
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) w[k][e] = lds1(at + 2 * (row * HD + 16 * k + (S::kE4 ? 4 * quad + 2 * e : 2 * quad + 8 * e)));
                const bool bf = a.dtype == SD_BF16;
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        x[k][e] = bf ? make_float2(__uint_as_float(w[k][e] << 16), __uint_as_float(w[k][e] & 0xffff0000u))
                                     : __half22float2(*reinterpret_cast<const __half2*>(&w[k][e]));
            }
            __syncwarp();
            if (lane == 0) mb_arrive(smem_u32(&s_uempty[nu % kUnits]));
            float down = 1.f, row_scale = a.scale * kLog2e * (a.k_scale ? __ldcg(a.k_scale + g) : 1.f);
            if (!S::kBf && a.dtype != SD_F16) {
                // wider exponents than fp16's: the row by a power of two to a largest element in [1, 2)
                float mx = 0.f;
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) mx = fmaxf(mx, fmaxf(fabsf(x[k][e].x), fabsf(x[k][e].y)));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const int e = min(max((int)(__float_as_uint(mx) >> 23), 1), 253);
                if (mx > 0.f && mx < INFINITY) {
                    down = __uint_as_float((uint32_t)(254 - e) << 23);
                    row_scale *= __uint_as_float((uint32_t)e << 23);
                }
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) split2<S::kBf>(x[k][e].x * down, x[k][e].y * down, qh[k][e], ql[k][e], kLow);
            scale[0] = __shfl_sync(0xffffffffu, row_scale, 8 * quad);
            scale[1] = __shfl_sync(0xffffffffu, row_scale, 8 * quad + 4);
        }
        // this lane's results: heads 2 quad and 2 quad + 1, dimensions `row` and `row` + 8 of each 16 (e4m3: 2 row, 2 row + 1)
        float o[kOut][4];
#pragma unroll
        for (int y = 0; y < kOut; ++y) o[y][0] = o[y][1] = o[y][2] = o[y][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        auto release = [&](uint32_t slot) {
            __syncwarp();
            if (lane == 0) mb_arrive(smem_u32(&s_empty[slot]));
        };

        // ---- this warp's eighth of every tile
        constexpr int kH = kChunk / 16;
        const int r0 = warp * kChunk;                                     // its first position in a tile
        for (int i = 0; i < pc.tiles; ++i) {
            const uint32_t st = 2 * (n + i), sk = st % kSt, sv = (st + 1) % kSt;
            const uint32_t kb = ring + sk * S::kStage, vb = ring + sv * S::kStage;
            warp_wait(smem_u32(&s_full[sk]), (st / kSt) & 1, bad);
            const uint32_t live = s_live[sk][warp];
            if (!live) {                                                  // nothing here
                release(sk);
                warp_wait(smem_u32(&s_full[sv]), ((st + 1) / kSt) & 1, bad);
                release(sv);
                continue;
            }
            // S^T = K q^T: rows are positions 16 h + row and + 8, columns this lane's heads
            float s[kH][4];
            auto scores = [&](const uint32_t (&q)[kSteps][2], float (&d)[kH][4]) {
#pragma unroll
                for (int h = 0; h < kH; ++h) d[h][0] = d[h][1] = d[h][2] = d[h][3] = 0.f;
                if constexpr (!S::kE4) {
#pragma unroll
                    for (int k = 0; k < kSteps; ++k)
#pragma unroll
                        for (int h = 0; h < kH; ++h) {
                            uint32_t f[4];
                            ldm4(kb + S::at(r0 + 16 * h + (mi & 1) * 8 + mr, 2 * k + (mi >> 1)), f);
                            mma<S::kBf>(d[h], f, q[k][0], q[k][1]);
                        }
                } else {
#pragma unroll
                    for (int k = 0; k < kSteps; k += 2)
#pragma unroll
                        for (int h = 0; h < kH; ++h) {
                            uint32_t f[4];
                            ldm4(kb + S::at(r0 + 16 * h + (mi & 1) * 8 + mr, k + (mi >> 1)), f);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t x[4] = {half2_of_e4m3(f[2 * e]), half2_of_e4m3(f[2 * e + 1]),
                                                       half2_of_e4m3(f[2 * e] >> 16), half2_of_e4m3(f[2 * e + 1] >> 16)};
                                mma<false>(d[h], x, q[k + e][0], q[k + e][1]);
                            }
                        }
                }
            };
            scores(qh, s);
            if (q_low) {
                float d[kH][4];
                scores(ql, d);
#pragma unroll
                for (int h = 0; h < kH; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[h][e] = add_low(s[h][e], d[h][e]);
            }
            release(sk);
#pragma unroll
            for (int h = 0; h < kH; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[h][e] *= scale[e & 1];
            if (live != 0xffffffffu >> (32 - kChunk)) {
#pragma unroll
                for (int h = 0; h < kH; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((live >> (16 * h + 8 * (e >> 1) + row)) & 1)) s[h][e] = -INFINITY;
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int h = 0; h < kH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) mx[e] = max_nan(mx[e], max_nan(s[h][e], s[h][2 + e]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
#pragma unroll
                for (int e = 0; e < 2; ++e) mx[e] = max_nan(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], x));
#pragma unroll
            for (int e = 0; e < 2; ++e) mx[e] = mx[e] == mx[e] ? fmaxf(mx[e], m[e]) : INFINITY;   // NaN reaches every result of its row
            if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
                float keep[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    keep[e] = m[e] == -INFINITY ? 0.f : ex2(m[e] - mx[e]);
                    l[e] *= keep[e];
                    m[e] = mx[e];
                }
#pragma unroll
                for (int x = 0; x < kOut; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[x][e] *= keep[e & 1];
            }
            float ref[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) ref[e] = m[e] == -INFINITY ? 0.f : m[e];
            // 2^(s - m + shift), the shift behind the exact difference: m - shift is rounded from 2^24 on, up to 2^16 and
            // beyond fp16
            auto prob = [&](float s, float r) { return S::kShift == 0.f ? ex2(s - r) : ex2((s - r) + S::kShift); };
            // P^T as the B operand: each 8 positions x 8 heads transposed
            uint32_t ph[kH][2], pl[kH][2];
#pragma unroll
            for (int h = 0; h < kH; ++h)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float p0 = prob(s[h][2 * y], ref[0]), p1 = prob(s[h][2 * y + 1], ref[1]);
                    l[0] += p0;
                    l[1] += p1;
                    split2<S::kBf>(p0, p1, ph[h][y], pl[h][y]);
                    ph[h][y] = transpose8(ph[h][y]);
                }
            warp_wait(smem_u32(&s_full[sv]), ((st + 1) / kSt) & 1, bad);
            if (live != 0xffffffffu >> (32 - kChunk)) {
                // values of positions that are not there: 0, whatever lies in memory
                for (int y = lane; y < kChunk * S::kCols; y += 32) {
                    const int r = y / S::kCols;
                    if (!((live >> r) & 1))
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + S::at(r0 + r, y % S::kCols)), "r"(0) : "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            // O^T += V^T P^T
            auto results = [&](const uint32_t (&p)[kH][2]) {
                if constexpr (!S::kE4) {
#pragma unroll
                    for (int h = 0; h < kH; ++h)
#pragma unroll
                        for (int x = 0; x < kOut; ++x) {
                            uint32_t f[4];
                            ldm4t(vb + S::at(r0 + 16 * h + (mi >> 1) * 8 + mr, 2 * x + (mi & 1)), f);
                            mma<S::kBf>(o[x], f, p[h][0], p[h][1]);
                        }
                } else {
                    // a transposed matrix of byte pairs: even dimensions in the low bytes, odd ones in the high
#pragma unroll
                    for (int h = 0; h < kH; ++h)
#pragma unroll
                        for (int x = 0; x < kOut; x += 2) {
                            uint32_t f[4];
                            ldm4t(vb + S::at(r0 + 16 * h + (mi & 1) * 8 + mr, x + (mi >> 1)), f);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t y[4] = {half2_of_e4m3(__byte_perm(f[2 * e], 0, 0x4420)), half2_of_e4m3(__byte_perm(f[2 * e], 0, 0x4431)),
                                                       half2_of_e4m3(__byte_perm(f[2 * e + 1], 0, 0x4420)), half2_of_e4m3(__byte_perm(f[2 * e + 1], 0, 0x4431))};
                                mma<false>(o[x + e], y, p[h][0], p[h][1]);
                            }
                        }
                }
            };
            results(ph);
            if (p_low) {
#pragma unroll
                for (int h = 0; h < kH; ++h)
#pragma unroll
                    for (int y = 0; y < 2; ++y) pl[h][y] = transpose8(pl[h][y]);
                results(pl);
            }
            release(sv);
        }
        n += max(pc.tiles, 0);

        // ---- the warps' results
        if (nu > 0) warp_wait(smem_u32(&s_free), (nu - 1) & 1, bad);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], x);
            const int head = 2 * quad + e;
            if (row == 0) {
                s_m[warp * kSplitRows + head] = m[e];
                s_l[warp * kSplitRows + head] = l[e];
            }
            float* so = s_o + (warp * kSplitRows + head) * S::kPitch;
            if (head < rows && m[e] != -INFINITY) {
#pragma unroll
                for (int x = 0; x < kOut; ++x) {
                    so[16 * x + (S::kE4 ? 2 * row : row)] = o[x][e];
                    so[16 * x + (S::kE4 ? 2 * row + 1 : row + 8)] = o[x][2 + e];
                }
            }
        }
        // the mergers take it from here
        __syncwarp();
        if (lane == 0) mb_arrive(smem_u32(&s_done));
    }
    if (tid == 0 && *bad) report_expired(a);
}

// K or V by strides, as [outer][head][position][hd]: boxes of `box` positions of up to 128 bytes of a row
bool map_kv(CUtensorMap* map, int dtype, const void* base, int hd, int positions, int heads, int outer, int64_t pos_stride,
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

template <int HD, int KV>
cudaError_t launch_one(const AttendArgs& a, int sms, cudaStream_t st) {
    using S = Shape<HD, KV>;
    SplitArgs t;
    int box = S::kTile;
    if (a.table)
        while (a.by_ps.d % box) box >>= 1;
    t.box = box;
    t.groups = S::kTile / box;
    const int positions = a.table ? (int)a.by_ps.d : std::max(a.max_len, 1), outer = a.table ? a.n_pages : a.B;
    const int64_t outer_stride = a.table ? a.page_stride : a.batch_stride;
    if (!map_kv(&t.k, KV, a.k, HD, positions, a.Hkv, outer, a.pos_stride, a.head_stride, outer_stride, box) ||
        !map_kv(&t.v, KV, a.v, HD, positions, a.Hkv, outer, a.pos_stride, a.head_stride, outer_stride, box))
        return cudaErrorInvalidValue;
    t.a = a;
    // no more blocks than tiles there can be
    const int64_t RT = ((int64_t)a.Lq * (a.H / a.Hkv) + kSplitRows - 1) / kSplitRows;
    const int64_t most = std::min<int64_t>((int64_t)1 << 30, (int64_t)a.B * RT * a.Hkv) * (a.max_len / S::kTile + 1);
    const int grid = (int)std::min<int64_t>(sms, most);
    return launch_k(k_attend_split<HD, KV>, dim3(grid), dim3(kThreads), S::kSmem, st, t);
}

template <int HD, int KV>
cudaError_t prepare_one() {
    return cudaFuncSetAttribute(k_attend_split<HD, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<HD, KV>::kSmem);
}

}  // namespace

cudaError_t prepare_attend_split() {
    cudaError_t e = prepare_one<64, SD_F16>();
    if (e == cudaSuccess) e = prepare_one<128, SD_F16>();
    if (e == cudaSuccess) e = prepare_one<64, SD_BF16>();
    if (e == cudaSuccess) e = prepare_one<128, SD_BF16>();
    if (e == cudaSuccess) e = prepare_one<64, SD_E4M3>();
    if (e == cudaSuccess) e = prepare_one<128, SD_E4M3>();
    return e;
}

cudaError_t launch_attend_split(const AttendArgs& a, int hd, int sms, cudaStream_t st) {
    switch (a.kv_dtype) {
        case SD_F16: return hd == 64 ? launch_one<64, SD_F16>(a, sms, st) : launch_one<128, SD_F16>(a, sms, st);
        case SD_BF16: return hd == 64 ? launch_one<64, SD_BF16>(a, sms, st) : launch_one<128, SD_BF16>(a, sms, st);
        default: return hd == 64 ? launch_one<64, SD_E4M3>(a, sms, st) : launch_one<128, SD_E4M3>(a, sms, st);
    }
}

}  // namespace sd
