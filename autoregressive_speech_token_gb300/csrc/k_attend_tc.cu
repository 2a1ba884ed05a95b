// Cross attention of many queries on the 5th-generation tensor cores: TMA loads,
// tcgen05 products with scores, probabilities and results in tensor memory.
//
// A work item is a pair of query tiles (128 queries of one head each) of one (row b,
// kv head g), against all of that row's positions in tiles of 128.  One block per SM
// takes whole items; where there are fewer items than SMs, they are cut into parts with a
// block each, and a second kernel joins the parts in order (64 queries over 1500 states, 16
// heads of 64: 12 us cut, 17 us whole; 128 over 32768, 16 heads of 128 in 8 groups: 38 and 324
// us).  Per position tile j and query tile i
//   S_i = Q_i K_j^T (fp32, 128 columns of tensor memory)
//   P_i = exp2(S_i scale log2(e) - m_i), rounded to the inputs' type, over S_i's columns
//   O_i += P_i V_j (fp32, head_dim columns)
// 8192 queries over 8000 and 8190 states, 16 heads of 128 in 8 groups, bf16: 608 us, 1.79 PFLOP/s, for some tens of
// calls, 655 us, 1.66 PFLOP/s, for hundreds, as the power limit then lowers the clocks (a library product of 8192^3:
// 1.92 and 1.73).  Bound by the tensor cores; heads of 64 by the exponentials (4 x 2048 over 2048: 81 us).
//
// One elected thread issues all products (from a lane compared by number it took 813 us
// for that first case), one warp all loads.  Two warpgroups each own one query
// tile, a thread per query: running maximum and sum need no exchange between
// threads, and while one warpgroup forms P of its tile the tensor cores work on the
// other's.  The reference m_i of the exponentials moves only when the maximum has
// grown by more than 2^8 (probabilities stay below 2^8, sums are fp32): results in
// tensor memory are seldom rescaled, and then by the same thread, which knows
// from S_i(j)'s completion that P_i V_(j-1) is complete (products of one thread
// complete in order).
//
// Rounding P to 16 bits is off by half a step of the output's own type and averages
// out over the positions; the sum uses the unrounded values.  fp16 probabilities
// carry a factor 2^7 to stay above the subnormal step.
//
// Every wait is bounded: on expiry the block records the error, lets its own copies
// and products finish (bounded), frees its tensor memory and returns.
#include "tc_dev.cuh"

namespace sd {
namespace {

constexpr int kM = 128, kN = 128;                    // queries and positions of a tile
constexpr int kSoftWarps = 8, kThreads = 32 * (kSoftWarps + 4);    // 2 softmax warpgroups; products, loads, 2 idle warps
constexpr int kMmaWarp = kSoftWarps, kLoadWarp = kSoftWarps + 1;
// Registers of a thread: 384 x 168 at launch = 2 x 128 x 216 + 128 x 72 (a softmax thread holds a row of 128 scores)
constexpr int kSoftRegs = 216, kOtherRegs = 72;
static_assert(256 * kSoftRegs + 128 * kOtherRegs <= 384 * 168, "the shares exceed what the block was launched with");
constexpr int kJoin = 4;                              // what cutting and joining items costs, in tiles
constexpr float kSlack = 8.f;                        // log2 of the growth that moves the reference
// Exponents from which a row subtracts its reference from the scores before they are scaled.  Below, s scale - ref in
// one rounding is off by at most 2^-3 with ref's own, and probabilities stay below 2^16; above, by whole powers of two.
constexpr float kFar = 0x1p20f;

struct alignas(128) TcArgs {
    CUtensorMap q, k, v, o;
    AttendArgs a;
    int32_t nq, pairs;                                // query tiles of a head, pairs of a (b, g)
    int32_t parts, blocks, join_blocks;               // items may be cut; blocks of the grid, and of the joining one
    int32_t staged;                                   // o is a map of the output
};

template <int HD>
struct Cfg {
    static constexpr int kPanel = kN * 128;                       // 128 rows of 64 elements, 128-byte swizzle
    static constexpr int kTileBytes = kPanel * (HD / 64);         // a Q, K or V tile
    static constexpr int kStages = HD == 128 ? 5 : 9;             // K and V tiles in flight
    // Heads of 64 leave room to hand results to TMA: 32 queries of a warp, swizzled.  (Stored row by row from the
    // registers they hold up the next item's first scores by about 2 us.)
    static constexpr bool kStaged = HD == 64;
    static constexpr int kSmem = (2 + kStages) * kTileBytes + (kStaged ? 8 * 32 * 128 : 0) + 1024;
    static constexpr uint32_t kO = 256;                           // tensor memory: S0, S1, O0, O1
};

__device__ __forceinline__ int tc_length(const AttendArgs& a, int b) {
    return min(max(a.len ? __ldcg(a.len + b) : a.max_len, 0), a.max_len);
}
__device__ __forceinline__ int tc_tiles(int len) { return (len + kN - 1) / kN; }

// How the items are shared out among `grid` blocks, found by every warp for itself; s_row (rows by falling length) and
// s_len are filled where there are at most 32 rows.  Called by all threads of a block.
struct Share {
    bool whole, sorted;
    int per;                                                       // tiles of a part at most
    int64_t per_b;                                                 // items of a row
    __device__ __forceinline__ int parts(int len) const { return max((tc_tiles(len) + per - 1) / per, 1); }
};
__device__ __forceinline__ Share tc_share(const TcArgs& t, int64_t grid, int* s_row, int* s_len) {
    const AttendArgs& a = t.a;
    const int lane = threadIdx.x & 31;
    Share s;
    s.per_b = (int64_t)a.Hkv * t.pairs;
    s.sorted = a.B <= 32;
    if (s.sorted) {
        const int mine = lane < a.B ? tc_length(a, lane) : -1;
        int rank = 0;
        for (int x = 0; x < a.B; ++x) {
            const int other = __shfl_sync(0xffffffffu, mine, x);
            rank += other > mine || (other == mine && x < lane);
        }
        if (threadIdx.x < a.B) {
            s_row[rank] = lane;
            s_len[lane] = mine;
        }
        __syncthreads();
    }
    // Each part has a block of its own: with `left` blocks more than items, parts of (all tiles) / left are short enough.
    // They cost their records and a second kernel, as much as about kJoin tiles.
    const int64_t left = grid - a.B * s.per_b;
    s.whole = true;
    s.per = 1;
    if (t.parts && left > 0) {
        int64_t all = 0;
        int most = 0;
        for (int b = lane; b < a.B; b += 32) {
            const int n = tc_tiles(s.sorted ? s_len[b] : tc_length(a, b));
            all += n;
            most = max(most, n);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            all += __shfl_xor_sync(0xffffffffu, all, o);
            most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        }
        const int64_t per = max((all * s.per_b + left - 1) / left, (int64_t)2);
        s.whole = per + kJoin >= most;
        s.per = s.whole ? max(most, 1) : (int)per;
    }
    return s;
}

template <int HD, bool BF>
__global__ void __launch_bounds__(kThreads, 1) k_attend_tc(const __grid_constant__ TcArgs t) {
    using C = Cfg<HD>;
    constexpr int kSt = C::kStages;
    constexpr float kShift = BF ? 0.f : 7.f;
    constexpr uint32_t kType = BF ? 1u : 0u;
    // fp32 result, A and B of one type, M = 128; scores: N = 128, both K-major; results: N = HD, V read along its rows
    constexpr uint32_t kIdescS = (1u << 4) | (kType << 7) | (kType << 10) | ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
    constexpr uint32_t kIdescO = (1u << 4) | (kType << 7) | (kType << 10) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
    extern __shared__ unsigned char smraw[];
    __shared__ __align__(8) unsigned long long s_full[kSt], s_empty[kSt], s_qfull, s_qempty, s_sfull[2], s_pfull[2][2], s_ofull[2], s_tail, s_never;
    __shared__ uint32_t s_tmem;
    __shared__ int s_bad, s_row[32], s_len[32];
    const AttendArgs& a = t.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sm = (smem_u32(smraw) + 1023u) & ~1023u;
    const uint32_t ring = sm + 2 * C::kTileBytes;

    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int s = 0; s < kSt; ++s) {
            mb_init(smem_u32(&s_full[s]), 1);
            mb_init(smem_u32(&s_empty[s]), 1);
        }
        mb_init(smem_u32(&s_qfull), 1);
        mb_init(smem_u32(&s_qempty), 1);
        mb_init(smem_u32(&s_tail), 1);
        mb_init(smem_u32(&s_never), 1);
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
    volatile int* bad = &s_bad;
    pdl_trigger();
    pdl_wait();

    const int G = a.H / a.Hkv;
    const int per_g = G * t.nq;                                    // query tiles of a (b, g)
    // ---- this block's share.  Whole items are taken in rounds, there and back over the blocks, the longest rows first
    // where a warp can sort them; or the block has one part of an item.
    const Share share = tc_share(t, gridDim.x, s_row, s_len);
    const int64_t per_b = share.per_b, items = per_b * a.B;
    int64_t round = 0;
    // A piece: tiles [i0, i0 + tiles) of an item; its parts are in blocks c_lo .. c_hi.
    struct Item {
        int b, g, len, i0, tiles, first, two, c_lo, c_hi;
    };
    auto next_item = [&](Item& p) -> bool {
        int64_t u;                                                 // item of its row
        if (share.whole) {
            const int64_t w = round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            if (w >= items) return false;
            const int r = (int)quot(w, per_b);
            u = w - r * per_b;
            p.b = share.sorted ? s_row[r] : r;
            p.len = share.sorted ? s_len[p.b] : tc_length(a, p.b);
            p.c_lo = p.c_hi = p.i0 = 0;
            p.tiles = tc_tiles(p.len);
        } else {
            if (round) return false;
            int64_t base = 0;                                      // blocks of the rows before (few rows: fewer items than SMs)
            int parts = 1;
            for (p.b = 0; p.b < a.B; ++p.b) {
                p.len = share.sorted ? s_len[p.b] : tc_length(a, p.b);
                parts = share.parts(p.len);
                if (blockIdx.x < base + parts * per_b) break;
                base += parts * per_b;
            }
            if (p.b == a.B) return false;
            u = quot(blockIdx.x - base, parts);
            p.c_lo = (int)(base + u * parts);
            p.c_hi = p.c_lo + parts - 1;
            const int n = tc_tiles(p.len), each = (n + parts - 1) / parts;   // equal parts, none empty
            p.i0 = ((int)blockIdx.x - p.c_lo) * each;
            p.tiles = min(n - p.i0, each);
        }
        ++round;
        p.g = (int)quot(u, t.pairs);
        p.first = (int)(u - (int64_t)p.g * t.pairs) * 2;
        p.two = p.first + 1 < per_g;
        return true;
    };

    if (warp >= kSoftWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      if (warp == kLoadWarp) {
        // ------------------------------------------------ loads (lane 0), and zeros behind a row's last position
        uint32_t n = 0, nq = 0, tail_n = 0;                        // tiles loaded, items; the last zeroed tile's number
        bool tails = false;
        bool ok = true;
        Item it;
        while (ok && next_item(it)) {
            if (!it.tiles) continue;
            if (nq > 0) ok = warp_wait(smem_u32(&s_qempty), (nq - 1) & 1, bad);
            if (!ok) break;
            if (lane == 0) {
                mb_expect(smem_u32(&s_qfull), (it.two ? 2 : 1) * C::kTileBytes);
                for (int i = 0; i <= it.two; ++i) {
                    const int x = it.first + i, h = it.g * G + x / t.nq, r = (x % t.nq) * kM;
                    for (int p = 0; p < HD / 64; ++p)
                        tma4(sm + i * C::kTileBytes + p * C::kPanel, &t.q, p * 64, h, r, it.b, smem_u32(&s_qfull));
                }
            }
            ++nq;
            for (int j = 0; j < 2 * it.tiles && ok; ++j, ++n) {
                const uint32_t s = n % kSt, turn = n / kSt;
                if (turn > 0) ok = warp_wait(smem_u32(&s_empty[s]), (turn - 1) & 1, bad);
                if (!ok) break;
                const uint32_t dst = ring + s * C::kTileBytes, mb = smem_u32(&s_full[s]);
                if (lane == 0) {
                    mb_expect(mb, C::kTileBytes);
                    for (int p = 0; p < HD / 64; ++p)
                        tma4(dst + p * C::kPanel, (j & 1) ? &t.v : &t.k, p * 64, it.g, (it.i0 + (j >> 1)) * kN, it.b, mb);
                }
                if (a.stall && blockIdx.x == 0) ok = warp_wait(smem_u32(&s_never), 0, bad, a.stall);
                const int rest = it.len - (it.i0 + it.tiles - 1) * kN;
                if (ok && j == 2 * it.tiles - 1 && rest < kN) {
                    // values behind the row's last position: 0 x anything must be 0
                    ok = warp_wait(mb, turn & 1, bad);
                    // one tail at a time: the products of the one before are complete (if its stage was loaded
                    // again since, that has been waited for)
                    if (ok && tails && tail_n + kSt > n)
                        ok = warp_wait(smem_u32(&s_empty[tail_n % kSt]), (tail_n / kSt) & 1, bad);
                    if (!ok) { ++n; break; }
                    for (int x = lane; x < (kN - rest) * 8 * (HD / 64); x += 32) {
                        const int p = x / ((kN - rest) * 8), y = x - p * (kN - rest) * 8;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + p * C::kPanel + rest * 128 + y * 16), "r"(0) : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mb_arrive(smem_u32(&s_tail));
                    tails = true;
                    tail_n = n;
                }
            }
        }
        if (!ok) {                                                 // bounded: this block's own copies
            for (uint32_t x = n > kSt ? n - kSt : 0; x < n; ++x) {
                const long long t0 = clock64();
                while (!mb_try(smem_u32(&s_full[x % kSt]), (x / kSt) & 1) && clock64() - t0 < kWaitClocks) {}
            }
            if (nq > 0) {
                const long long t0 = clock64();
                while (!mb_try(smem_u32(&s_qfull), (nq - 1) & 1) && clock64() - t0 < kWaitClocks) {}
            }
        }
      } else if (warp == kMmaWarp) {
        if (elect_one()) {
            // -------------------------------------------- products
            // descriptors: a tile or a K step further is an addition (addresses / 16 stay within their 14 bits)
            const uint64_t qdesc = sdesc(sm, 16), kdesc = sdesc(ring, 16), vdesc = sdesc(ring, C::kPanel);
            uint32_t n = 0, nq = 0, ntail = 0, np[2] = {0, 0}, no[2] = {0, 0};
            bool ok = true, any = false;
            Item it;
            while (ok && next_item(it)) {
                if (!it.tiles) continue;
                ok = mb_wait(smem_u32(&s_qfull), nq & 1, bad) && mb_wait(smem_u32(&s_full[n % kSt]), (n / kSt) & 1, bad);
                if (!ok) break;
                ++nq;
                tm_after();
                auto scores = [&](int i, uint32_t stage) {
                    const uint64_t q = qdesc + (uint32_t)(i * (C::kTileBytes >> 4)), kd = kdesc + stage * (uint32_t)(C::kTileBytes >> 4);
                    score_steps<HD, C::kPanel>(tmem + i * kN, q, kd, kIdescS);
                    commit(smem_u32(&s_sfull[i]));
                    any = true;
                };
                for (int i = 0; i <= it.two; ++i) scores(i, n % kSt);
                commit(smem_u32(&s_empty[n % kSt]));
                if (it.tiles == 1) commit(smem_u32(&s_qempty));
                ++n;
                const bool tail = it.len - (it.i0 + it.tiles - 1) * kN < kN;
                for (int j = 0; j < it.tiles && ok; ++j) {
                    const uint32_t sv = n % kSt, pv = (n / kSt) & 1, sk = (n + 1) % kSt, pk = ((n + 1) / kSt) & 1;
                    const bool more = j + 1 < it.tiles;
                    ok = mb_wait(smem_u32(&s_full[sv]), pv, bad);
                    if (ok && !more && tail) ok = mb_wait(smem_u32(&s_tail), ntail++ & 1, bad);
                    for (int i = 0; i <= it.two && ok; ++i) {
                        // the products of P's first half begin while its second half is formed
                        const uint64_t vd = vdesc + sv * (uint32_t)(C::kTileBytes >> 4);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            ok = mb_wait(smem_u32(&s_pfull[i][half]), np[i] & 1, bad);
                            if (!ok) break;
                            tm_after();
                            const uint32_t o = tmem + C::kO + i * HD, p = tmem + i * kN;
                            if (half == 0) result_steps<0, kN / 32>(o, p, vd, kIdescO, j > 0);
                            else result_steps<kN / 32, kN / 16>(o, p, vd, kIdescO, 1);
                        }
                        if (!ok) break;
                        ++np[i];
                        if (more) {
                            if (i == 0) ok = mb_wait(smem_u32(&s_full[sk]), pk, bad);
                            if (!ok) break;
                            scores(i, sk);
                        } else {
                            commit(smem_u32(&s_ofull[i]));
                            ++no[i];
                        }
                    }
                    if (!ok) break;
                    commit(smem_u32(&s_empty[sv]));
                    ++n;
                    if (more) {
                        commit(smem_u32(&s_empty[sk]));
                        ++n;
                        if (j + 2 == it.tiles) commit(smem_u32(&s_qempty));
                    }
                }
            }
            if (!ok && any) {                                      // bounded: products in flight
                commit(smem_u32(&s_ofull[0]));
                const long long t0 = clock64();
                while (!mb_try(smem_u32(&s_ofull[0]), no[0] & 1) && clock64() - t0 < kWaitClocks) {}
            }
        }
        __syncwarp();
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // ------------------------------------------------ softmax: a thread per query
        const int i = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + i * kN, to = tmem + lanes + C::kO + i * HD;
        const float sl = a.scale * kLog2e, slack = fminf(kSlack / sl, 3.0e38f), l_first = __ldcg(a.dead) ? NAN : 0.f;
        uint32_t ns = 0, no = 0;
        bool ok = true;
        Item it;
        while (ok && next_item(it)) {
            if (i && !it.two) continue;
            // the score that the reference stands at, and the one from which it moves (far rows: they subtract in every
            // tile); P = exp2((s - sub) sl - ref)
            float top = -INFINITY, limit = -INFINITY, sub = 0.f, ref = 0.f, l = l_first;
            for (int j = 0; j < it.tiles; ++j) {
                ok = warp_wait(smem_u32(&s_sfull[i]), ns & 1, bad);
                if (!ok) break;
                ++ns;
                tm_after();
                float s[kN];
#pragma unroll
                for (int c = 0; c < kN; c += 32) tm_ld32(ts + c, s + c);
                tm_wait_ld();
#pragma unroll
                for (int c = 0; c < kN; c += 16) after_wait(s + c);
                const int rest = it.len - (it.i0 + j) * kN;
                if (rest < kN) {
#pragma unroll
                    for (int c = 0; c < kN; ++c) s[c] = c < rest ? s[c] : -INFINITY;
                }
                float m0 = s[0], m1 = s[1], m2 = s[2], m3 = s[3];
#pragma unroll
                for (int c = 4; c + 8 <= kN; c += 8) {
                    m0 = max3(m0, s[c], s[c + 1]);
                    m1 = max3(m1, s[c + 2], s[c + 3]);
                    m2 = max3(m2, s[c + 4], s[c + 5]);
                    m3 = max3(m3, s[c + 6], s[c + 7]);
                }
                m0 = max3(m0, s[kN - 4], s[kN - 3]);
                m1 = max3(m1, s[kN - 2], s[kN - 1]);
                const float mx = fmaxf(max3(m0, m1, m2), m3);
                if (__any_sync(0xffffffffu, mx > limit)) {
                    const bool grow = mx > (sub != 0.f ? top : limit);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = !grow ? 1.f : top == -INFINITY ? 0.f : ex2((top - mx) * sl);
                        if (grow) top = mx;
                        l *= f;
                        if (j > 0) {
#pragma unroll
                            for (int c = 0; c < HD; c += 16) {
                                float o[16];
                                tm_ld16(to + c, o);
                                tm_wait_ld();
                                after_wait(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] *= f;
                                tm_st16(to + c, reinterpret_cast<uint32_t*>(o));
                            }
                            tm_wait_st();
                        }
                    }
                    const float m = top * sl;
                    const bool far = fabsf(m) >= kFar && m != -INFINITY;
                    sub = far ? top : 0.f;
                    ref = (far || m == -INFINITY ? 0.f : m) - kShift;
                    limit = far ? -INFINITY : top + slack;
                    if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                        for (int c = 0; c < kN; ++c) s[c] -= sub;
                    }
                }
                float2 l0 = make_float2(0.f, 0.f), l1 = l0;
                const float2 sl2 = make_float2(sl, sl), ref2 = make_float2(-ref, -ref);
#pragma unroll
                for (int c = 0; c < kN; c += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 x = fma2(make_float2(s[c + 2 * e], s[c + 2 * e + 1]), sl2, ref2);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        if (e & 1) l1 = add2(l1, x); else l0 = add2(l0, x);
                        p[e] = pack2<BF>(x.x, x.y);
                    }
                    tm_st16(ts + c / 2, p);
                    if (c == kN / 2 - 32 || c == kN - 32) {
                        tm_wait_st();
                        tm_before();
                        __syncwarp();
                        if (lane == 0) mb_arrive(smem_u32(&s_pfull[i][c == kN - 32]));
                    }
                }
                l += (l0.x + l0.y) + (l1.x + l1.y);
            }
            if (!ok) break;
            // ---- the result
            const float m = top * sl;
            const int x = it.first + i, h = it.g * G + x / t.nq, qi = (x % t.nq) * kM + r;
            if (it.tiles) {
                ok = warp_wait(smem_u32(&s_ofull[i]), no & 1, bad);
                if (!ok) break;
                ++no;
                tm_after();
            }
            const bool staged = C::kStaged && t.staged && it.c_lo == it.c_hi;
            const uint32_t stage = ring + kSt * C::kTileBytes + warp * 4096 + lane * 128;
            if (staged) {
                // the store of the item before has read this warp's part
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
            }
            uint16_t* out = static_cast<uint16_t*>(a.out) + it.b * a.o_batch + (int64_t)qi * a.o_stride + (int64_t)h * HD;
            auto put = [&](int c, const float* o, float inv) {         // 16 columns
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    uint32_t u[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        u[y] = l == 0.f ? 0u : pack2<BF>(o[e + 2 * y] * inv, o[e + 2 * y + 1] * inv);
                    if (staged)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + ((((c + e) >> 3) ^ (lane & 7)) << 4)),
                                     "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
                    else
                        *reinterpret_cast<uint4*>(out + c + e) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            };
            // a part of an item: its record of 4-column pieces [piece][query], then (maximum, sum) of each query
            float* rec = a.part + (int64_t)blockIdx.x * kTcRecord;
            const int at4 = i * (HD / 4) * kM + r, at_ml = 2 * kM * HD + 2 * (i * kM + r);
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                float o[16];
                if (it.tiles) {
                    tm_ld16(to + c, o);
                    tm_wait_ld();
                    after_wait(o);
                }
                if (it.c_lo == it.c_hi) {
                    if (staged || qi < a.Lq) put(c, o, 1.f / l);
                } else if (qi < a.Lq) {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        __stcg(reinterpret_cast<float4*>(rec) + at4 + (c / 4 + y) * kM, make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]));
                }
            }
            tm_before();
            if (staged) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                // queries behind the last are outside the map's range and are not written
                if (lane == 0 && qi < a.Lq) {
                    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];"
                                 ::"l"(reinterpret_cast<uint64_t>(&t.o)), "r"(0), "r"(h), "r"(qi), "r"(it.b), "r"(stage) : "memory");
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
            }
            if (it.c_lo != it.c_hi) {
                if (qi < a.Lq) __stcg(reinterpret_cast<float2*>(rec + at_ml), make_float2(m, l));
                continue;
            }
            if (a.lse && qi < a.Lq)
                a.lse[((int64_t)it.b * a.Lq + qi) * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l) - kShift) * kLn2;
        }
    }
    if (C::kStaged && warp < kSoftWarps && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    tm_before();
    __syncthreads();
    tm_after();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    if (tid == 0 && s_bad) report_expired(a);
}

// Joins the parts of the items that were cut: a block for each query tile of an item, the records in block order.
constexpr int kJoinThreads = 256;
template <int HD, bool BF>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(const __grid_constant__ TcArgs t) {
    constexpr float kShift = BF ? 0.f : 7.f;
    __shared__ int s_row[32], s_len[32];
    pdl_trigger();
    pdl_wait();
    const AttendArgs& a = t.a;
    const Share s = tc_share(t, t.blocks, s_row, s_len);
    if (s.whole) return;
    const int G = a.H / a.Hkv;
    constexpr int kCols = HD / 8 / (kJoinThreads / kM);            // blocks across a row's columns
    for (int64_t piece = blockIdx.x; piece < 2 * kCols * s.per_b * a.B; piece += gridDim.x) {
        const int64_t w = piece / (2 * kCols), u = w % s.per_b;
        const int i = (int)(piece / kCols & 1), b = (int)(w / s.per_b);
        // the blocks of the rows before
        int64_t base = 0;
        for (int x = 0; x < b; ++x) base += s.parts(tc_length(a, x)) * s.per_b;
        const int parts = s.parts(tc_length(a, b)), c_lo = (int)(base + u * parts), c_hi = c_lo + parts - 1;
        const int g = (int)(u / t.pairs), x = (int)(u - (int64_t)g * t.pairs) * 2 + i;
        if (c_lo == c_hi || x >= G * t.nq) continue;
        // a query of the tile, 8 of its columns; the records in batches whose loads are in flight together
        const int r = threadIdx.x % kM, c8 = (int)(piece % kCols) * (kJoinThreads / kM) + threadIdx.x / kM;
        const int h = g * G + x / t.nq, qi = (x % t.nq) * kM + r;
        if (qi >= a.Lq) continue;
        const int at4 = (i * (HD / 4) + 2 * c8) * kM + r, at_ml = 2 * kM * HD + 2 * (i * kM + r);
        auto record = [&](int c) { return a.part + (int64_t)c * kTcRecord; };
        float m = -INFINITY, l = 0.f, o[8] = {};
        constexpr int kBatch = 6;
        for (int c = c_lo; c <= c_hi; c += kBatch) {
            float2 ml[kBatch];
            float4 v[kBatch][2];
            float mx = m;
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                const float* p = record(min(c + y, c_hi));
                ml[y] = __ldcg(reinterpret_cast<const float2*>(p + at_ml));
                v[y][0] = __ldcg(reinterpret_cast<const float4*>(p) + at4);
                v[y][1] = __ldcg(reinterpret_cast<const float4*>(p) + at4 + kM);
            }
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                if (c + y > c_hi) ml[y] = make_float2(-INFINITY, 0.f);
                mx = fmaxf(mx, ml[y].x);
            }
            const float keep = m == -INFINITY ? 1.f : ex2(m - mx);
            m = mx;
            l *= keep;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= keep;
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                if (ml[y].y == 0.f) continue;                          // nothing in this part
                const float f = ml[y].x == -INFINITY ? 1.f : ex2(ml[y].x - m);
                l = fmaf(f, ml[y].y, l);
                o[0] = fmaf(v[y][0].x, f, o[0]); o[1] = fmaf(v[y][0].y, f, o[1]); o[2] = fmaf(v[y][0].z, f, o[2]); o[3] = fmaf(v[y][0].w, f, o[3]);
                o[4] = fmaf(v[y][1].x, f, o[4]); o[5] = fmaf(v[y][1].y, f, o[5]); o[6] = fmaf(v[y][1].z, f, o[6]); o[7] = fmaf(v[y][1].w, f, o[7]);
            }
        }
        const float inv = 1.f / l;
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = l == 0.f ? 0u : pack2<BF>(o[2 * e] * inv, o[2 * e + 1] * inv);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + b * a.o_batch + (int64_t)qi * a.o_stride + (int64_t)h * HD + c8 * 8) =
            make_uint4(y[0], y[1], y[2], y[3]);
        if (a.lse && c8 == 0)
            a.lse[((int64_t)b * a.Lq + qi) * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l) - kShift) * kLn2;
    }
}

// [batch][row][head][hd] of 16-bit elements by strides: boxes of rows of 64 elements of one head
bool map4(CUtensorMap* map, bool bf, const void* base, int hd, int heads, int rows, int batch, int64_t head_stride,
          int64_t row_stride, int64_t batch_stride, int box_rows = 128) {
    EncodeFn enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)batch};
    // the stride of a dimension of one element is not used: any legal value
    const cuuint64_t strides[3] = {heads > 1 ? (cuuint64_t)head_stride * 2 : (cuuint64_t)hd * 2,
                                   rows > 1 ? (cuuint64_t)row_stride * 2 : (cuuint64_t)hd * 2,
                                   batch > 1 ? (cuuint64_t)batch_stride * 2 : (cuuint64_t)hd * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1}, one[4] = {1, 1, 1, 1};
    return enc(map, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(base), dims,
               strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool BF>
cudaError_t launch_tc(const TcArgs& t, cudaStream_t st) {
    const cudaError_t e = launch_k(k_attend_tc<HD, BF>, dim3(t.blocks), dim3(kThreads), Cfg<HD>::kSmem, st, t);
    return e != cudaSuccess || !t.parts ? e : launch_k(k_attend_join<HD, BF>, dim3(t.join_blocks), dim3(kJoinThreads), 0, st, t);
}
template <int HD, bool BF>
cudaError_t prepare_tc() {
    return cudaFuncSetAttribute(k_attend_tc<HD, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<HD>::kSmem);
}

}  // namespace

cudaError_t prepare_attend_tc() {
    cudaError_t e = prepare_tc<64, false>();
    if (e == cudaSuccess) e = prepare_tc<128, false>();
    if (e == cudaSuccess) e = prepare_tc<64, true>();
    if (e == cudaSuccess) e = prepare_tc<128, true>();
    return e;
}

// *taken false: strides that a tensor map cannot hold, nothing launched
cudaError_t launch_attend_tc(const AttendArgs& a, int hd, int sms, cudaStream_t st, bool* taken) {
    TcArgs t;
    const bool bf = a.dtype == SD_BF16;
    *taken = map4(&t.q, bf, a.q, hd, a.H, a.Lq, a.B, hd, a.q_stride, a.q_batch) &&
             map4(&t.k, bf, a.k, hd, a.Hkv, a.max_len, a.B, a.head_stride, a.pos_stride, a.batch_stride) &&
             map4(&t.v, bf, a.v, hd, a.Hkv, a.max_len, a.B, a.head_stride, a.pos_stride, a.batch_stride);
    if (!*taken) return cudaSuccess;
    t.staged = hd == 64 && map4(&t.o, bf, a.out, hd, a.H, a.Lq, a.B, hd, a.o_stride, a.o_batch, 32);
    t.a = a;
    t.nq = (a.Lq + kM - 1) / kM;
    const int64_t pairs = ((int64_t)(a.H / a.Hkv) * t.nq + 1) / 2;
    t.pairs = (int32_t)pairs;
    // Items may be cut where there are fewer than SMs, and the longest is worth more than the second launch
    const int64_t items = (int64_t)a.B * a.Hkv * pairs, tiles = (a.max_len + kN - 1) / kN;
    t.parts = items < sms && tiles > 2 + kJoin;
    t.blocks = (int)std::min<int64_t>(sms, t.parts ? items * tiles : items);
    t.join_blocks = (int)std::min<int64_t>(3 * (int64_t)sms, 2 * items * (hd / 8 / (kJoinThreads / kM)));
    if (hd == 64) return bf ? launch_tc<64, true>(t, st) : launch_tc<64, false>(t, st);
    return bf ? launch_tc<128, true>(t, st) : launch_tc<128, false>(t, st);
}

}  // namespace sd
