// The requests' own part of attention with shared first pages: each request's positions behind the shared ones, and
// the join with what k_attend_shared.cu found for its group.
//
// Own parts are short (what a rollout has said since the fork) and there are many: a unit is (request, kv head, up
// to 8 query rows) with a block of two or four warps, twelve warps to an SM, so that the latencies of one unit pass
// under others.  (The split kernel, one block to an SM, takes 3.4 us a unit: 24 us for 64 x 16 units of 51 positions.)  A warp
// takes chunks of 16 or 32 positions in turn with the others, by itself: its copies (cp.async into two stages, 0 where
// no position is), scores and sums need no other warp until the unit ends.  The products are mma.sync in transposed form,
// S^T = K q^T and O^T = V^T P^T, as in the split kernel, with the same precision.
//
// Measured: 30 us for 776 units of up to 500 positions of 128, 50 MB from memory (1.7 TB/s); 19 us for 1024 units of up to 125
// positions of 64.  Bound by the chain of a unit: lengths, table, first copies, products, records, join.
#include "mma_dev.cuh"

namespace sd {
namespace {

constexpr int kStages = 2;

template <int HD>
struct Own {
    // Two warps a unit, six blocks to an SM, for heads of 64; four warps and three blocks for heads of 128, whose rows keep a
    // warp twice as long (64 x 16 units of 51 positions 19 and 22 us, 97 x 8 units of 430 positions of 128: 33 and 28 us)
    static constexpr int kWarps = HD == 64 ? 2 : 4, kThreads = 32 * kWarps, kBlocks = 12 / kWarps, kPerRow = kThreads / kSplitRows;
    static constexpr int kChunk = HD == 128 ? 16 : 32;            // positions of a warp at a time
    static constexpr int kRow = HD * 2, kCols = HD / 8;           // bytes and 16-byte columns of a position
    static constexpr int kBytes = kChunk * kRow;                  // a chunk's keys, or its values
    static constexpr int kPitch = HD + 4;
    static constexpr int kSmem = kWarps * kStages * 2 * kBytes + 128;
    static_assert(kWarps * kSplitRows * (kPitch + 2) * 4 <= kWarps * kStages * 2 * kBytes, "results take the stages' place");
    static __device__ __forceinline__ uint32_t at(int row, int col) { return row * kRow + ((col ^ (row & 7)) << 4); }
};

template <int HD, bool BF>
__global__ void __launch_bounds__(Own<HD>::kThreads, Own<HD>::kBlocks) k_attend_own(const __grid_constant__ AttendArgs a) {
    using S = Own<HD>;
    constexpr int kWarps = S::kWarps, kPerRow = S::kPerRow;
    constexpr int kSteps = HD / 16, kOut = HD / 16, kChunk = S::kChunk, kH = kChunk / 16, kVec = HD / kPerRow;
    constexpr float kShift = BF ? 0.f : 15.f;
    constexpr uint32_t kAll = 0xffffffffu >> (32 - kChunk);
    extern __shared__ unsigned char smraw[];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.H / a.Hkv, RT = (G + kSplitRows - 1) / kSplitRows, ps = (int)a.by_ps.d;
    const int unit = blockIdx.x, rg = unit / RT, tile = unit - rg * RT, b = rg / a.Hkv, g = rg - b * a.Hkv;
    const int rows = min(kSplitRows, G - tile * kSplitRows), h0 = g * G + tile * kSplitRows;
    // asked for together: whatever is not in L2 costs microseconds here
    const int serve = __ldcg(a.shared), len = __ldcg(a.len + b);
    SharedRow d;
    {
        const int4 x = __ldcg(reinterpret_cast<const int4*>(a.desc + b)), y = __ldcg(reinterpret_cast<const int4*>(a.desc + b) + 1);
        const longlong2 z = *reinterpret_cast<const longlong2*>(reinterpret_cast<const int4*>(a.desc + b) + 2);
        d.skip = x.x; d.r0 = x.y; d.size = x.z; d.tiles = x.w;
        d.rows = y.x; d.base = z.x; d.per = z.y;
    }
    if (!serve) return;
    const int own = (int)max(min(max(len, 0), a.max_len) - (int64_t)d.skip * ps, (int64_t)0);
    const bool dead = __ldcg(a.dead) != 0;
    const uint32_t sm = (smem_u32(smraw) + 127u) & ~127u, mine = sm + warp * (kStages * 2 * S::kBytes);

    // ---- copies of chunk `c` into a stage; the page of a lane's position is looked up a chunk ahead
    const int chunks = (own + kChunk - 1) / kChunk;
    const int32_t* table = a.table + (int64_t)b * a.table_stride + d.skip;
    auto lookup = [&](int c) -> int {
        const int p = c * kChunk + (lane & (kChunk - 1));
        return c < chunks && p < own ? __ldcg(table + a.by_ps.div((uint32_t)p)) : -1;
    };
    auto copy = [&](int c, int id, int stage) -> uint32_t {
        const int p = c * kChunk + (lane & (kChunk - 1));
        const bool have = (uint32_t)id < (uint32_t)a.n_pages;
        const int in = p - (int)(a.by_ps.div((uint32_t)p) * a.by_ps.d);
        const int64_t off = have ? id * a.page_stride + in * a.pos_stride + g * a.head_stride : -1;
        const uint32_t live = __ballot_sync(0xffffffffu, have) & kAll;
        const uint32_t to = mine + stage * 2 * S::kBytes;
#pragma unroll
        for (int j = 0; j < kChunk * S::kCols / 32; ++j) {
            const int y = lane + 32 * j, row = y / S::kCols, col = y % S::kCols;
            const int64_t o = __shfl_sync(0xffffffffu, off, row);
            const uint32_t n = o >= 0 ? 16 : 0;
            const int64_t at = o >= 0 ? o + col * 8 : 0;
            const uint32_t dst = to + S::at(row, col);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(static_cast<const uint16_t*>(a.k) + at), "r"(n) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + S::kBytes), "l"(static_cast<const uint16_t*>(a.v) + at), "r"(n) : "memory");
        }
        return live;
    };
    uint32_t live[kStages];
    {
        const int id0 = lookup(warp), id1 = lookup(warp + kWarps);
        live[0] = live[1] = 0;
        if (warp < chunks) live[0] = copy(warp, id0, 0);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (warp + kWarps < chunks) live[1] = copy(warp + kWarps, id1, 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    int ahead = lookup(warp + kStages * kWarps);

    // ---- the queries as the B operand: row `row`, 4 elements of each 16 a lane
    const int row = lane >> 2, quad = lane & 3, mi = lane >> 3, mr = lane & 7;
    const bool q_low = a.dtype == SD_F32 || (BF && a.dtype == SD_F16), p_low = a.dtype == SD_F32 || BF;
    uint32_t qh[kSteps][2], ql[kSteps][2];
    float scale[2];                                               // of this lane's two columns of the scores
    {
        float2 x[kSteps][2];
        const int64_t src = b * a.q_batch + (int64_t)(h0 + row) * HD;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t at = src + 16 * k + 2 * quad + 8 * e;
                x[k][e] = make_float2(0.f, 0.f);
                if (row < rows) {
                    if (a.dtype == SD_F32) x[k][e] = *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at);
                    else {
                        const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + at);
                        x[k][e] = a.dtype == SD_BF16 ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u))
                                                     : __half22float2(*reinterpret_cast<const __half2*>(&w));
                    }
                }
            }
        float down = 1.f, row_scale = a.scale * kLog2e;
        if (!BF && a.dtype != SD_F16) {
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
            for (int e = 0; e < 2; ++e) split2<BF>(x[k][e].x * down, x[k][e].y * down, qh[k][e], ql[k][e], kLow);
        scale[0] = __shfl_sync(0xffffffffu, row_scale, 8 * quad);
        scale[1] = __shfl_sync(0xffffffffu, row_scale, 8 * quad + 4);
    }

    // ---- what the group's common pages give to row rr: the records of the blocks that had part of them, in order
    const int rr = tid / kPerRow, c0 = tid % kPerRow * kVec;
    float pre[kVec], pm = -INFINITY, pl = 0.f;
#pragma unroll
    for (int x = 0; x < kVec; ++x) pre[x] = 0.f;
    if (d.skip && rr < rows) {
        const int row = (b - d.r0) * G + tile * kSplitRows + rr, pair = row / d.rows, m0 = pair * d.rows, local = row - m0;
        const int n = min(d.rows, d.size * G - m0), pairs = (d.size * G + d.rows - 1) / d.rows;
        const int64_t t0 = d.base + (int64_t)(g * pairs + pair) * (d.tiles + kShareLead) + kShareLead;
        const int c_lo = (int)quot(t0, d.per), c_hi = (int)quot(t0 + d.tiles - 1, d.per);
        const int64_t first = (int64_t)d.r0 * a.H + g * (d.size * G) + m0;
        constexpr int kBatch = 4;                                 // records whose loads are in flight together
        for (int c = c_lo; c <= c_hi; c += kBatch) {
            float2 ml[kBatch];
            float4 v[kBatch][kVec / 4];
            float mx = pm;
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                const int cc = min(c + y, c_hi);
                const float* p = shared_records(a, cc == c_lo, first, cc);
                ml[y] = __ldcg(reinterpret_cast<const float2*>(p + (int64_t)HD * n) + local);
#pragma unroll
                for (int x = 0; x < kVec / 4; ++x) v[y][x] = __ldcg(reinterpret_cast<const float4*>(p) + (c0 / 4 + x) * n + local);
            }
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                if (c + y > c_hi) ml[y] = make_float2(-INFINITY, 0.f);
                mx = fmaxf(mx, ml[y].x);
            }
            const float keep = pm == -INFINITY ? 1.f : ex2(pm - mx);
            pm = mx;
            pl *= keep;
#pragma unroll
            for (int x = 0; x < kVec; ++x) pre[x] *= keep;
#pragma unroll
            for (int y = 0; y < kBatch; ++y) {
                if (ml[y].y == 0.f) continue;                     // nothing in this part (NaN is something)
                const float f = ml[y].x == -INFINITY ? 1.f : ex2(ml[y].x - pm);
                pl = fmaf(f, ml[y].y, pl);
#pragma unroll
                for (int x = 0; x < kVec / 4; ++x) {
                    pre[4 * x] = fmaf(v[y][x].x, f, pre[4 * x]);
                    pre[4 * x + 1] = fmaf(v[y][x].y, f, pre[4 * x + 1]);
                    pre[4 * x + 2] = fmaf(v[y][x].z, f, pre[4 * x + 2]);
                    pre[4 * x + 3] = fmaf(v[y][x].w, f, pre[4 * x + 3]);
                }
            }
        }
    }

    // ---- this warp's chunks.  Its results: rows 2 quad and 2 quad + 1, dimensions `row` and `row` + 8 of each 16
    float o[kOut][4];
#pragma unroll
    for (int y = 0; y < kOut; ++y) o[y][0] = o[y][1] = o[y][2] = o[y][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int stage = 0;
    for (int c = warp; c < chunks; c += kWarps, stage ^= 1) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        const uint32_t kb = mine + stage * 2 * S::kBytes, vb = kb + S::kBytes, here = stage ? live[1] : live[0];
        if (here) {
            float s[kH][4];
            auto scores = [&](const uint32_t (&q)[kSteps][2], float (&x)[kH][4]) {
#pragma unroll
                for (int h = 0; h < kH; ++h) x[h][0] = x[h][1] = x[h][2] = x[h][3] = 0.f;
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int h = 0; h < kH; ++h) {
                        uint32_t f[4];
                        ldm4(kb + S::at(16 * h + (mi & 1) * 8 + mr, 2 * k + (mi >> 1)), f);
                        mma<BF>(x[h], f, q[k][0], q[k][1]);
                    }
            };
            scores(qh, s);
            if (q_low) {
                float x[kH][4];
                scores(ql, x);
#pragma unroll
                for (int h = 0; h < kH; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[h][e] = add_low(s[h][e], x[h][e]);
            }
#pragma unroll
            for (int h = 0; h < kH; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[h][e] *= scale[e & 1];
                    if (!((here >> (16 * h + 8 * (e >> 1) + row)) & 1)) s[h][e] = -INFINITY;
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
            // P^T as the B operand: each 8 positions x 8 rows transposed
            uint32_t ph[kH][2], plo[kH][2];
#pragma unroll
            for (int h = 0; h < kH; ++h)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float p0 = ex2((s[h][2 * y] - ref[0]) + kShift), p1 = ex2((s[h][2 * y + 1] - ref[1]) + kShift);
                    l[0] += p0;
                    l[1] += p1;
                    split2<BF>(p0, p1, ph[h][y], plo[h][y]);
                    ph[h][y] = transpose8(ph[h][y]);
                }
            auto results = [&](const uint32_t (&p)[kH][2]) {
#pragma unroll
                for (int h = 0; h < kH; ++h)
#pragma unroll
                    for (int x = 0; x < kOut; ++x) {
                        uint32_t f[4];
                        ldm4t(vb + S::at(16 * h + (mi >> 1) * 8 + mr, 2 * x + (mi & 1)), f);
                        mma<BF>(o[x], f, p[h][0], p[h][1]);
                    }
            };
            results(ph);
            if (p_low) {
#pragma unroll
                for (int h = 0; h < kH; ++h)
#pragma unroll
                    for (int y = 0; y < 2; ++y) plo[h][y] = transpose8(plo[h][y]);
                results(plo);
            }
        }
        __syncwarp();                                             // every lane has read the stage
        const int next = c + kStages * kWarps;
        uint32_t coming = 0;
        if (next < chunks) coming = copy(next, ahead, stage);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (stage) live[1] = coming;
        else live[0] = coming;
        ahead = lookup(next + kWarps);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // ---- the warps' results, and the common pages'
    float* s_o = reinterpret_cast<float*>(smraw + (sm - smem_u32(smraw)));        // [warp][row][HD]
    float* s_m = s_o + kWarps * kSplitRows * S::kPitch;
    float* s_l = s_m + kWarps * kSplitRows;
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
#pragma unroll
        for (int x = 0; x < kOut; ++x) {
            so[16 * x + row] = o[x][e];
            so[16 * x + row + 8] = o[x][2 + e];
        }
    }
    __syncthreads();
    if (rr >= rows) return;
    float mm = -INFINITY, ll = 0.f, val[kVec];
#pragma unroll
    for (int x = 0; x < kVec; ++x) val[x] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * kSplitRows + rr]);
    if (pl != 0.f) mm = fmaxf(mm, pm);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float mw = s_m[w * kSplitRows + rr];
        if (mw == -INFINITY) continue;
        const float f = ex2(mw - mm);
        ll = fmaf(f, s_l[w * kSplitRows + rr], ll);
        const float* so = s_o + (w * kSplitRows + rr) * S::kPitch + c0;
#pragma unroll
        for (int x = 0; x < kVec; ++x) val[x] = fmaf(f, so[x], val[x]);
    }
    if (pl != 0.f) {
        const float f = (pm == -INFINITY ? 1.f : ex2(pm - mm)) * ex2(kShift);
        ll = fmaf(f, pl, ll);
#pragma unroll
        for (int x = 0; x < kVec; ++x) val[x] = fmaf(f, pre[x], val[x]);
    }
    if (dead) ll = NAN;
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
    for (int x = 0; x < kVec; ++x) val[x] = ll == 0.f ? 0.f : val[x] * inv;
    const int h = h0 + rr;
    const int64_t at = b * a.o_batch + (int64_t)h * HD + c0;
#pragma unroll
    for (int x = 0; x < kVec; x += 4) storev<4>(a.out, at + x, a.dtype, val + x);
    if (c0 == 0 && a.lse) a.lse[(int64_t)b * a.H + h] = ll == 0.f ? -INFINITY : (mm + log2f(ll) - kShift) * kLn2;
}

template <int HD, bool BF>
cudaError_t prepare_one() {
    return cudaFuncSetAttribute(k_attend_own<HD, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, Own<HD>::kSmem);
}

}  // namespace

cudaError_t prepare_attend_own() {
    cudaError_t e = prepare_one<64, false>();
    if (e == cudaSuccess) e = prepare_one<128, false>();
    if (e == cudaSuccess) e = prepare_one<64, true>();
    if (e == cudaSuccess) e = prepare_one<128, true>();
    return e;
}

cudaError_t launch_attend_own(const AttendArgs& a, int hd, cudaStream_t st) {
    const int G = a.H / a.Hkv;
    const dim3 grid(a.B * a.Hkv * ((G + kSplitRows - 1) / kSplitRows));           // at most kSharedRows
    const bool bf = a.kv_dtype == SD_BF16;
    if (hd == 64) return bf ? launch_k(k_attend_own<64, true>, grid, dim3(Own<64>::kThreads), Own<64>::kSmem, st, a)
                            : launch_k(k_attend_own<64, false>, grid, dim3(Own<64>::kThreads), Own<64>::kSmem, st, a);
    return bf ? launch_k(k_attend_own<128, true>, grid, dim3(Own<128>::kThreads), Own<128>::kSmem, st, a)
              : launch_k(k_attend_own<128, false>, grid, dim3(Own<128>::kThreads), Own<128>::kSmem, st, a);
}

}  // namespace sd
