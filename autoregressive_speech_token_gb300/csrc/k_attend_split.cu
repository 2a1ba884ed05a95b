// Split-length attention: few queries over many positions, reached through a
// page table or by strides.
//
// A unit is (row b, kv head g, tile of up to 8 query rows of that head's group);
// a row is (query i, head of the group).  Its positions are cut into tiles of
// 64 or 128, and the tiles of all units, laid end to end, are dealt evenly to the
// resident blocks: every block streams the same number of bytes whatever the
// lengths are, and no host needs to know them.  A unit that ends up in several
// blocks is joined by the last of them to arrive, in block order (results do not
// depend on the order of arrival).
//
// The kernel is bound by the key and value bytes.  Each of a block's four warps
// streams its own 16 or 32 positions of a tile through a ring of cp.async stages and
// keeps its own running maximum and sum, so that the loop has no block-wide
// barrier.  Scores are mma.sync products (m16n8k16): a decode step's 8 rows fill
// half of the 16 rows of the instruction, and the other half holds the rows'
// low-order parts, so q (fp32 as fp16 high + low) and the probabilities enter with
// twice the bits at no further instruction.  (tcgen05 needs 64 or 128 rows, of
// which 1 to 8 would hold work, while the tensor time here is a fraction of
// the memory time.)
#include "attend_dev.cuh"

namespace sd {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
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
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two e4m3 values (a 16-bit half of w) as fp16x2: exact
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t w) {
    uint32_t d;
    asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(d) : "r"(w));
    return d;
}
// x, y rounded to the product's type, and what the rounding left
template <bool BF>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const float2 f = __bfloat1622float2(h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = *reinterpret_cast<const uint32_t*>(&l);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = *reinterpret_cast<const uint32_t*>(&l);
    }
}
// a / b for a >= 0, b > 0: in 32 bits where both fit (a 64-bit division costs a few hundred cycles)
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// high and low product; an infinite high product has no low one (0 * inf)
__device__ __forceinline__ float add_low(float hi, float lo) { return hi - hi == 0.f ? hi + lo : hi; }

__device__ __forceinline__ float2 load2(const void* p, int64_t i, int dt) {
    if (dt == SD_F32) return *reinterpret_cast<const float2*>(static_cast<const float*>(p) + i);
    if (dt == SD_F16) return __half22float2(*reinterpret_cast<const __half2*>(static_cast<const __half*>(p) + i));
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(static_cast<const __nv_bfloat16*>(p) + i));
}
__device__ __forceinline__ void store1(void* p, int64_t i, int dt, float v) {
    if (dt == SD_F32) static_cast<float*>(p)[i] = v;
    else if (dt == SD_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

template <int HD, int KV>
struct Shape {
    static constexpr bool kBf = KV == SD_BF16, kE4 = KV == SD_E4M3;
    static constexpr int kRow = HD * (kE4 ? 1 : 2);             // bytes of a position's row
    static constexpr int kCols = kRow / 16;                     // 16-byte columns
    static constexpr int kChunk = kRow >= 256 ? 16 : 32;        // positions of a warp's step: independent products hide
    static constexpr int kTile = kChunk * kWarps;               // each other's latency, registers allow 16 rows of 256 bytes
    static constexpr int kStage = 2 * kChunk * kRow;            // K and V of a step
    static constexpr int kStages = kStage >= 8192 ? 3 : 5;
    // What beginning and ending a unit costs (about 4 us), in tiles: the share of a block counts it
    static constexpr int kLead = 96 * 1024 / (kWarps * kStage);
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kMerge = kWarps * kSplitRows * (HD + 2) * 4;
    static constexpr int kSmem = kRing + kMerge;
    // fp16 probabilities are kept as 2^15 p: the smallest ones stay above fp16's subnormal step
    static constexpr float kShift = kBf ? 0.f : 15.f;
    // column of a row in shared memory: the 8 rows of a matrix fall into 8 different 16-byte bank groups
    static __device__ __forceinline__ uint32_t at(int row, int col) {
        return row * kRow + ((kCols >= 8 ? col ^ (row & 7) : col ^ ((row >> 1) & 3)) << 4);
    }
};

template <int HD, int KV>
__global__ void __launch_bounds__(kThreads, kSplitBlocksPerSm) k_attend_split(const __grid_constant__ AttendArgs a) {
    using S = Shape<HD, KV>;
    constexpr int kSteps = HD / 16, kOut = HD / 8, kSt = S::kStages, kChunk = S::kChunk, kTile = S::kTile;
    pdl_trigger();
    pdl_wait();
    extern __shared__ __align__(128) unsigned char smem[];
    float* s_o = reinterpret_cast<float*>(smem + S::kRing);              // [warp][row][HD]
    float* s_m = s_o + kWarps * kSplitRows * HD;                          // [warp][row]
    float* s_l = s_m + kWarps * kSplitRows;
    __shared__ int64_t s_sum[kWarps];
    __shared__ int64_t s_base;
    __shared__ int s_b, s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = lane >> 2, quad = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * kSt * S::kStage;
    const int G = a.H / a.Hkv;
    const int64_t M = (int64_t)a.Lq * G;                                  // query rows of a (b, kv head)
    const int64_t RT = (M + kSplitRows - 1) / kSplitRows;
    const int64_t U = RT * a.Hkv;                                         // units of a row b

    auto length = [&](int b) { return min(max(a.len ? __ldcg(a.len + b) : a.max_len, 0), a.max_len); };
    // tiles of a unit, the first kLead of them empty
    auto tiles = [&](int len) { return (len + kTile - 1) / kTile + S::kLead; };

    // ---- this block's share of all tiles
    int64_t mine = 0;
    for (int b = tid; b < a.B; b += kThreads) mine += tiles(length(b));
    // inclusive sums over the threads: of a row each where B <= kThreads
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    int64_t T = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) sum += s_sum[w];
        T += s_sum[w];
    }
    T *= U;
    const int64_t per = max(quot(T + gridDim.x - 1, gridDim.x), (int64_t)1);
    const int64_t t_begin = blockIdx.x * per, t_end = min(T, t_begin + per);
    if (t_begin >= t_end) return;
    // the row b that holds tile t_begin, and the first tile of that row
    if (a.B <= kThreads) {
        if ((sum - mine) * U <= t_begin && t_begin < sum * U) {
            s_b = tid;
            s_base = (sum - mine) * U;
        }
    } else {
        for (int64_t b0 = 0, before = 0; b0 < a.B; b0 += kThreads) {
            const int64_t b = b0 + tid;
            const int64_t n = b < a.B ? tiles(length((int)b)) * U : 0;
            int64_t x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            __syncthreads();
            if (lane == 31) s_sum[warp] = x;
            __syncthreads();
            int64_t base = before;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) base += s_sum[w];
                before += s_sum[w];
            }
            if (n && base + x - n <= t_begin && t_begin < base + x) {
                s_b = (int)b;
                s_base = base + x - n;
            }
            if (before > t_begin) break;
        }
    }
    __syncthreads();
    int b = s_b;
    int64_t base = s_base;                                                // first tile of row b

    for (int64_t t = t_begin; t < t_end;) {
        const int len = length(b);
        const int nt = tiles(len);
        const int64_t in_b = t - base;
        const int64_t u = quot(in_b, nt);
        const int64_t u0 = base + u * nt;                                  // the unit's tiles [u0, u0 + nt)
        const int64_t next = min(u0 + nt, t_end);
        // blocks with a part of its tiles (an empty unit: the block with its last empty tile)
        const int64_t real = min(u0 + S::kLead, u0 + nt - 1);
        const int c_lo = (int)quot(real, per), c_hi = (int)quot(u0 + nt - 1, per);
        if (next <= real) {                                                // only empty tiles here
            t = next;
            continue;
        }
        const int i0 = (int)max(t - u0 - S::kLead, (int64_t)0);
        const int i1 = (int)(next - u0) - S::kLead;
        const int g = (int)quot(u, RT);
        const int64_t m0 = (u - g * RT) * kSplitRows;
        const int rows = (int)min((int64_t)kSplitRows, M - m0);

        // ---- this warp's chunks: positions (i * 4 + warp) * kChunk ... for i in [i0, i1)
        int n = 0;
        {
            const int first = i0 * kTile + warp * kChunk;
            if (first < len) n = min(i1 - i0, (len - first + kTile - 1) / kTile);
        }
        const int64_t head = g * a.head_stride;
        // element offset of position p, -1 without one
        auto offset = [&](int p, int id) -> int64_t {
            if (!a.table) return b * a.batch_stride + p * a.pos_stride + head;
            const uint32_t page = a.by_ps.div((uint32_t)p);
            return (uint32_t)id < (uint32_t)a.n_pages
                       ? id * a.page_stride + (int64_t)((uint32_t)p - page * a.by_ps.d) * a.pos_stride + head : -1;
        };
        auto page_of = [&](int c) -> int {                                 // of this lane's position of chunk c
            const int p = (i0 + c) * kTile + warp * kChunk + (lane & (kChunk - 1));
            return a.table && c < n && p < len ? __ldcg(a.table + (int64_t)b * a.table_stride + a.by_ps.div((uint32_t)p)) : -1;
        };
        int ids[kSt];                                                     // page ids, a ring ahead of the copies
#pragma unroll
        for (int c = 0; c < kSt; ++c) ids[c] = page_of(c);
        // ---- queries of this lane: a row, 4 elements of each 16
        float2 x[kSteps][2];
        {
            const bool live = row < rows;
            const int64_t m = m0 + (live ? row : 0), qi = quot(m, G);
            const int64_t at = b * a.q_batch + qi * a.q_stride + ((int64_t)g * G + (m - qi * G)) * HD;
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int d = 16 * k + (S::kE4 ? 4 * quad + 2 * e : 2 * quad + 8 * e);
                    x[k][e] = live ? load2(a.q, at + d, a.dtype) : make_float2(0.f, 0.f);
                }
        }
        auto issue = [&](int c, int slot) {
            const int p = (i0 + c) * kTile + warp * kChunk + (lane & (kChunk - 1));
            const int64_t off = p < len ? offset(p, ids[slot]) : -1;
            ids[slot] = page_of(c + kSt);
            const uint32_t live = __ballot_sync(0xffffffffu, off >= 0);
            const uint32_t dst = ring + slot * S::kStage;
#pragma unroll
            for (int r0 = 0; r0 < kChunk; r0 += 32 / S::kCols) {
                const int r = r0 + lane / S::kCols, col = lane % S::kCols;
                const int64_t ro = __shfl_sync(0xffffffffu, off, r);
                const int64_t bytes = ro < 0 ? 0 : ro * (S::kE4 ? 1 : 2) + col * 16;
                const uint32_t size = ro < 0 ? 0 : 16;
                cp16(dst + S::at(r, col), static_cast<const char*>(a.k) + bytes, size);
                cp16(dst + kChunk * S::kRow + S::at(r, col), static_cast<const char*>(a.v) + bytes, size);
            }
            return live;
        };
        uint32_t live[kSt];                                               // live positions of the chunks in flight
#pragma unroll
        for (int s = 0; s < kSt; ++s) live[s] = 0;
#pragma unroll
        for (int c = 0; c < kSt - 1; ++c) {
            if (c < n) live[c] = issue(c, c);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        // ---- rows 0-7 of the A operand: the rounded rows; rows 8-15: what the rounding left
        uint32_t qa[kSteps][4];
        float row_scale = a.scale * kLog2e * (a.k_scale ? __ldcg(a.k_scale + g) : 1.f);
        {
            float down = 1.f;
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
                for (int e = 0; e < 2; ++e)
                    split2<S::kBf>(x[k][e].x * down, x[k][e].y * down, qa[k][2 * e], qa[k][2 * e + 1]);
        }
        float o[kOut][4];
#pragma unroll
        for (int n = 0; n < kOut; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        float mrow = -INFINITY, lrow = 0.f;

        for (int c0 = 0; c0 < n; c0 += kSt) {
#pragma unroll
            for (int s = 0; s < kSt; ++s) {
                const int c = c0 + s;
                if (c >= n) break;
                __syncwarp();
                if (c + kSt - 1 < n) live[(s + kSt - 1) % kSt] = issue(c + kSt - 1, (s + kSt - 1) % kSt);
                asm volatile("cp.async.commit_group;" ::: "memory");
                asm volatile("cp.async.wait_group %0;" ::"n"(kSt - 1) : "memory");
                __syncwarp();
                const uint32_t kb = ring + s * S::kStage, vb = kb + kChunk * S::kRow;
                const int mi = lane >> 3, mr = lane & 7;

                constexpr int kN = kChunk / 8, kH = kChunk / 16;          // products of 8, halves of 16 positions
                float sc[kN][4] = {};
                if constexpr (!S::kE4) {
#pragma unroll
                    for (int k = 0; k < kSteps; ++k)
#pragma unroll
                        for (int h = 0; h < kH; ++h) {
                            uint32_t f[4];
                            ldm4(kb + S::at(16 * h + (mi >> 1) * 8 + mr, 2 * k + (mi & 1)), f);
                            mma<S::kBf>(sc[2 * h], qa[k], f[0], f[1]);
                            mma<S::kBf>(sc[2 * h + 1], qa[k], f[2], f[3]);
                        }
                } else {
#pragma unroll
                    for (int k = 0; k < kSteps; k += 2)
#pragma unroll
                        for (int h = 0; h < kH; ++h) {
                            uint32_t f[4];
                            ldm4(kb + S::at(16 * h + (mi & 1) * 8 + mr, k + (mi >> 1)), f);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                mma<false>(sc[2 * h], qa[k + e], half2_of_e4m3(f[2 * e]), half2_of_e4m3(f[2 * e] >> 16));
                                mma<false>(sc[2 * h + 1], qa[k + e], half2_of_e4m3(f[2 * e + 1]),
                                           half2_of_e4m3(f[2 * e + 1] >> 16));
                            }
                        }
                }
                // this lane's scores: row `row`, positions 8j + 2 quad and the next
                float p[kN][2], mx = -INFINITY;
                const uint32_t lv = live[s] >> (2 * quad);
#pragma unroll
                for (int j = 0; j < kN; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = add_low(sc[j][e], sc[j][2 + e]) * row_scale;
                        p[j][e] = (lv >> (8 * j + e)) & 1 ? x : -INFINITY;
                        mx = fmaxf(mx, p[j][e] == p[j][e] ? p[j][e] : INFINITY);   // NaN reaches every result of its row
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(mrow, mx);
                if (__any_sync(0xffffffffu, mn > mrow)) {
                    const float keep = mrow == -INFINITY ? 0.f : ex2(mrow - mn);
                    lrow *= keep;
#pragma unroll
                    for (int x = 0; x < kOut; ++x) {
                        o[x][0] *= keep; o[x][1] *= keep;
                        o[x][2] *= keep; o[x][3] *= keep;
                    }
                    mrow = mn;
                }
                const float ref = mrow == -INFINITY ? 0.f : mrow - S::kShift;
                uint32_t pa[kH][4];
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    const float p0 = ex2(p[j][0] - ref), p1 = ex2(p[j][1] - ref);
                    lrow += p0 + p1;
                    split2<S::kBf>(p0, p1, pa[j / 2][2 * (j & 1)], pa[j / 2][2 * (j & 1) + 1]);
                }
                if constexpr (!S::kE4) {
#pragma unroll
                    for (int h = 0; h < kH; ++h)
#pragma unroll
                        for (int x = 0; x < kOut; x += 2) {
                            uint32_t f[4];
                            ldm4t(vb + S::at(16 * h + (mi & 1) * 8 + mr, x + (mi >> 1)), f);
                            mma<S::kBf>(o[x], pa[h], f[0], f[1]);
                            mma<S::kBf>(o[x + 1], pa[h], f[2], f[3]);
                        }
                } else {
                    // a transposed matrix of byte pairs: even dimensions in the low bytes, odd ones in the high
#pragma unroll
                    for (int h = 0; h < kH; ++h)
#pragma unroll
                        for (int x = 0; x < kOut; x += 4) {
                            uint32_t f[4];
                            ldm4t(vb + S::at(16 * h + (mi & 1) * 8 + mr, x / 2 + (mi >> 1)), f);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                mma<false>(o[x + 2 * e], pa[h], half2_of_e4m3(__byte_perm(f[2 * e], 0, 0x4420)),
                                           half2_of_e4m3(__byte_perm(f[2 * e + 1], 0, 0x4420)));
                                mma<false>(o[x + 2 * e + 1], pa[h], half2_of_e4m3(__byte_perm(f[2 * e], 0, 0x4431)),
                                           half2_of_e4m3(__byte_perm(f[2 * e + 1], 0, 0x4431)));
                            }
                        }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();

        // ---- the four warps' results
        lrow += __shfl_xor_sync(0xffffffffu, lrow, 1);
        lrow += __shfl_xor_sync(0xffffffffu, lrow, 2);
        if (quad == 0) {
            s_m[warp * kSplitRows + row] = mrow;
            s_l[warp * kSplitRows + row] = lrow;
        }
        float* so = s_o + (warp * kSplitRows + row) * HD;
        if (row < rows) {
#pragma unroll
            for (int x = 0; x < kOut; ++x) {
                const float v0 = add_low(o[x][0], o[x][2]), v1 = add_low(o[x][1], o[x][3]);
                if constexpr (S::kE4) {
                    const int d = 16 * (x / 2) + 4 * quad + (x & 1);
                    so[d] = v0;
                    so[d + 2] = v1;
                } else {
                    *reinterpret_cast<float2*>(so + 8 * x + 2 * quad) = make_float2(v0, v1);
                }
            }
        }
        __syncthreads();
        const float vs = a.v_scale ? __ldcg(a.v_scale + g) : 1.f;
        auto put = [&](int r, int d, float val, float mm, float ll) {
            const int64_t m = m0 + r, qi = quot(m, G);
            const int64_t h = (int64_t)g * G + (m - qi * G);
            store1(a.out, b * a.o_batch + qi * a.o_stride + h * HD + d, a.dtype, ll == 0.f ? 0.f : val * vs / ll);
            if (d == 0 && a.lse)
                a.lse[((int64_t)b * a.Lq + qi) * a.H + h] = ll == 0.f ? -INFINITY : (mm + log2f(ll) - S::kShift) * kLn2;
        };
        float* rec = a.part + (int64_t)(2 * blockIdx.x + (real >= t_begin ? 1 : 0)) * kSplitRecord;
        for (int x = tid; x < rows * HD; x += kThreads) {
            const int r = x / HD, d = x % HD;
            float mm = -INFINITY, ll = 0.f, val = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * kSplitRows + r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = s_m[w * kSplitRows + r], f = mw == -INFINITY ? 0.f : ex2(mw - mm);
                ll = fmaf(f, s_l[w * kSplitRows + r], ll);
                if (mw != -INFINITY) val = fmaf(f, s_o[(w * kSplitRows + r) * HD + d], val);
            }
            if (c_lo == c_hi) {
                put(r, d, val, mm, ll);
            } else {
                __stcg(rec + r * HD + d, val);
                if (d == 0) {
                    __stcg(rec + kSplitRows * 128 + 2 * r, mm);
                    __stcg(rec + kSplitRows * 128 + 2 * r + 1, ll);
                }
            }
        }
        if (c_lo != c_hi) {
            // ---- the last block of the unit to arrive joins the records in block order
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                s_last = atomicAdd(a.cnt + c_lo, 1) == c_hi - c_lo;
                __threadfence();
            }
            __syncthreads();
            if (s_last) {
                for (int x = tid; x < rows * HD; x += kThreads) {
                    const int r = x / HD, d = x % HD;
                    float mm = -INFINITY, ll = 0.f, val = 0.f;
                    for (int c = c_lo; c <= c_hi; ++c) {
                        const float* p = a.part + (int64_t)(2 * c + (c == c_lo ? 1 : 0)) * kSplitRecord;
                        const float mc = __ldcg(p + kSplitRows * 128 + 2 * r), lc = __ldcg(p + kSplitRows * 128 + 2 * r + 1);
                        const float oc = __ldcg(p + r * HD + d);
                        if (mc == -INFINITY) continue;
                        const float mx = fmaxf(mm, mc);
                        const float f0 = mm == -INFINITY ? 0.f : ex2(mm - mx), f1 = ex2(mc - mx);
                        ll = ll * f0 + lc * f1;
                        val = val * f0 + oc * f1;
                        mm = mx;
                    }
                    put(r, d, val, mm, ll);
                }
                if (tid == 0) a.cnt[c_lo] = 0;
            }
        }
        __syncthreads();
        t = next;
        if (t - base == nt * U) {
            base = t;
            ++b;
        }
    }
}

template <int HD, int KV>
cudaError_t launch_one(const AttendArgs& a, int sms, cudaStream_t st) {
    using S = Shape<HD, KV>;
    // no more blocks than tiles there can be
    const int64_t RT = ((int64_t)a.Lq * (a.H / a.Hkv) + kSplitRows - 1) / kSplitRows;
    const int64_t most = std::min<int64_t>((int64_t)1 << 30, (int64_t)a.B * RT * a.Hkv) * (a.max_len / S::kTile + 1);
    const int grid = (int)std::min<int64_t>(kSplitBlocksPerSm * sms, most);
    return launch_k(k_attend_split<HD, KV>, dim3(grid), dim3(kThreads), S::kSmem, st, a);
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
