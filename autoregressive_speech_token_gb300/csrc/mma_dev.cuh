// Warp-level products (mma.sync m16n8k16) in attention, and what goes with them.
#pragma once
#include "attend_dev.cuh"

namespace sd {

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

}  // namespace sd
