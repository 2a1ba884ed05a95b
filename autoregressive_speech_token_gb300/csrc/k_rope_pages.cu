// sd_rope_init and sd_rope_write_pages: rotary positions with one or several axes,
// fused with the write of keys and values into a cache's pages.
//
// Pair i of a head, (x_i, x_{i+hd/2}), turns by pos[axis(i)] theta^(-2i/hd).  The
// frequency is kept as a 64-bit fraction of a turn: position times fraction modulo
// 2^64 is the angle of any position without a long reduction (one integer
// product; 64-bit floats would be needed otherwise).  The fraction is off by less than one of its
// units, so the angle at position 2^31 by less than 2^-33 of a turn; a fraction rounded to a
// double's 53 bits would be off by 2^-25 of a turn there.  Its upper 32 bits, taken
// to the nearest quarter turn, leave |r| <= 1/8 turn, which fp32 holds to 2^-28
// of a turn, and sincospif of it gives cos and sin to about their last bit.
//
// The call moves its data once and is bound by memory.  A block takes one token or four:
// their sines and cosines are formed once, in shared memory, for all heads, while the
// block's first loads are in flight; then each thread rotates 8 pairs of one head per
// step with 16-byte loads and stores.  30011 tokens (483 MB) take 84 us, 0.85 of the copy rate,
// into single positions of random pages.  Into e4m3 pages (424 MB) they take 93 us, 0.67: as many scattered rows,
// half as long (with and without scales alike); fp32 tokens into fp16 pages (847 MB) 129 us, 0.97.
#include <cmath>

#include "pages_dev.cuh"

namespace sd {
namespace {


struct RopeArgs {
    sd_rope rope;
    const int32_t *pos, *slot;
    const void *q, *k, *v;
    void* q_out;
    sd_pages c;
    FastDiv by_ps;
    int64_t pos_stride, q_stride, qo_stride, kv_stride, slots;
    int32_t n, H, rotate;
};

// 8 consecutive elements as fp32
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f;
            if constexpr (std::is_same<T, __half>::value)
                f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            else
                f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

struct e4m3_t { uint8_t v; };

template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    } else if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3)
                         << (16 * (i & 1));
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// A number as the sum of two doubles: these steps are good to about 2^-100 of it, whatever a host compiler contracts.
struct Twice {
    double hi, lo;
};
inline Twice sum(double a, double b) {                     // |a| >= |b|
    const double s = a + b;
    return {s, b - (s - a)};
}
inline Twice times(Twice a, Twice b) {
    const double p = a.hi * b.hi;
    return sum(p, std::fma(a.hi, b.lo, std::fma(a.lo, b.hi, std::fma(a.hi, b.hi, -p))));
}
// One Newton step from the double root: x = r + (a - r^2) / (2 r)
inline Twice root(Twice a) {
    const double r = std::sqrt(a.hi);
    return sum(r, (std::fma(-r, r, a.hi) + a.lo) / (2.0 * r));
}
// One correction of the double quotient
inline Twice inverse(Twice a) {
    const double r = 1.0 / a.hi;
    return sum(r, std::fma(-r, a.lo, std::fma(-r, a.hi, 1.0)) * r);
}

template <typename T, typename TC, int HD, int kThreads>
__global__ void __launch_bounds__(kThreads) k_rope_pages(const __grid_constant__ RopeArgs a, int tokens) {
    constexpr int kHalf = HD / 2, kChunks = kHalf / 8;   // 8-pair chunks of a head
    pdl_trigger();
    pdl_wait();
    extern __shared__ float s_cs[];                        // [tokens][cos kHalf | sin kHalf]
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * tokens;
    const int nt = min(tokens, a.n - t0);
    const int heads = a.H + 2 * a.c.n_kv_head, per = heads * kChunks;   // work items of a token: q, k and v heads
    const int items = nt * per;
    float x[8], y[8];
    int32_t slot = -1;
    auto place = [&](int i, int& t, int& head, int& d) {
        t = i / per;
        const int j = i - t * per;
        head = j / kChunks;
        d = (j - head * kChunks) * 8;
    };
    auto load = [&](int i) {
        int t, head, d;
        place(i, t, head, d);
        const int64_t tok = t0 + t;
        slot = a.slot[tok];
        const T* src = head < a.H ? static_cast<const T*>(a.q) + tok * a.q_stride + head * HD
                       : head < a.H + a.c.n_kv_head ? static_cast<const T*>(a.k) + tok * a.kv_stride + (head - a.H) * HD
                                                    : static_cast<const T*>(a.v) + tok * a.kv_stride + (head - a.H - a.c.n_kv_head) * HD;
        load8(src + d, x);
        load8(src + d + kHalf, y);
    };
    if (tid < items) load(tid);
    if (a.rotate) {
        for (int i = tid; i < nt * kHalf; i += kThreads) {
            const int t = i / kHalf, p = i - t * kHalf;
            const int64_t pos = a.pos[a.rope.axis[p] * a.pos_stride + t0 + t];
            const uint32_t turn = (uint32_t)((uint64_t)pos * a.rope.turn[p] >> 32);
            const uint32_t quarter = (turn + (1u << 29)) >> 30;
            float s, c;
            sincospif((float)(int32_t)(turn - (quarter << 30)) * 0x1p-31f, &s, &c);
            // a quarter turn takes (c, s) to (-s, c)
            const float cc = (quarter & 1) ? -s : c, ss = (quarter & 1) ? c : s;
            s_cs[t * HD + p] = (quarter & 2) ? -cc : cc;
            s_cs[t * HD + kHalf + p] = (quarter & 2) ? -ss : ss;
        }
        __syncthreads();
    }
    for (int i = tid; i < items; i += kThreads) {
        if (i != tid) load(i);
        if (slot < 0 || slot >= a.slots) continue;
        int t, head, d;
        place(i, t, head, d);
        const bool is_q = head < a.H, is_k = !is_q && head < a.H + a.c.n_kv_head;
        if (a.rotate && (is_q || is_k)) {
            const float* cs = s_cs + t * HD + d;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float c = cs[e], s = cs[kHalf + e];
                const float u = x[e] * c - y[e] * s, w = x[e] * s + y[e] * c;
                x[e] = u;
                y[e] = w;
            }
        }
        if (is_q) {
            T* dst = static_cast<T*>(a.q_out) + (int64_t)(t0 + t) * a.qo_stride + head * HD + d;
            store8(dst, x);
            store8(dst + kHalf, y);
        } else {
            const int g = is_k ? head - a.H : head - a.H - a.c.n_kv_head;
            const uint32_t page = a.by_ps.div((uint32_t)slot);
            const int64_t off = page * a.c.page_stride + (slot - page * a.by_ps.d) * a.c.pos_stride + g * a.c.head_stride + d;
            if constexpr (sizeof(TC) == 1) {
                const float* sp = is_k ? a.c.k_scale_dev : a.c.v_scale_dev;
                const float sc = sp ? sp[g] : 1.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = x[e] / sc;
                    y[e] = y[e] / sc;
                }
            }
            TC* dst = static_cast<TC*>(is_k ? a.c.k_dev : a.c.v_dev) + off;
            store8(dst, x);
            store8(dst + kHalf, y);
        }
    }
}

template <typename T, typename TC>
cudaError_t launch_hd(const RopeArgs& a, cudaStream_t st) {
    // Many tokens: four to a block of 128 threads, so that an SM holds many blocks at different points (30011 tokens of
    // 16 + 8 + 8 heads of 128, bf16: 84 us; 87 us with two tokens, 86 with eight, 110 with 512 threads).  Few tokens: one
    // each and more threads, so that no thread takes a third piece.
    const bool many = a.n > 512;
    const int tokens = many ? 4 : 1;
    const dim3 grid((a.n - 1) / tokens + 1);
    const size_t smem = sizeof(float) * tokens * a.c.head_dim;
    if (a.c.head_dim == 64)
        return many ? launch_k(k_rope_pages<T, TC, 64, 128>, grid, dim3(128), smem, st, a, tokens)
                    : launch_k(k_rope_pages<T, TC, 64, 256>, grid, dim3(256), smem, st, a, tokens);
    return many ? launch_k(k_rope_pages<T, TC, 128, 128>, grid, dim3(128), smem, st, a, tokens)
                : launch_k(k_rope_pages<T, TC, 128, 256>, grid, dim3(256), smem, st, a, tokens);
}
template <typename T>
cudaError_t launch_cache(const RopeArgs& a, cudaStream_t st) {
    return a.c.dtype == SD_F16 ? launch_hd<T, __half>(a, st)
           : a.c.dtype == SD_BF16 ? launch_hd<T, __nv_bfloat16>(a, st) : launch_hd<T, e4m3_t>(a, st);
}

}  // namespace
}  // namespace sd

extern "C" {

int sd_rope_init(int32_t head_dim, double theta, int32_t n_axes, const int32_t* pairs, int32_t interleaved,
                 sd_rope* out) {
    using namespace sd;
    static const char* who = "sd_rope_init";
    if (!out) return op_fail(SD_ERR_INVALID_ARG, "%s: out is NULL", who);
    if (head_dim != 64 && head_dim != 128)
        return op_fail(SD_ERR_UNSUPPORTED, "%s: head_dim %d is not 64 or 128", who, head_dim);
    const int half = head_dim / 2;
    if (!(theta > 1.0) || !std::isfinite(theta)) return op_fail(SD_ERR_INVALID_ARG, "%s: theta %g", who, theta);
    if (n_axes < 1 || n_axes > 4 || (n_axes > 1 && !pairs))
        return op_fail(SD_ERR_INVALID_ARG, "%s: %d axes (1 to 4), pairs %s", who, n_axes, pairs ? "given" : "NULL");
    int left[4] = {half, 0, 0, 0};
    if (pairs) {
        int64_t sum = 0;
        for (int a = 0; a < n_axes; ++a) {
            if (pairs[a] < 0) return op_fail(SD_ERR_INVALID_ARG, "%s: pairs[%d] = %d", who, a, pairs[a]);
            left[a] = pairs[a];
            sum += pairs[a];
        }
        if (sum != half) return op_fail(SD_ERR_INVALID_ARG, "%s: the axes' pairs do not add up to head_dim/2", who);
    }
    // theta^(-2/head_dim): 32 and 64 are powers of two, so square roots lead to it; the pairs are its powers, times 1/(2 pi)
    Twice step = {theta, 0.0}, f = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};
    for (int n = 1; n < half; n *= 2) step = root(step);
    step = inverse(step);
    *out = sd_rope{};
    out->head_dim = head_dim;
    out->n_axes = n_axes;
    for (int i = 0, a = 0; i < half; ++i) {
        while (!left[a]) a = (a + 1) % n_axes;
        out->axis[i] = (uint8_t)a;
        --left[a];
        if (interleaved) a = (a + 1) % n_axes;
        // turns per position, below 1/6, in units of 2^-64, rounded down; below 2^-11 the high part has a fraction
        const double high = std::floor(std::ldexp(f.hi, 64));
        out->turn[i] = (uint64_t)high + (uint64_t)(int64_t)std::floor(std::ldexp(f.lo, 64) + (std::ldexp(f.hi, 64) - high));
        f = times(f, step);
    }
    return SD_OK;
}

int sd_rope_write_pages(const sd_rope* rope, const int32_t* pos_dev, int64_t pos_stride, const int32_t* slot_dev,
                        int32_t n, int32_t dtype, const void* q_dev, int64_t q_stride, void* q_out_dev,
                        int64_t q_out_stride, int32_t n_head, const void* k_dev, const void* v_dev, int64_t kv_stride,
                        const sd_pages* cache, void* stream) {
    using namespace sd;
    static const char* who = "sd_rope_write_pages";
    if (n == 0) return SD_OK;
    RopeArgs a;
    if (int rc = check_pages(who, cache, &a.c)) return rc;
    const int b = dtype == SD_E4M3 ? 0 : dtype_bytes(dtype);
    if (!b) return op_fail(SD_ERR_INVALID_ARG, "%s: type %d is not SD_F32, SD_F16 or SD_BF16", who, dtype);
    if (n < 0 || n_head < 0) return op_fail(SD_ERR_INVALID_ARG, "%s: n %d, n_head %d", who, n, n_head);
    if (!slot_dev || !k_dev || !v_dev || (rope && !pos_dev))
        return op_fail(SD_ERR_INVALID_ARG, "%s: NULL argument", who);
    if ((n_head > 0) != (q_dev != nullptr) || (n_head > 0) != (q_out_dev != nullptr))
        return op_fail(SD_ERR_INVALID_ARG, "%s: q_dev and q_out_dev come with n_head > 0, and only then", who);
    if (!aligned16(k_dev) || !aligned16(v_dev) || !aligned16(q_dev) || !aligned16(q_out_dev) ||
        !stride16(kv_stride, b) || !stride16(q_stride, b) || !stride16(q_out_stride, b))
        return op_fail(SD_ERR_INVALID_ARG, "%s: pointers and row strides must be multiples of 16 bytes", who);
    if (q_dev && q_dev == q_out_dev && q_stride != q_out_stride)
        return op_fail(SD_ERR_INVALID_ARG, "%s: q_out_dev is q_dev with another stride", who);
    if (rope) {
        if (rope->head_dim != a.c.head_dim || rope->n_axes < 1 || rope->n_axes > 4)
            return op_fail(SD_ERR_INVALID_ARG, "%s: rope is for head_dim %d, the cache has %d", who, rope->head_dim,
                           a.c.head_dim);
        for (int i = 0; i < rope->head_dim / 2; ++i)
            if (rope->axis[i] >= rope->n_axes) return op_fail(SD_ERR_INVALID_ARG, "%s: rope is not initialised", who);
        a.rope = *rope;
    }
    a.pos = pos_dev; a.slot = slot_dev; a.q = q_dev; a.k = k_dev; a.v = v_dev; a.q_out = q_out_dev;
    a.pos_stride = pos_stride; a.q_stride = q_stride; a.qo_stride = q_out_stride; a.kv_stride = kv_stride;
    a.slots = (int64_t)a.c.n_pages * a.c.page_size; a.n = n; a.H = n_head; a.rotate = rope != nullptr;
    a.by_ps = FastDiv((uint32_t)a.c.page_size);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == SD_F32 ? launch_cache<float>(a, st)
                          : dtype == SD_F16 ? launch_cache<__half>(a, st) : launch_cache<__nv_bfloat16>(a, st);
    if (e != cudaSuccess) return op_fail(SD_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return SD_OK;
}

}  // extern "C"
