// sd_attend_pages and sd_attend_cross: softmax attention of queries of any number
// over key/value positions reached through a page table or by strides.
//
// The plainest form that is right for every case: one block per query head, a
// running maximum and sum over tiles of kTile positions, fp32 throughout.
#include <new>

#include "pages_dev.cuh"

struct sd_attn_ws {
    int device = 0;
};

namespace sd {
namespace {

constexpr int kTile = 128;

struct AttendArgs {
    const void *q, *k, *v;
    void* out;
    float* lse;
    const int32_t *table, *len;
    const float *k_scale, *v_scale;
    FastDiv by_ps;
    int64_t batch_stride, page_stride, head_stride, pos_stride, q_batch, q_stride, o_batch, o_stride;
    int32_t B, Lq, H, Hkv, n_pages, table_stride, max_len, dtype, kv_dtype;
    float scale;
};

__device__ __forceinline__ float load1(const void* p, int64_t i, int dt) {
    if (dt == SD_F32) return static_cast<const float*>(p)[i];
    if (dt == SD_F16) return __half2float(static_cast<const __half*>(p)[i]);
    if (dt == SD_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p)[i], __NV_E4M3);
    return __half2float(__half(h));
}
__device__ __forceinline__ void store1(void* p, int64_t i, int dt, float v) {
    if (dt == SD_F32) static_cast<float*>(p)[i] = v;
    else if (dt == SD_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

template <int HD>
__global__ void __launch_bounds__(kTile) k_attend(const AttendArgs a) {
    pdl_trigger();
    pdl_wait();
    __shared__ float s_q[HD], s_p[kTile], s_red[kTile / 32];
    __shared__ int64_t s_off[kTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, g = h / (a.H / a.Hkv);
    const float ks = a.k_scale ? a.k_scale[g] : 1.f, vs = a.v_scale ? a.v_scale[g] : 1.f;
    for (int64_t bi = blockIdx.x; bi < (int64_t)a.B * a.Lq; bi += gridDim.x) {
        const int b = (int)(bi / a.Lq), i = (int)(bi - (int64_t)b * a.Lq);
        const int len = min(max(a.len ? a.len[b] : a.max_len, 0), a.max_len);
        for (int d = tid; d < HD; d += kTile) s_q[d] = load1(a.q, b * a.q_batch + i * a.q_stride + (int64_t)h * HD + d, a.dtype);
        float m = -INFINITY, l = 0.f, o = 0.f;
        __syncthreads();
        for (int j0 = 0; j0 < len; j0 += kTile) {
            const int j = j0 + tid;
            int64_t off = -1;
            float s = -INFINITY;
            if (j < len) {
                if (a.table) {
                    const int page = a.by_ps.div(j);
                    const int id = a.table[(int64_t)b * a.table_stride + page];
                    if (id >= 0 && id < a.n_pages)
                        off = id * a.page_stride + (j - page * (int)a.by_ps.d) * a.pos_stride + g * a.head_stride;
                } else {
                    off = b * a.batch_stride + j * a.pos_stride + g * a.head_stride;
                }
            }
            if (off >= 0) {
                s = 0.f;
                for (int d = 0; d < HD; ++d) s = fmaf(s_q[d], load1(a.k, off + d, a.kv_dtype), s);
                s *= a.scale * ks;
            }
            s_off[tid] = off;
            float mx = s;
            for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            if (lane == 0) s_red[warp] = mx;
            __syncthreads();
            const float mn = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
            const float base = mn == -INFINITY ? 0.f : mn, keep = m == -INFINITY ? 0.f : expf(m - base);
            s_p[tid] = off >= 0 ? expf(s - base) : 0.f;
            __syncthreads();
            l *= keep;
            o *= keep;
            const int n = min(kTile, len - j0);
            for (int x = 0; x < n; ++x) {
                if (s_off[x] < 0) continue;
                l += s_p[x];
                if (tid < HD) o = fmaf(s_p[x], load1(a.v, s_off[x] + tid, a.kv_dtype), o);
            }
            m = mn;
            __syncthreads();
        }
        if (tid < HD)
            store1(a.out, b * a.o_batch + i * a.o_stride + (int64_t)h * HD + tid, a.dtype, l == 0.f ? 0.f : o * vs / l);
        if (a.lse && tid == 0) a.lse[((int64_t)b * a.Lq + i) * a.H + h] = l == 0.f ? -INFINITY : m + logf(l);
        __syncthreads();
    }
}

int check_q(const char* who, int dtype, int kv_dtype, const void* q, int64_t q_stride, const void* out,
            int64_t out_stride, int n_head, int n_kv, float scale) {
    const int b = dtype == SD_E4M3 ? 0 : dtype_bytes(dtype);
    if (!b) return op_fail(SD_ERR_INVALID_ARG, "%s: type %d is not SD_F32, SD_F16 or SD_BF16", who, dtype);
    if (dtype == SD_F32 && kv_dtype == SD_BF16)
        return op_fail(SD_ERR_UNSUPPORTED, "%s: SD_F32 queries need SD_F16 or SD_E4M3 keys and values", who);
    if (!q || !out || !aligned16(q) || !aligned16(out) || !stride16(q_stride, b) || !stride16(out_stride, b))
        return op_fail(SD_ERR_INVALID_ARG, "%s: q_dev, out_dev and their strides must be multiples of 16 bytes", who);
    if (n_head < 1 || n_head % n_kv)
        return op_fail(SD_ERR_INVALID_ARG, "%s: n_head %d is not a multiple of n_kv_head %d", who, n_head, n_kv);
    if (!(scale - scale == 0.f)) return op_fail(SD_ERR_INVALID_ARG, "%s: scale is not finite", who);
    return SD_OK;
}

int launch(const char* who, sd_attn_ws* ws, const AttendArgs& a, int hd, void* stream) {
    if (!ws) return op_fail(SD_ERR_INVALID_ARG, "%s: ws is NULL", who);
    DeviceScope scope(ws->device);
    if (scope.err != cudaSuccess) return op_fail(SD_ERR_CUDA, "%s: %s", who, cudaGetErrorString(scope.err));
    const dim3 grid((unsigned)std::min<int64_t>((int64_t)a.B * a.Lq, 65536), a.H);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = hd == 64 ? launch_k(k_attend<64>, grid, dim3(kTile), 0, st, a)
                                   : launch_k(k_attend<128>, grid, dim3(kTile), 0, st, a);
    if (e != cudaSuccess) return op_fail(SD_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return SD_OK;
}

}  // namespace
}  // namespace sd

extern "C" {

int sd_attn_ws_create(int32_t device, sd_attn_ws** out) {
    using namespace sd;
    if (!out) return op_fail(SD_ERR_INVALID_ARG, "sd_attn_ws_create: out is NULL");
    *out = nullptr;
    if (device < 0) {
        const cudaError_t e = cudaGetDevice(&device);
        if (e != cudaSuccess) return op_fail(SD_ERR_CUDA, "sd_attn_ws_create: %s", cudaGetErrorString(e));
    }
    DeviceScope scope(device);
    if (scope.err != cudaSuccess) return op_fail(SD_ERR_CUDA, "sd_attn_ws_create: %s", cudaGetErrorString(scope.err));
    sd_attn_ws* ws = new (std::nothrow) sd_attn_ws;
    if (!ws) return op_fail(SD_ERR_OOM, "sd_attn_ws_create: out of host memory");
    ws->device = device;
    *out = ws;
    return SD_OK;
}

void sd_attn_ws_destroy(sd_attn_ws* ws) { delete ws; }

int sd_attend_pages(sd_attn_ws* ws, const sd_pages* cache, const int32_t* table_dev, int32_t table_stride,
                    const int32_t* len_dev, int32_t R, int32_t dtype, const void* q_dev, int64_t q_stride,
                    int32_t n_head, float scale, void* out_dev, int64_t out_stride, float* lse_dev, void* stream) {
    using namespace sd;
    static const char* who = "sd_attend_pages";
    sd_pages c;
    if (int rc = check_pages(who, cache, &c)) return rc;
    if (!table_dev || !len_dev) return op_fail(SD_ERR_INVALID_ARG, "%s: table_dev or len_dev is NULL", who);
    if (R < 0 || table_stride < 1) return op_fail(SD_ERR_INVALID_ARG, "%s: R %d, table_stride %d", who, R, table_stride);
    if (int rc = check_q(who, dtype, c.dtype, q_dev, q_stride, out_dev, out_stride, n_head, c.n_kv_head, scale)) return rc;
    if (!ws) return op_fail(SD_ERR_INVALID_ARG, "%s: ws is NULL", who);
    if (R == 0) return SD_OK;
    AttendArgs a = {};
    a.q = q_dev; a.k = c.k_dev; a.v = c.v_dev; a.out = out_dev; a.lse = lse_dev; a.table = table_dev; a.len = len_dev;
    a.k_scale = c.k_scale_dev; a.v_scale = c.v_scale_dev; a.by_ps = FastDiv((uint32_t)c.page_size);
    a.page_stride = c.page_stride; a.head_stride = c.head_stride; a.pos_stride = c.pos_stride;
    a.q_batch = q_stride; a.q_stride = 0; a.o_batch = out_stride; a.o_stride = 0;
    a.B = R; a.Lq = 1; a.H = n_head; a.Hkv = c.n_kv_head; a.n_pages = c.n_pages; a.table_stride = table_stride;
    a.max_len = (int32_t)std::min<int64_t>((int64_t)table_stride * c.page_size, INT32_MAX);
    a.dtype = dtype; a.kv_dtype = c.dtype; a.scale = scale;
    return launch(who, ws, a, c.head_dim, stream);
}

int sd_attend_cross(sd_attn_ws* ws, const sd_states* states, int32_t dtype, const void* q_dev, int64_t q_batch,
                    int64_t q_stride, int32_t Lq, int32_t n_head, float scale, void* out_dev, int64_t out_batch,
                    int64_t out_stride, float* lse_dev, void* stream) {
    using namespace sd;
    static const char* who = "sd_attend_cross";
    if (!states) return op_fail(SD_ERR_INVALID_ARG, "%s: states is NULL", who);
    sd_states s = *states;
    if (s.dtype != SD_F16 && s.dtype != SD_BF16)
        return op_fail(SD_ERR_INVALID_ARG, "%s: states of type %d, not SD_F16 or SD_BF16", who, s.dtype);
    if (s.head_dim != 64 && s.head_dim != 128)
        return op_fail(SD_ERR_UNSUPPORTED, "%s: head_dim %d is not 64 or 128", who, s.head_dim);
    if (s.B < 0 || s.n_pos < 0 || s.n_kv_head < 1 || Lq < 0)
        return op_fail(SD_ERR_INVALID_ARG, "%s: B %d, n_pos %d, n_kv_head %d, Lq %d", who, s.B, s.n_pos, s.n_kv_head, Lq);
    if (!s.k_dev || !s.v_dev || !aligned16(s.k_dev) || !aligned16(s.v_dev))
        return op_fail(SD_ERR_INVALID_ARG, "%s: k_dev or v_dev is NULL or not 16-byte aligned", who);
    if (!s.batch_stride && !s.head_stride && !s.pos_stride) {
        s.head_stride = s.head_dim;
        s.pos_stride = (int64_t)s.n_kv_head * s.head_dim;
        s.batch_stride = s.pos_stride * s.n_pos;
    }
    if (s.batch_stride < 0 || s.head_stride < 0 || s.pos_stride < 0 || s.batch_stride % 8 || s.head_stride % 8 ||
        s.pos_stride % 8)
        return op_fail(SD_ERR_INVALID_ARG, "%s: the states' strides must be multiples of 16 bytes", who);
    if (int rc = check_q(who, dtype, s.dtype, q_dev, q_stride, out_dev, out_stride, n_head, s.n_kv_head, scale)) return rc;
    if (s.B > 1 && (!stride16(q_batch, dtype_bytes(dtype)) || !stride16(out_batch, dtype_bytes(dtype))))
        return op_fail(SD_ERR_INVALID_ARG, "%s: q_batch and out_batch must be multiples of 16 bytes", who);
    if (!ws) return op_fail(SD_ERR_INVALID_ARG, "%s: ws is NULL", who);
    if (s.B == 0 || Lq == 0) return SD_OK;
    AttendArgs a = {};
    a.q = q_dev; a.k = s.k_dev; a.v = s.v_dev; a.out = out_dev; a.lse = lse_dev; a.len = s.len_dev;
    a.batch_stride = s.batch_stride; a.head_stride = s.head_stride; a.pos_stride = s.pos_stride;
    a.q_batch = q_batch; a.q_stride = q_stride; a.o_batch = out_batch; a.o_stride = out_stride;
    a.B = s.B; a.Lq = Lq; a.H = n_head; a.Hkv = s.n_kv_head; a.max_len = s.n_pos;
    a.dtype = dtype; a.kv_dtype = s.dtype; a.scale = scale;
    return launch(who, ws, a, s.head_dim, stream);
}

}  // extern "C"
