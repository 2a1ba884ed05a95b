// sd_attend_pages and sd_attend_cross: arguments, workspace, and the choice of kernel.
#include <algorithm>
#include <cstdlib>
#include <new>

#include "attend_dev.cuh"

namespace sd {
namespace {

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

// Which kernel takes Lq queries of G heads to a kv head, where queries, keys and values have one 16-bit type: the
// tensor-core kernel (true) or the split one.  Per kv head both walk the row's states once for each of their pieces,
// the split kernel for every 8 (query, head) rows, the tensor-core kernel for every pair of tiles, a tile being up to
// 128 queries of ONE head.  A walk of a pair takes as long as 3 of the split kernel's for heads of 64, 2 for heads of
// 128.  GPU time in us, split / tensor cores, over 16 rows of 1500 states, bf16:
//   heads of 64    64 to 1: 1 query 12 / 65, 8: 47 / 65    64 to 8: 8: 47 / 65, 12: 65 / 65, 16: 87 / 65
//                  16 to 8: 12: 24.0 / 23.6, 16: 29 / 24   16 to 16: 16: 29 / 32, 24: 38 / 32
//   heads of 128   64 to 1: 1: 17 / 74, 6: 62 / 74, 8: 79 / 74    32 to 8: 6: 38 / 41, 8: 47 / 41
//                  16 to 8: 12: 38 / 27
// Over bf16 the split kernel's probabilities have 16 bits, the other's 8: up to 16 rows to a kv head they keep them,
// though 16 queries of 16 heads of 128 take 68 us there and 41 on tiles.  (fp16 probabilities have 11 in both.)
bool on_tiles(int Lq, int G, int hd, bool bf) {
    const int64_t rows = (int64_t)Lq * G, units = (rows + kSplitRows - 1) / kSplitRows;
    const int64_t pairs = ((int64_t)G * (((int64_t)Lq + 127) / 128) + 1) / 2;
    return units >= (hd == 64 ? 3 : 2) * pairs && (!bf || rows > 2 * kSplitRows);
}

size_t counters(int sms) { return (size_t)sms * kSplitRows / 2; }

int launch(const char* who, sd_attn_ws* ws, AttendArgs& a, int hd, void* stream) {
    DeviceScope scope(ws->device);
    if (scope.err != cudaSuccess) return op_fail(SD_ERR_CUDA, "%s: %s", who, cudaGetErrorString(scope.err));
    if (*static_cast<volatile int*>(ws->err))
        return op_fail(SD_ERR_TIMEOUT, "%s: a wait of an earlier call on this workspace expired", who);
    a.part = ws->part;
    a.cnt = ws->cnt;
    a.err = ws->err;
    a.dead = ws->cnt + counters(ws->sms);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (ws->test_stall > 0) {
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(st, &cs) == cudaSuccess && cs == cudaStreamCaptureStatusNone) {
            a.stall = ws->test_stall;
            ws->test_stall = 0;
        }
    }
    cudaError_t e = cudaSuccess;
    bool taken = false;
    if (!a.table && a.dtype == a.kv_dtype && a.scale > 0.f && a.max_len > 0 && on_tiles(a.Lq, a.H / a.Hkv, hd, a.dtype == SD_BF16))
        e = launch_attend_tc(a, hd, ws->sms, st, &taken);
    if (!taken) e = launch_attend_split(a, hd, ws->sms, st);
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
    cudaError_t e = cudaDeviceGetAttribute(&ws->sms, cudaDevAttrMultiProcessorCount, device);
    const size_t blocks = (size_t)ws->sms;
    if (e == cudaSuccess) e = cudaMalloc(&ws->part, blocks * kTcRecord * sizeof(float));
    const size_t words = counters(ws->sms) + 1;
    if (e == cudaSuccess) e = cudaMalloc(&ws->cnt, words * sizeof(int));
    // on the legacy stream, and waited for: the first call may be on any stream
    if (e == cudaSuccess) e = cudaMemset(ws->cnt, 0, words * sizeof(int));
    if (e == cudaSuccess) e = cudaStreamSynchronize(0);
    if (e == cudaSuccess) e = cudaHostAlloc(&ws->err, sizeof(int), cudaHostAllocDefault);
    if (e == cudaSuccess) *ws->err = 0;
    if (const char* ts = getenv("SD_TEST_STALL_US")) {
        int khz = 0;
        cudaDeviceGetAttribute(&khz, cudaDevAttrClockRate, device);
        ws->test_stall = (long long)(khz > 0 ? khz : 2000000) * std::max(1, atoi(ts)) / 1000;
    }
    if (e == cudaSuccess) e = prepare_attend_split();
    if (e == cudaSuccess) e = prepare_attend_tc();
    if (e != cudaSuccess) {
        sd_attn_ws_destroy(ws);
        return op_fail(e == cudaErrorMemoryAllocation ? SD_ERR_OOM : SD_ERR_CUDA, "sd_attn_ws_create: %s",
                       cudaGetErrorString(e));
    }
    *out = ws;
    return SD_OK;
}

void sd_attn_ws_destroy(sd_attn_ws* ws) {
    if (!ws) return;
    sd::DeviceScope scope(ws->device);
    cudaFree(ws->part);
    cudaFree(ws->cnt);
    cudaFreeHost(ws->err);
    delete ws;
}

int sd_attend_pages(sd_attn_ws* ws, const sd_pages* cache, const int32_t* table_dev, int32_t table_stride,
                    const int32_t* len_dev, int32_t R, int32_t dtype, const void* q_dev, int64_t q_stride,
                    int32_t n_head, float scale, void* out_dev, int64_t out_stride, float* lse_dev, void* stream) {
    using namespace sd;
    static const char* who = "sd_attend_pages";
    if (R == 0) return SD_OK;
    sd_pages c;
    if (int rc = check_pages(who, cache, &c)) return rc;
    if (R < 0 || table_stride < 1) return op_fail(SD_ERR_INVALID_ARG, "%s: R %d, table_stride %d", who, R, table_stride);
    if (!table_dev || !len_dev) return op_fail(SD_ERR_INVALID_ARG, "%s: table_dev or len_dev is NULL", who);
    if (int rc = check_q(who, dtype, c.dtype, q_dev, q_stride, out_dev, out_stride, n_head, c.n_kv_head, scale)) return rc;
    if (c.dtype == SD_E4M3 && c.head_dim == 64 && c.page_size % 2)
        return op_fail(SD_ERR_UNSUPPORTED, "%s: pages of an odd number of 64-byte rows", who);
    if (!ws) return op_fail(SD_ERR_INVALID_ARG, "%s: ws is NULL", who);
    AttendArgs a = {};
    a.q = q_dev; a.k = c.k_dev; a.v = c.v_dev; a.out = out_dev; a.lse = lse_dev; a.table = table_dev; a.len = len_dev;
    a.k_scale = c.k_scale_dev; a.v_scale = c.v_scale_dev; a.by_ps = FastDiv((uint32_t)c.page_size);
    a.page_stride = c.page_stride; a.head_stride = c.head_stride; a.pos_stride = c.pos_stride;
    a.q_batch = q_stride; a.q_stride = 0; a.o_batch = out_stride; a.o_stride = 0;
    a.B = R; a.Lq = 1; a.H = n_head; a.Hkv = c.n_kv_head; a.n_pages = c.n_pages; a.table_stride = table_stride;
    a.max_len = (int32_t)std::min<int64_t>((int64_t)table_stride * c.page_size, kMaxPositions);
    a.dtype = dtype; a.kv_dtype = c.dtype; a.scale = scale;
    return launch(who, ws, a, c.head_dim, stream);
}

int sd_attend_cross(sd_attn_ws* ws, const sd_states* states, int32_t dtype, const void* q_dev, int64_t q_batch,
                    int64_t q_stride, int32_t Lq, int32_t n_head, float scale, void* out_dev, int64_t out_batch,
                    int64_t out_stride, float* lse_dev, void* stream) {
    using namespace sd;
    static const char* who = "sd_attend_cross";
    if (Lq == 0) return SD_OK;
    if (!states) return op_fail(SD_ERR_INVALID_ARG, "%s: states is NULL", who);
    sd_states s = *states;
    if (s.B == 0) return SD_OK;
    if (s.dtype != SD_F16 && s.dtype != SD_BF16)
        return op_fail(SD_ERR_INVALID_ARG, "%s: states of type %d, not SD_F16 or SD_BF16", who, s.dtype);
    if (s.head_dim != 64 && s.head_dim != 128)
        return op_fail(SD_ERR_UNSUPPORTED, "%s: head_dim %d is not 64 or 128", who, s.head_dim);
    if (s.B < 0 || s.n_pos < 0 || s.n_kv_head < 1 || Lq < 0)
        return op_fail(SD_ERR_INVALID_ARG, "%s: B %d, n_pos %d, n_kv_head %d, Lq %d", who, s.B, s.n_pos, s.n_kv_head, Lq);
    if (s.n_pos == 0) {                                            // nothing is read: any legal address and strides
        s.k_dev = s.v_dev = q_dev;
        s.head_stride = s.pos_stride = s.batch_stride = s.head_dim;
    }
    if (!s.k_dev || !s.v_dev || !aligned16(s.k_dev) || !aligned16(s.v_dev))
        return op_fail(SD_ERR_INVALID_ARG, "%s: k_dev or v_dev is NULL or not 16-byte aligned", who);
    if (!s.batch_stride && !s.head_stride && !s.pos_stride) {
        s.head_stride = s.head_dim;
        s.pos_stride = (int64_t)s.n_kv_head * s.head_dim;
        s.batch_stride = s.pos_stride * s.n_pos;
    }
    if (!tma_stride(s.batch_stride, 2, s.B) || !tma_stride(s.head_stride, 2, s.n_kv_head) ||
        !tma_stride(s.pos_stride, 2, s.n_pos))
        return op_fail(SD_ERR_INVALID_ARG, "%s: the states' strides must be positive multiples of 16 bytes", who);
    if (int rc = check_q(who, dtype, s.dtype, q_dev, q_stride, out_dev, out_stride, n_head, s.n_kv_head, scale)) return rc;
    if (s.B > 1 && (!stride16(q_batch, dtype_bytes(dtype)) || !stride16(out_batch, dtype_bytes(dtype))))
        return op_fail(SD_ERR_INVALID_ARG, "%s: q_batch and out_batch must be multiples of 16 bytes", who);
    if (!ws) return op_fail(SD_ERR_INVALID_ARG, "%s: ws is NULL", who);
    AttendArgs a = {};
    a.q = q_dev; a.k = s.k_dev; a.v = s.v_dev; a.out = out_dev; a.lse = lse_dev; a.len = s.len_dev;
    a.batch_stride = s.batch_stride; a.head_stride = s.head_stride; a.pos_stride = s.pos_stride;
    a.q_batch = q_batch; a.q_stride = q_stride; a.o_batch = out_batch; a.o_stride = out_stride;
    a.B = s.B; a.Lq = Lq; a.H = n_head; a.Hkv = s.n_kv_head; a.max_len = std::min(s.n_pos, kMaxPositions);
    a.dtype = dtype; a.kv_dtype = s.dtype; a.scale = scale;
    return launch(who, ws, a, s.head_dim, stream);
}

}  // extern "C"
