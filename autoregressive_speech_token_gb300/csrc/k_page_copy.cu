// sd_page_copy: pages copied within every layer's cache, as the copy lists of
// sd_page_fork and sd_page_compact say.
//
// Bound by memory: each byte is read and written once.  A piece is up to
// kUnits 16-byte units a thread of one page's keys or values in one layer, all loads in
// flight before the first store.  Units run along memory whichever of heads and positions is the
// outer dimension.  How many copies there are is known on the device only: resident
// blocks take the pieces in turn.
//
// Measured: 2000 pages of 262 KB moved, 1.05 GB read and written, 166 us, 0.92 of the rate of a plain copy;
// 15 partly filled pages in each of 28 layers, 41 MB (in L2), 6.8 us.
#include <algorithm>

#include "pages_dev.cuh"

namespace sd {
namespace {

constexpr int kThreads = 256, kUnits = 8, kPiece = kThreads * kUnits, kMaxCaches = 128;

struct CopyArgs {
    char *k[kMaxCaches], *v[kMaxCaches];
    const int32_t *copies, *count;
    int64_t page_bytes, head_bytes, pos_bytes;
    int32_t caches, most, n_pages, ps, heads, log_row, pieces;   // 16-byte units of a row: 1 << log_row; pieces of a whole page
    int32_t pos_outer;
};

__global__ void __launch_bounds__(kThreads) k_page_copy(const __grid_constant__ CopyArgs a) {
    pdl_trigger();
    pdl_wait();
    const int64_t n = min(max(__ldg(a.count), 0), a.most);
    const int64_t tasks = n * a.caches * 2 * a.pieces;
    for (int64_t t = blockIdx.x; t < tasks; t += gridDim.x) {
        const int64_t x = t / a.pieces;
        const int piece = (int)(t - x * a.pieces);
        const int64_t y = x >> 1, c = y / a.caches;
        const int layer = (int)(y - c * a.caches);
        const int32_t from = __ldg(a.copies + 3 * c), to = __ldg(a.copies + 3 * c + 1);
        const int32_t count = min(max(__ldg(a.copies + 3 * c + 2), 0), a.ps);
        if ((uint32_t)from >= (uint32_t)a.n_pages || (uint32_t)to >= (uint32_t)a.n_pages || from == to) continue;
        const int64_t units = ((int64_t)count * a.heads) << a.log_row;
        const int64_t u0 = (int64_t)piece * kPiece + threadIdx.x;
        if ((int64_t)piece * kPiece >= units) continue;
        char* base = (x & 1) ? a.v[layer] : a.k[layer];
        const char* src = base + from * a.page_bytes;
        char* dst = base + to * a.page_bytes;
        const uint32_t inner = a.pos_outer ? a.heads : count;
        uint4 v[kUnits];
        int64_t off[kUnits];
#pragma unroll
        for (int e = 0; e < kUnits; ++e) {
            const int64_t u = u0 + e * kThreads;
            off[e] = -1;
            if (u >= units) continue;
            const uint32_t row = (uint32_t)(u >> a.log_row), unit = (uint32_t)u & ((1u << a.log_row) - 1);
            const uint32_t outer = row / inner, in = row - outer * inner;
            off[e] = (a.pos_outer ? outer * a.pos_bytes + in * a.head_bytes : outer * a.head_bytes + in * a.pos_bytes) + unit * 16;
            v[e] = *reinterpret_cast<const uint4*>(src + off[e]);
        }
#pragma unroll
        for (int e = 0; e < kUnits; ++e)
            if (off[e] >= 0) *reinterpret_cast<uint4*>(dst + off[e]) = v[e];
    }
}

}  // namespace
}  // namespace sd

extern "C" int sd_page_copy(const sd_pages* caches, int32_t n_caches, const int32_t* copy_dev, const int32_t* count_dev,
                            int32_t max_copies, void* stream) {
    using namespace sd;
    static const char* who = "sd_page_copy";
    if (n_caches == 0 || max_copies == 0) return SD_OK;
    if (n_caches < 0 || n_caches > kMaxCaches || max_copies < 0)
        return op_fail(SD_ERR_INVALID_ARG, "%s: n_caches %d (up to %d), max_copies %d", who, n_caches, kMaxCaches, max_copies);
    if (!caches || !copy_dev || !count_dev) return op_fail(SD_ERR_INVALID_ARG, "%s: NULL argument", who);
    CopyArgs a = {};
    sd_pages c0 = {};
    for (int i = 0; i < n_caches; ++i) {
        sd_pages c;
        if (int rc = check_pages(who, caches + i, &c)) return rc;
        if (i == 0) c0 = c;
        if (c.dtype != c0.dtype || c.n_pages != c0.n_pages || c.page_size != c0.page_size || c.n_kv_head != c0.n_kv_head ||
            c.head_dim != c0.head_dim || c.page_stride != c0.page_stride || c.head_stride != c0.head_stride ||
            c.pos_stride != c0.pos_stride)
            return op_fail(SD_ERR_INVALID_ARG, "%s: cache %d has another type, shape or strides than the first", who, i);
        a.k[i] = static_cast<char*>(c.k_dev);
        a.v[i] = static_cast<char*>(c.v_dev);
    }
    const int b = dtype_bytes(c0.dtype);
    a.copies = copy_dev; a.count = count_dev; a.caches = n_caches; a.most = max_copies;
    a.page_bytes = c0.page_stride * b; a.head_bytes = c0.head_stride * b; a.pos_bytes = c0.pos_stride * b;
    a.n_pages = c0.n_pages; a.ps = c0.page_size; a.heads = c0.n_kv_head;
    while ((16 << a.log_row) < c0.head_dim * b) ++a.log_row;
    a.pos_outer = c0.pos_stride > c0.head_stride;
    const int64_t units = ((int64_t)a.ps * a.heads) << a.log_row, pieces = (units + kPiece - 1) / kPiece;
    if (pieces > INT32_MAX || ((int64_t)a.ps * a.heads) > INT32_MAX)
        return op_fail(SD_ERR_UNSUPPORTED, "%s: pages of %d positions of %d heads", who, a.ps, a.heads);
    a.pieces = (int32_t)pieces;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t tasks = std::min<int64_t>((int64_t)max_copies * n_caches * 2, (int64_t)1 << 30) * pieces;
    if (e == cudaSuccess)
        e = launch_k(k_page_copy, dim3((unsigned)std::min<int64_t>(tasks, (int64_t)sms * 6)), dim3(kThreads), 0,
                     reinterpret_cast<cudaStream_t>(stream), a);
    if (e != cudaSuccess) return op_fail(SD_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return SD_OK;
}
