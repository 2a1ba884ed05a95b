// Shared by the paged-cache and cross-attention entry points: argument checks,
// element types, and division by a page size that is known at launch.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdarg>
#include <cstdio>

#include "../../include/sd_ops.h"
#include "sd_internal.cuh"

namespace sd {

// Message for sd_last_error(NULL), and the code to return.
inline int op_fail(int code, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return code;
}

inline int dtype_bytes(int dt) {
    return dt == SD_F32 ? 4 : dt == SD_F16 || dt == SD_BF16 ? 2 : dt == SD_E4M3 ? 1 : 0;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool stride16(int64_t elements, int bytes) { return elements % (16 / bytes) == 0; }
// A stride of a dimension of `count` elements that TMA can hold (not used where there is one element)
inline bool tma_stride(int64_t elements, int bytes, int64_t count) {
    return count <= 1 || (stride16(elements, bytes) && elements > 0 && elements < ((int64_t)1 << 40) / bytes);
}

// Makes `device` current for one call and puts the caller's back.
struct DeviceScope {
    int prev = -1;
    cudaError_t err = cudaSuccess;
    explicit DeviceScope(int device) {
        int cur = -1;
        err = cudaGetDevice(&cur);
        if (err == cudaSuccess && cur != device) {
            err = cudaSetDevice(device);
            if (err == cudaSuccess) prev = cur;
        }
    }
    ~DeviceScope() {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

// x / d for 0 <= x < 2^31 by one high product: m = floor(2^(31+s) / d) + 1 with
// 2^(s-1) < d <= 2^s has an error below 2^-31 * d / 2^s of one, so the floor is exact.
struct FastDiv {
    uint32_t d = 1, m = 0, s = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div) {
        while ((1ull << s) < div) ++s;
        m = div == 1 ? 0 : (uint32_t)(((uint64_t)1 << (31 + s)) / div + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t x) const {
        return d == 1 ? x : (uint32_t)(((uint64_t)x * m) >> 31) >> s;
    }
};

// The strides and the shape of a cache, checked.
inline int check_pages(const char* who, const sd_pages* c, sd_pages* out) {
    if (!c) return op_fail(SD_ERR_INVALID_ARG, "%s: cache is NULL", who);
    *out = *c;
    const int b = c->dtype == SD_F32 ? 0 : dtype_bytes(c->dtype);
    if (!b) return op_fail(SD_ERR_INVALID_ARG, "%s: cache type %d is not SD_F16, SD_BF16 or SD_E4M3", who, c->dtype);
    if (c->head_dim != 64 && c->head_dim != 128)
        return op_fail(SD_ERR_UNSUPPORTED, "%s: head_dim %d is not 64 or 128", who, c->head_dim);
    if (c->n_pages < 1 || c->n_kv_head < 1 || c->page_size < 1 || c->page_size > 65536 ||
        (int64_t)c->n_pages * c->page_size > INT32_MAX)
        return op_fail(SD_ERR_INVALID_ARG, "%s: %d pages of %d positions, %d kv heads", who, c->n_pages, c->page_size,
                       c->n_kv_head);
    if (!c->k_dev || !c->v_dev || !aligned16(c->k_dev) || !aligned16(c->v_dev))
        return op_fail(SD_ERR_INVALID_ARG, "%s: k_dev or v_dev is NULL or not 16-byte aligned", who);
    if (c->dtype != SD_E4M3 && (c->k_scale_dev || c->v_scale_dev))
        return op_fail(SD_ERR_INVALID_ARG, "%s: scales belong to an SD_E4M3 cache", who);
    if (!c->page_stride && !c->head_stride && !c->pos_stride) {
        out->pos_stride = c->head_dim;
        out->head_stride = (int64_t)c->page_size * c->head_dim;
        out->page_stride = out->head_stride * c->n_kv_head;
    }
    if (!tma_stride(out->page_stride, b, c->n_pages) || !tma_stride(out->head_stride, b, c->n_kv_head) ||
        !tma_stride(out->pos_stride, b, c->page_size))
        return op_fail(SD_ERR_INVALID_ARG, "%s: cache strides must be positive multiples of 16 bytes", who);
    return SD_OK;
}

}  // namespace sd
