// lm.h -- host-side pieces shared by the language-model operators: the window handle, argument
// checks, and per-device kernel setup.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/st_attn.h"

struct st_window {
    int32_t heads = 0, kv_heads = 0;
    int64_t window = 0, sinks = 0;
    bool uploaded = false;
    int device = -1;
    int32_t *d_err = nullptr;  // bit 0: a bounded wait gave up, bit 1: misaligned shared memory,
                               // bit 2: a page outside the cache
};

namespace st {

constexpr int32_t ERR_PAGE = 4;
constexpr int64_t MAX_POS = 1ll << 30;  // positions, lengths and row counts of these operators

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
inline int elem_bytes(int32_t dtype) { return dtype == ST_FP32 ? 4 : 2; }
inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Strides of a [batch, heads, rows, width] tensor: positive and a multiple of 16 bytes wherever the
// dimension is longer than 1, rows not overlapping.  Strides of dimensions of extent 1 are not read.
inline st_status_t check_strides(const st_strides_t &s, int64_t batch, int64_t heads, int64_t rows, int64_t width,
                                 int es)
{
    const int64_t ext[3] = {batch, heads, rows}, str[3] = {s.batch, s.head, s.row};
    for (int i = 0; i < 3; ++i) {
        if (ext[i] <= 1) continue;
        if (str[i] < width || str[i] > (1ll << 38)) return ST_ERR_INVALID_ARG;
        if (str[i] * es % 16 != 0) return ST_ERR_ALIGNMENT;
    }
    return ST_OK;
}

// Whether one of the outputs starts where an input or another output does: it would be overwritten
// while it is still read.  (Overlaps beyond that cannot be told from interleaved views.)
template <int NOUT, int NIN>
bool same_start(const void *const (&outs)[NOUT], const void *const (&ins)[NIN])
{
    for (int i = 0; i < NOUT; ++i) {
        for (int j = 0; j < i; ++j)
            if (outs[i] == outs[j]) return true;
        for (int j = 0; j < NIN; ++j)
            if (outs[i] == ins[j]) return true;
    }
    return false;
}

// Same layout of a [batch, heads, rows, width] tensor.
inline bool same_strides(const st_strides_t &a, const st_strides_t &b, int64_t batch, int64_t heads, int64_t rows)
{
    return (batch == 1 || a.batch == b.batch) && (heads == 1 || a.head == b.head) && (rows == 1 || a.row == b.row);
}

inline st_status_t check_window(const st_window_t *w)
{
    if (!w) return ST_ERR_INVALID_ARG;
    if (!w->uploaded) return ST_ERR_NOT_UPLOADED;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return ST_ERR_CUDA;
    return dev == w->device ? ST_OK : ST_ERR_INVALID_ARG;
}

// Raise a kernel's dynamic shared memory limit once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

}  // namespace st
