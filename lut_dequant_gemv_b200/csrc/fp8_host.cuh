// fp8_host.cuh -- host helpers of the block-scaled 8-bit entry points: error
// reporting, the device's sizes, tensor maps, launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>

#include "../../include/sqz.h"

void sqz_internal_set_last_error(const char* msg);

namespace sqz {
namespace f8 {

inline sqz_status host_fail(sqz_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    sqz_internal_set_last_error(buf);
    return st;
}

inline sqz_status host_cuda_fail(cudaError_t e, const char* what) {
    (void)cudaGetLastError();
    return host_fail(e == cudaErrorMemoryAllocation ? SQZ_ERR_OOM : SQZ_ERR_CUDA, "%s: %s (%s)", what,
                     cudaGetErrorName(e), cudaGetErrorString(e));
}

#define SQZ_F8_TRY(expr, what)                                             \
    do {                                                                   \
        const cudaError_t e_ = (expr);                                     \
        if (e_ != cudaSuccess) return sqz::f8::host_cuda_fail(e_, (what)); \
    } while (0)

// SM count and opt-in shared memory of the current device.  Asked once per
// device (the values never change; the answer is stored before the mark, so
// concurrent first calls only ask twice).
struct DeviceSizes {
    int device = 0, sms = 0, smem = 0;
};
inline sqz_status device_sizes(DeviceSizes* out) {
    constexpr int kMax = 64;
    static std::atomic<int> sms[kMax], smem[kMax];
    SQZ_F8_TRY(cudaGetDevice(&out->device), "cudaGetDevice");
    const int d = out->device;
    const bool keep = d >= 0 && d < kMax;
    if (keep && (out->smem = smem[d].load(std::memory_order_acquire)) > 0) {
        out->sms = sms[d].load(std::memory_order_relaxed);
        return SQZ_OK;
    }
    SQZ_F8_TRY(cudaDeviceGetAttribute(&out->sms, cudaDevAttrMultiProcessorCount, d), "SM count");
    SQZ_F8_TRY(cudaDeviceGetAttribute(&out->smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, d), "shared memory size");
    if (keep) {
        sms[d].store(out->sms, std::memory_order_relaxed);
        smem[d].store(out->smem, std::memory_order_release);
    }
    return SQZ_OK;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (looked up once; the library does not link
// against the driver).
inline sqz_status encoder(EncodeTiled* out) {
    static std::atomic<EncodeTiled> known{nullptr};
    *out = known.load(std::memory_order_acquire);
    if (*out) return SQZ_OK;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    SQZ_F8_TRY(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found),
               "cuTensorMapEncodeTiled lookup");
    if (!fn || found != cudaDriverEntryPointSuccess)
        return host_fail(SQZ_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
    *out = reinterpret_cast<EncodeTiled>(fn);
    known.store(*out, std::memory_order_release);
    return SQZ_OK;
}

// A map of `depth` byte matrices [rows][cols] (row pitch `ld`, matrix pitch
// `plane`, both multiples of 16 bytes), read as tiles of 128 columns x
// `box_rows` rows with the 128-byte swizzle; zeros past the edges.
inline sqz_status tile_map(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_rows,
                           int64_t depth = 0, int64_t plane = 0) {
    EncodeTiled enc;
    const sqz_status st = encoder(&enc);
    if (st != SQZ_OK) return st;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)(depth ? depth : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)plane};
    const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1}, ones[3] = {1, 1, 1};
    const CUresult r =
        enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, depth ? 3 : 2, const_cast<void*>(base), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return host_fail(SQZ_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return SQZ_OK;
}

// Raise a kernel's dynamic shared memory limit, once per device.
template <class Kernel>
sqz_status allow_smem(Kernel kernel, const DeviceSizes& d, std::atomic<uint64_t>* done) {
    const uint64_t bit = d.device < 64 ? 1ull << d.device : 0;
    if (bit && (done->load(std::memory_order_acquire) & bit)) return SQZ_OK;
    cudaFuncAttributes a;
    SQZ_F8_TRY(cudaFuncGetAttributes(&a, kernel), "cudaFuncGetAttributes");
    SQZ_F8_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    d.smem - (int)a.sharedSizeBytes),
               "cudaFuncSetAttribute");
    done->fetch_or(bit, std::memory_order_release);
    return SQZ_OK;
}

}  // namespace f8
}  // namespace sqz
