// wsm_ops.cuh -- shared by the decode-step operators around the GEMMs (paged cache and attention, expert
// products, token log probabilities): host-side error and launch helpers, element types, and the status
// block their kernels record device-side errors in.  Not part of the public C ABI.
#pragma once

#include "wsm_internal.cuh"
#include "../../include/wsm.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdarg>
#include <cstdio>

namespace wsm {

void set_last_error_message(const char *msg);   // wsm_api.cu: what wsm_last_error() returns
unsigned long long take_launch_stall();         // wsm_api.cu: wsm_debug_stall's limit for the next launch, 0 = none
wsm_status device_sms(int *dev, int *sms);      // wsm_api.cu: the current device, checked to be an sm_100 part
wsm_status encode_tiled(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims,
                        const cuuint64_t *strides, const cuuint32_t *box);  // wsm_api.cu: 128-byte swizzle

// Device addresses, on the current device, of what wsm_operator_status (wsm_opstatus.cu) takes: an error word of
// each operator family for values out of range (record_op_error), and the block of the expert products' waits.
wsm_status cache_error_ptr(void **p);     // wsm_cache.cu
wsm_status experts_error_ptr(void **p);   // wsm_experts.cu
wsm_status experts_status_ptr(void **p);  // wsm_experts.cu
wsm_status logprobs_error_ptr(void **p);  // wsm_logprobs.cu

// The block of an operator's waits on one device, in the library's device image: [0] the code of the first one that
// ran out since the host last read it (sticky), [2] the CTA, [3] the site; [5] never written (what a stalled launch
// waits on).  The same words as the GEMMs' status block (wsm_internal.cuh); [4] is not used: no operator's launch
// consults another's errors.
constexpr int kOpStatusInts = 16;

// Sites of the operators' errors.
enum : int { kSitePage = 32, kSiteLength = 33, kSiteSlot = 34, kSiteOffsets = 35, kSiteToken = 36 };

static inline wsm_status op_fail(wsm_status code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error_message(buf);
    return code;
}

#define WSM_OP_CUDA(call)                                                                                       \
    do {                                                                                                        \
        cudaError_t e_ = (call);                                                                                \
        if (e_ != cudaSuccess)                                                                                  \
            return op_fail(WSM_ERR_CUDA, "%s: %s (%s)", #call, cudaGetErrorName(e_), cudaGetErrorString(e_));   \
    } while (0)

// One launch with programmatic dependent launch: every operator kernel waits for the kernel before it
// (griddepcontrol.wait) before it touches global memory and lets the next one launch only after that, as
// the GEMMs do, so stream order holds through any mix of them.  A kernel that is an operator's last to use the
// caller's scratch lets the next one launch only when it is through with it: independent calls do not wait, and
// the caller may have given the scratch to one.
template <typename P>
static inline wsm_status op_launch(void (*fn)(P), dim3 grid, int threads, size_t smem, cudaStream_t stream, const P &p,
                                   int cluster = 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    int na = 1;
    if (cluster > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = (unsigned)cluster;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    WSM_OP_CUDA(cudaLaunchKernelEx(&cfg, fn, p));
    return WSM_OK;
}

// Dynamic shared memory above the default 48 KB is opted into once per kernel and device.  The calls are
// idempotent, so two threads that both find the flag clear do no harm.
constexpr int kMaxOpDevices = 64;
template <typename P>
static inline wsm_status op_allow_smem(void (*fn)(P), int bytes, int dev, volatile bool *done) {
    if (dev < 0 || dev >= kMaxOpDevices) return op_fail(WSM_ERR_UNSUPPORTED, "device index %d is too large", dev);
    if (done[dev]) return WSM_OK;
    WSM_OP_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    done[dev] = true;
    return WSM_OK;
}

static inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

#if defined(__CUDACC__)

// Record a value out of range: the first of the family since the host last took one.  The site and which (the
// sequence, row or expert) in one word: who takes it gets both or neither.
__device__ __forceinline__ void record_op_error(unsigned long long *word, int which, int site) {
    atomicCAS(word, 0ull, (unsigned long long)site << 32 | (uint32_t)which);
}

// 2^y: the hardware approximation, relative error 2^-22, subnormal results 0
__device__ __forceinline__ float ex2(float y) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    return e;
}

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two values packed into one 32-bit register, the first in the low half.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t v);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<__half2 *>(&v));
}

#endif  // __CUDACC__

}  // namespace wsm
