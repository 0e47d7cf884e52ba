// wsm_opstatus.cu -- wsm_operator_status: what the decode-step operators recorded on a device, taken on the device.
#include "wsm_ops.cuh"

#include <mutex>

namespace wsm {

namespace {

// The error words of the families, in the order in which they are reported.
constexpr int kFamilies = 3;
struct ErrorWords {
    int *waits;                                 // the expert products' device-side waits
    unsigned long long *error[kFamilies];       // values out of range: cache and attention, experts, log probabilities
};
struct Taken {
    int code, family, which, cta, site;
};
__device__ Taken g_taken;

// Takes one error and leaves the others.  Exchanges on the words themselves: what a kernel on another stream records
// meanwhile is either taken or still there for the next query.
__global__ void take_error_kernel(const __grid_constant__ ErrorWords w) {
    pdl_wait();
    Taken t = {};
    // a wait that ran out first: it left outputs unfinished
    if (*(volatile int *)w.waits != 0) {
        t.cta = ((volatile int *)w.waits)[2];
        t.site = ((volatile int *)w.waits)[3];
        t.code = atomicExch(w.waits, 0);
        t.family = 1;
    }
    for (int f = 0; f < kFamilies && t.code == 0; ++f) {
        const unsigned long long e = atomicExch(w.error[f], 0ull);
        if (e == 0ull) continue;
        t.code = WSM_ERR_INVALID;
        t.family = f;
        t.which = (int)(uint32_t)e;
        t.site = (int)(e >> 32);
    }
    g_taken = t;
}

}  // namespace

}  // namespace wsm

using namespace wsm;

extern "C" wsm_status wsm_operator_status(wsm_stream_t stream_, int *code) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (code) *code = 0;
    WSM_OP_CUDA(cudaStreamSynchronize(stream));
    Taken t = {};
    {
        static std::mutex mu;                   // one query at a time: they share g_taken
        std::lock_guard<std::mutex> lk(mu);
        ErrorWords w;
        void *p = nullptr;
        wsm_status st;
        if ((st = experts_status_ptr(&p)) != WSM_OK) return st;
        w.waits = static_cast<int *>(p);
        static wsm_status (*const words[kFamilies])(void **) = {cache_error_ptr, experts_error_ptr, logprobs_error_ptr};
        for (int f = 0; f < kFamilies; ++f) {
            if ((st = words[f](&p)) != WSM_OK) return st;
            w.error[f] = static_cast<unsigned long long *>(p);
        }
        if ((st = op_launch(&take_error_kernel, dim3(1), 1, 0, stream, w)) != WSM_OK) return st;
        WSM_OP_CUDA(cudaGetSymbolAddress(&p, g_taken));
        WSM_OP_CUDA(cudaMemcpyAsync(&t, p, sizeof t, cudaMemcpyDeviceToHost, stream));
        WSM_OP_CUDA(cudaStreamSynchronize(stream));
    }
    if (t.code == 0) return WSM_OK;
    if (code) *code = t.code;
    static const char *const names[kFamilies] = {"the paged cache or its attention", "the expert products", "the log probabilities"};
    if (t.code == WSM_ERR_TIMEOUT)
        return op_fail(WSM_ERR_TIMEOUT, "device-side wait ran out in %s (cta %d, site %d)", names[t.family], t.cta, t.site);
    return op_fail(WSM_ERR_INVALID, "an index out of range in %s (row, sequence or expert %d, site %d)", names[t.family], t.which,
                   t.site);
}
