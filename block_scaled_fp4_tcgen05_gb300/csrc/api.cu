// api.cu -- library-wide entry points of libqfp4: version, status text,
// device check and the device status poll.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>
#include <mutex>
#include <set>
#include <thread>
#include <utility>

#include "qfp4_common.cuh"
#include "qfp4_gemm_fp8.cuh"
#include "qfp4_gemm_internal.cuh"

namespace qfp4 {

int ensure_thread_context()
{
    // The runtime makes the primary context current on a host thread only
    // when that thread makes certain runtime calls; a driver-API call (the
    // tensor-map encode) from a thread that has made none fails with
    // CUDA_ERROR_INVALID_CONTEXT.  cudaSetDevice binds the current device's
    // primary context to the calling thread; done once per thread and device.
    thread_local int bound = -1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QFP4_ERR_CUDA;
    if (dev != bound) {
        if (cudaSetDevice(dev) != cudaSuccess) return QFP4_ERR_CUDA;
        bound = dev;
    }
    return QFP4_OK;
}

int ensure_smem_attr(const void *kern, int bytes)
{
    static std::mutex mu;
    static std::set<std::pair<const void *, int>> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QFP4_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count({kern, dev})) return QFP4_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return QFP4_ERR_CUDA;
    done.insert({kern, dev});
    return QFP4_OK;
}

namespace {

// The status poll: one launch takes every kernel's word and leaves zero (in one
// atomic step: a word set once is reported once, whichever poll meets it), and
// one copy brings the result back: 19 us instead of 142 with a copy and a wait to
// read and as much to clear each word.
constexpr int kWords = 8;
constexpr int (*kWordOf[kWords])(uint32_t **) = {
    status_word_quant,       status_word_gemm,     status_word_gemm_pair,      status_word_gemm_decode,
    status_word_gemm_sparse, status_word_gemm_fp8, status_word_gemm_fp8_small, status_word_fp8_quant};

struct StatusWords {
    uint32_t *word[kWords];
};

constexpr int kPollSlots = 32;
__device__ uint32_t g_poll_results[kPollSlots];

__global__ void gather_status_kernel(const StatusWords w, uint32_t *result)
{
    const int i = threadIdx.x;
    uint32_t v = 0;
#pragma unroll
    for (int k = 0; k < kWords; ++k)
        if (i == k) v = atomicExch(w.word[k], 0u);
    v = __reduce_or_sync(0xffffffffu, v);
    if (i == 0) *result = v;
}

// Where a poll's result waits to be copied: one of its own for each poll under
// way (another thread's would overwrite it).
struct PollSlot {
    int index = 0;

    PollSlot()
    {
        while (taken()[index].exchange(true, std::memory_order_acquire)) {
            if (++index == kPollSlots) {
                index = 0;
                std::this_thread::yield();
            }
        }
    }
    ~PollSlot() { taken()[index].store(false, std::memory_order_release); }

    static std::atomic<bool> *taken()
    {
        static std::atomic<bool> t[kPollSlots];
        return t;
    }
};

}  // namespace
}  // namespace qfp4

extern "C" int qfp4_version(void) { return 100; }   // 0.1.0

extern "C" const char *qfp4_status_string(int status)
{
    switch (status) {
    case QFP4_OK: return "ok";
    case QFP4_ERR_INVALID_ARG: return "invalid argument";
    case QFP4_ERR_UNSUPPORTED: return "unsupported shape or option";
    case QFP4_ERR_MISALIGNED: return "pointer not aligned as required";
    case QFP4_ERR_CUDA: return "CUDA call failed";
    case QFP4_ERR_TIMEOUT: return "device-side bounded wait ran out";
    case QFP4_ERR_ARCH: return "current device is not an sm_103 GPU";
    case QFP4_ERR_WORKSPACE: return "workspace missing or too small";
    default: return "unknown status";
    }
}

extern "C" int qfp4_device_check(void)
{
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QFP4_ERR_CUDA;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return QFP4_ERR_CUDA;
    return (major == 10 && minor == 3) ? QFP4_OK : QFP4_ERR_ARCH;
}

extern "C" int qfp4_poll_device_status(void *stream)
{
    using namespace qfp4;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    StatusWords words;
    int rc = QFP4_OK;
    for (int i = 0; i < kWords && rc == QFP4_OK; ++i) rc = kWordOf[i](&words.word[i]);
    uint32_t *results = nullptr;
    if (rc == QFP4_OK) rc = status_word(g_poll_results, &results);
    if (rc != QFP4_OK) return rc;
    PollSlot slot;
    // without programmatic launch: it starts once all earlier work on the stream is complete
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(32);
    cfg.stream = s;
    uint32_t all = 0;
    if (cudaLaunchKernelEx(&cfg, gather_status_kernel, words, results + slot.index) != cudaSuccess ||
        cudaMemcpyAsync(&all, results + slot.index, sizeof(all), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return QFP4_ERR_CUDA;
    if (all & kStatusTimeout) return QFP4_ERR_TIMEOUT;
    if (all & (kStatusBadGroup | kStatusBadSparsity)) return QFP4_ERR_INVALID_ARG;
    return QFP4_OK;
}
