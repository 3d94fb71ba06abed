// handle.cuh -- what the library's translation units share: the handle, the
// last CUDA error of a thread, and the guard of the current device.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstdio>

#include "../../include/specv.h"

struct specv_ctx {
    int device = 0;
    int sm_count = 0;
    int max_batch = 0;
    int max_k = 0;
    int64_t vocab = 0;
    std::atomic<int64_t> launches{0};
    // most clusters of each size (1..16) that can be resident at once, per
    // logits type (index 0: fp32, 1: bf16); 0 if that size cannot launch
    int max_clusters[2][17] = {};
    // device staging for specv_verify_sample_host
    void* stage = nullptr;
    size_t stage_bytes = 0;
    // one-shot test hook: the next cluster-kernel launch withholds one
    // pass-1 stage of CTA 0 and waits at most `test_polls` polls
    int test_withhold = -1;
    uint32_t test_polls = 0;
};

inline thread_local char g_last_error[256] = "";

inline specv_status cuda_fail(cudaError_t e, const char* what) {
    snprintf(g_last_error, sizeof g_last_error, "%s: %s", what, cudaGetErrorString(e));
    return SPECV_ERR_CUDA;
}

#define SPECV_CUDA(call)                                         \
    do {                                                         \
        cudaError_t e_ = (call);                                 \
        if (e_ != cudaSuccess) return cuda_fail(e_, #call);      \
    } while (0)

namespace {

struct DeviceGuard {
    int prev = -1;
    bool ok = false;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) == cudaSuccess) ok = (prev == dev) || cudaSetDevice(dev) == cudaSuccess;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

}  // namespace
