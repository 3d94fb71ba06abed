// cache_host.cuh -- host side that all calls on the paged KV cache share:
// argument checks and launches.
#pragma once
#include "handle.cuh"
#include "kv_cache.cuh"

using namespace specv;

namespace {


bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The cache of a call as the kernels see it; false if a size, pointer or
// alignment is outside what specv_kv_cache allows.
bool make_view(const specv_ctx* h, const specv_kv_cache* c, int batch, KvView& view) {
    if (!h || !c || batch < 0 || batch > h->max_batch) return false;
    if (c->dtype != SPECV_F32 && c->dtype != SPECV_BF16) return false;
    if (c->kv_heads < 1 || c->kv_heads > 65536 || c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16)
        return false;
    if (c->block_size < 1 || c->block_size > 65536 || c->max_blocks < 0 || c->blocks < 0 || c->blocks > INT32_MAX)
        return false;
    const int64_t inner = static_cast<int64_t>(c->kv_heads) * c->block_size * c->head_dim;
    const int64_t vec = c->dtype == SPECV_BF16 ? 8 : 4;
    if (c->block_stride < inner || c->block_stride % vec) return false;
    if (c->block_stride > INT64_MAX / 8 / (c->blocks > 0 ? c->blocks : 1)) return false;
    if (batch > 0 && (!c->seq_lens || (c->max_blocks > 0 && !c->block_tables) || (c->blocks > 0 && (!c->k || !c->v))))
        return false;
    if (!aligned16(c->k) || !aligned16(c->v)) return false;
    view.k = c->k;
    view.v = c->v;
    view.tables = c->block_tables;
    view.lens = c->seq_lens;
    view.block_stride = c->block_stride;
    view.blocks = static_cast<int>(c->blocks);
    view.max_blocks = c->max_blocks;
    view.heads = c->kv_heads;
    view.dim = c->head_dim;
    view.block = FastDiv(static_cast<uint32_t>(c->block_size));
    return true;
}

// A tensor of rows [.., heads, head_dim]: its pointer and row stride.
bool rows_ok(const specv_kv_cache* c, const void* p, int64_t stride) {
    const int64_t vec = c->dtype == SPECV_BF16 ? 8 : 4;
    return p && aligned16(p) && stride >= 0 && stride % vec == 0;
}

// Launch errors of the calls below.
specv_status launched(specv_ctx* h, const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, what);
    h->launches.fetch_add(1, std::memory_order_relaxed);
    return SPECV_OK;
}

// A launch whose CTAs may be placed while the kernel before still runs (they wait
// for its end on the device), so that launches overlap what runs before them.
template <typename... Params>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                         const Params&... params) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, params...);
}

// Lets a kernel have `bytes` of dynamic shared memory; once a device (a bit
// of `done` each) is enough.
cudaError_t allow_smem(std::atomic<uint64_t>& done, const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace
