// host.h - host-side helpers shared by the library's translation units:
// descriptor checks, per-device attributes and kernel launches. Nothing here
// allocates memory or synchronises.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "pagedkv.h"

#include "last_error.h"

namespace pagedkv {

constexpr int kMaxDevices = 64;

inline pa_status cuda_fail(cudaError_t e, const char *what)
{
    return fail(PA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int sm_count_of_current_device()
{
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return 148;
    }
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n > 0)
        return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return 148;
    }
    cache[dev].store(n, std::memory_order_relaxed);
    return n;
}

inline pa_status check_cache(const pa_cache_desc *c)
{
    if (!c)
        return fail(PA_ERR_INVALID_ARG, "cache descriptor is NULL");
    if (c->num_blocks < 0 || c->block_size <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0)
        return fail(PA_ERR_INVALID_ARG, "cache descriptor has a non-positive size");
    if (c->dtype != PA_F16 && c->dtype != PA_BF16 && c->dtype != PA_FP8_E4M3)
        return fail(PA_ERR_UNSUPPORTED, "cache dtype %d (need PA_F16, PA_BF16 or PA_FP8_E4M3)",
                    (int)c->dtype);
    if (c->dtype == PA_FP8_E4M3 && c->io_dtype != PA_F16 && c->io_dtype != PA_BF16)
        return fail(PA_ERR_UNSUPPORTED, "fp8 cache io_dtype %d (need PA_F16 or PA_BF16)",
                    (int)c->io_dtype);
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(PA_ERR_UNSUPPORTED, "head_dim %d (built: 64, 128)", c->head_dim);
    if (c->block_size != 8 && c->block_size != 16 && c->block_size != 32)
        return fail(PA_ERR_UNSUPPORTED, "block_size %d (built: 8, 16, 32)", c->block_size);
    return PA_OK;
}

// Bytes of one (block, head) tile and of one block (all heads).
inline size_t tile_bytes(const pa_cache_desc *c)
{
    const size_t rows = (size_t)c->block_size;
    return c->dtype == PA_FP8_E4M3 ? rows * c->head_dim + 4 * rows : rows * c->head_dim * 2;
}

inline size_t block_bytes(const pa_cache_desc *c) { return tile_bytes(c) * (size_t)c->num_kv_heads; }

// Raise a kernel's dynamic shared-memory limit once per device. `done` must
// be distinct for every kernel (one static per template instantiation of the
// caller), since the attribute belongs to the function.
template <typename Kernel>
inline cudaError_t allow_smem(Kernel k, size_t bytes, std::atomic<size_t> (&done)[kMaxDevices])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_relaxed) >= bytes)
        return cudaSuccess;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess)
        return e;
    e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess)
        return e;
    if (dev >= 0 && dev < kMaxDevices)
        done[dev].store(bytes, std::memory_order_relaxed);
    return cudaSuccess;
}

// Every kernel of the library is launched with programmatic stream
// serialisation: it may be scheduled while the previous kernel of the stream
// drains, and it waits (griddepcontrol.wait) for that kernel before reading
// or writing anything, in every CTA, so stream order holds for all data.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The driver's tensor-map encoder, looked up once.
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn tensor_map_encoder()
{
    static std::atomic<EncodeTiledFn> cached{nullptr};
    EncodeTiledFn f = cached.load(std::memory_order_acquire);
    if (f)
        return f;
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn) {
        cudaGetLastError();
        return nullptr;
    }
    f = reinterpret_cast<EncodeTiledFn>(fn);
    cached.store(f, std::memory_order_release);
    return f;
}

} // namespace pagedkv
