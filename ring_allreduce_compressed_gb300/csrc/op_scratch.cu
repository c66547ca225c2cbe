// op_scratch.cu -- scratch memory of the training-step operators.
#include <map>
#include <new>
#include <utility>

#include "op_common.cuh"

namespace rra {

namespace {

std::mutex g_mu;
std::map<std::pair<int, cudaStream_t>, std::pair<unsigned char *, size_t>> g_ws;

std::mutex g_fn_mu;
std::map<std::pair<int, const void *>, int> g_fn_smem;

} // namespace

rra_status op_scratch(cudaStream_t st, size_t bytes, std::unique_lock<std::mutex> &lk,
                      unsigned char **out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return RRA_ERR_CUDA;
    lk = std::unique_lock<std::mutex>(g_mu);
    std::pair<unsigned char *, size_t> *ws = nullptr;
    try {
        ws = &g_ws[{dev, st}];
    } catch (const std::bad_alloc &) {
        return RRA_ERR_NOMEM;
    }
    if (ws->second < bytes) {
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(st, &cap) != cudaSuccess)
            return RRA_ERR_CUDA;
        if (cap != cudaStreamCaptureStatusNone)
            return RRA_ERR_INVALID;
        const size_t want = std::max({bytes, 2 * ws->second, (size_t)1 << 20});
        unsigned char *p = nullptr;
        if (cudaMalloc(&p, want) != cudaSuccess) {
            cudaGetLastError(); // reported here, not by the next launch
            return RRA_ERR_NOMEM;
        }
        // on the caller's stream: ordered before the launches that follow
        if (cudaMemsetAsync(p, 0, kScratchHead, st) != cudaSuccess) {
            cudaFree(p);
            return RRA_ERR_CUDA;
        }
        ws->first = p;
        ws->second = want;
    }
    *out = ws->first;
    return RRA_OK;
}

cudaError_t op_allow(const void *fn, int smem, bool large_clusters)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    std::lock_guard<std::mutex> lk(g_fn_mu);
    int *have = nullptr;
    try {
        have = &g_fn_smem[{dev, fn}];
    } catch (const std::bad_alloc &) {
        return cudaErrorMemoryAllocation;
    }
    if (smem <= *have)
        return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && large_clusters)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
        *have = smem;
    return e;
}

} // namespace rra
