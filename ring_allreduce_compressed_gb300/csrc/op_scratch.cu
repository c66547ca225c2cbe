// op_scratch.cu -- scratch memory of the training-step operators.
#include <map>
#include <new>
#include <utility>
#include <vector>

#include "op_common.cuh"
#include "stream_slot.h"

namespace rra {

namespace {

// Numbers of the threads that use their default stream: the lowest that no
// living thread has, and how many threads have had one.
struct Threads {
    std::mutex mu;
    std::vector<char> used;
    unsigned long long count = 0;
};

Threads &threads() // never destroyed: threads may end after static objects do
{
    static Threads *const t = new Threads;
    return *t;
}

struct ThreadNumber {
    size_t number = 0;
    unsigned long long id = 0;

    ThreadNumber()
    {
        Threads &t = threads();
        std::lock_guard<std::mutex> lk(t.mu);
        while (number < t.used.size() && t.used[number])
            ++number;
        if (number == t.used.size())
            t.used.push_back(1);
        t.used[number] = 1;
        id = ++t.count;
    }
    ~ThreadNumber()
    {
        Threads &t = threads();
        std::lock_guard<std::mutex> lk(t.mu);
        t.used[number] = 0;
    }
};

struct Buffer {
    unsigned char *p = nullptr;
    size_t bytes = 0;
    unsigned long long id = 0; // of the stream that it belongs to
    bool captured = false;     // a graph may hold its address
};

std::mutex g_mu;
std::map<StreamSlot, Buffer> g_ws;

std::mutex g_fn_mu;
std::map<std::pair<int, const void *>, int> g_fn_smem;

} // namespace

cudaError_t stream_slot(cudaStream_t st, StreamSlot *slot)
{
    cudaError_t e = cudaGetDevice(&slot->device);
    if (e != cudaSuccess)
        return e;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if ((e = cudaStreamIsCapturing(st, &cap)) != cudaSuccess)
        return e;
    slot->capturing = cap != cudaStreamCaptureStatusNone;
    slot->thread = st == cudaStreamPerThread;
    if (!slot->thread) {
        slot->number = reinterpret_cast<uintptr_t>(st);
        return slot->capturing ? cudaSuccess : cudaStreamGetId(st, &slot->id);
    }
    try {
        static thread_local const ThreadNumber mine;
        slot->number = mine.number;
        slot->id = mine.id;
    } catch (const std::bad_alloc &) {
        return cudaErrorMemoryAllocation;
    }
    return cudaSuccess;
}

rra_status op_scratch(cudaStream_t st, size_t bytes, std::unique_lock<std::mutex> &lk,
                      unsigned char **out)
{
    StreamSlot slot;
    cudaError_t e = stream_slot(st, &slot);
    if (e != cudaSuccess)
        return e == cudaErrorMemoryAllocation ? RRA_ERR_NOMEM : RRA_ERR_CUDA;
    lk = std::unique_lock<std::mutex>(g_mu);
    Buffer *ws = nullptr;
    try {
        ws = &g_ws[slot];
    } catch (const std::bad_alloc &) {
        return RRA_ERR_NOMEM;
    }
    if (ws->bytes < bytes || !slot.owns(ws->id)) {
        if (slot.capturing)
            return RRA_ERR_INVALID;
        const size_t want = ws->id == slot.id
                                ? std::max({bytes, 2 * ws->bytes, (size_t)1 << 20})
                                : std::max(bytes, (size_t)1 << 20);
        const AllocationAllowed allowed;
        unsigned char *const old = ws->captured ? nullptr : ws->p;
        *ws = Buffer{};
        // cudaFree waits for all of the device's work: the last calls that used
        // the buffer too, and those of a stream that is gone
        if (old && cudaFree(old) != cudaSuccess)
            return RRA_ERR_CUDA;
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
        *ws = Buffer{p, want, slot.id, false};
    }
    ws->captured |= slot.capturing;
    *out = ws->p;
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
