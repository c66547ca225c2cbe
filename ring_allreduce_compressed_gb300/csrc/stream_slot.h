// stream_slot.h -- what scratch memory that is kept per stream is kept by.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <tuple>

namespace rra {

// A stream's place among those of its device: its handle or, for the
// per-thread default stream (one handle, a stream of its own in every host
// thread), the number of the calling thread.  A handle or a number comes back
// when its stream is destroyed or its thread ends; `id` does not.  A buffer
// that was kept under another id belongs to a stream that is gone, whose last
// work may still be running.  A stream that is being captured cannot be asked
// for its id (the question ends the capture): it is taken for the one that the
// place's buffer belongs to.
struct StreamSlot {
    int device = 0;
    bool thread = false;
    uintptr_t number = 0;
    bool capturing = false;
    unsigned long long id = 0;

    bool owns(unsigned long long buffer_id) const { return capturing || id == buffer_id; }

    bool operator<(const StreamSlot &o) const // places, whatever the id
    {
        return std::tie(device, thread, number) < std::tie(o.device, o.thread, o.number);
    }
};

// While one lives, its thread may allocate and free although a stream is being
// captured, by this thread or another: those calls are otherwise refused, and
// end the capture.
class AllocationAllowed {
public:
    AllocationAllowed() { cudaThreadExchangeStreamCaptureMode(&mode_); }
    ~AllocationAllowed() { cudaThreadExchangeStreamCaptureMode(&mode_); }
    AllocationAllowed(const AllocationAllowed &) = delete;
    AllocationAllowed &operator=(const AllocationAllowed &) = delete;

private:
    cudaStreamCaptureMode mode_ = cudaStreamCaptureModeRelaxed;
};

// A buffer of words that is kept for a slot.
struct StreamWords {
    uint32_t *p = nullptr;
    long long count = 0;
    unsigned long long id = 0; // of the stream that it belongs to
    bool captured = false;     // a graph may hold its address
};

// The slot of `st` on the current device; cudaErrorMemoryAllocation when there
// is no memory for a thread's number.
cudaError_t stream_slot(cudaStream_t st, StreamSlot *slot);

} // namespace rra
