// A stand-in for the parts of the HIP runtime that the library's host code calls, for
// tests without a GPU of what it does before and between its launches: memory is the
// host's, kernels are counted and not run, and failures are set by the test.  Loaded
// ahead of the library, its functions are the ones found.
#define __HIP_PLATFORM_AMD__
#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <set>

namespace {
thread_local hipStreamCaptureMode mode = hipStreamCaptureModeGlobal;
thread_local hipError_t last = hipSuccess;
std::set<void*> live;
thread_local struct {
    dim3 grid, block;
    size_t lds;
    hipStream_t stream;
} config;
hipError_t told(hipError_t e) {
    if (e != hipSuccess) last = e;
    return e;
}
}  // namespace

extern "C" {

struct {
    int64_t launches, mallocs, syncs;
    int64_t device;          // the current one
    int64_t largest;         // allocations above this fail
    int64_t stream_captured; // the calls' own stream is
    int64_t other_capture;   // another thread's capture is open ...
    int64_t ended;           // ... until a call that it does not allow
    int64_t live;            // allocations not freed
    int64_t blocks;          // workgroups of the last launch
} stub = {0, 0, 0, 0, INT64_MAX, 0, 0, 0, 0, 0};

// what no other thread may do while one captures, but for threads in relaxed mode
static bool forbidden() {
    if (mode != hipStreamCaptureModeGlobal || !(stub.other_capture || stub.stream_captured)) return false;
    stub.ended = 1;
    return true;
}

hipError_t hipMalloc(void** p, size_t n) {
    ++stub.mallocs;
    if (forbidden()) return told(hipErrorStreamCaptureUnsupported);
    if ((int64_t)n > stub.largest) return told(hipErrorOutOfMemory);
    *p = aligned_alloc(256, (n + 255) / 256 * 256);
    live.insert(*p);
    stub.live = (int64_t)live.size();
    return hipSuccess;
}
hipError_t hipFree(void* p) {
    if (forbidden()) return told(hipErrorStreamCaptureUnsupported);
    if (!p) return hipSuccess;
    if (!live.erase(p)) return told(hipErrorInvalidValue);
    stub.live = (int64_t)live.size();
    free(p);
    return hipSuccess;
}
hipError_t hipMemcpyAsync(void* d, const void* s, size_t n, hipMemcpyKind, hipStream_t) {
    memcpy(d, s, n);
    return hipSuccess;
}
hipError_t hipMemcpy2DAsync(void* d, size_t dp, const void* s, size_t sp, size_t w, size_t h, hipMemcpyKind, hipStream_t) {
    for (size_t i = 0; i < h; ++i) memcpy((char*)d + i * dp, (const char*)s + i * sp, w);
    return hipSuccess;
}
hipError_t hipMemsetAsync(void* d, int v, size_t n, hipStream_t) {
    memset(d, v, n);
    return hipSuccess;
}
hipError_t hipStreamSynchronize(hipStream_t) {
    ++stub.syncs;
    if (stub.stream_captured) {  // in every mode
        stub.ended = 1;
        return told(hipErrorStreamCaptureUnsupported);
    }
    return hipSuccess;
}
hipError_t hipDeviceSynchronize() {
    ++stub.syncs;
    if (stub.stream_captured || stub.other_capture) {  // in every mode
        stub.ended = 1;
        return told(hipErrorStreamCaptureUnsupported);
    }
    return hipSuccess;
}
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* s) {
    *s = stub.stream_captured ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
    return hipSuccess;
}
hipError_t hipThreadExchangeStreamCaptureMode(hipStreamCaptureMode* m) {
    const hipStreamCaptureMode was = mode;
    mode = *m;
    *m = was;
    return hipSuccess;
}
hipError_t hipGetDevice(int* d) {
    *d = (int)stub.device;
    return hipSuccess;
}
hipError_t hipSetDevice(int d) {
    stub.device = d;
    return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
    memset(p, 0, sizeof *p);
    p->multiProcessorCount = 256;
    return hipSuccess;
}
hipError_t hipPointerGetAttributes(hipPointerAttribute_t* a, const void*) {
    memset(a, 0, sizeof *a);
    a->type = hipMemoryTypeDevice;
    return hipSuccess;
}
hipError_t hipGetLastError() {
    const hipError_t e = last;
    last = hipSuccess;
    return e;
}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t s) {
    config = {grid, block, lds, s};
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* s) {
    *grid = config.grid, *block = config.block, *lds = config.lds, *s = config.stream;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
    if (!grid.x || !grid.y || !grid.z || grid.y > 65535 || grid.z > 65535 || (uint64_t)grid.x * block.x >= (uint64_t)1 << 32)
        return told(hipErrorInvalidConfiguration);
    ++stub.launches;
    stub.blocks = (int64_t)grid.x * grid.y * grid.z;
    return hipSuccess;
}

}  // extern "C"
