// The runtime calls that csrc/kv.cu makes, as a host program: memory is the host's, streams
// are names with identities, and every call that matters is written to a log.  Linked with
// csrc/kv.cu and fake_kernels.cu it runs the cache's C entry points without a GPU.
#include <cuda_runtime_api.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <condition_variable>
#include <mutex>
#include <string>

namespace {

std::string g_log;
unsigned long long g_id[16];   // identity of the stream behind a handle value
bool g_capturing[16];
std::mutex g_mu;
std::condition_variable g_cv;
bool g_blocking = false, g_inside = false;

int slot(cudaStream_t s) { return (int)((uintptr_t)s & 15); }

}  // namespace

void say(const char* what, cudaStream_t s) { g_log += std::string(what) + " " + std::to_string((uintptr_t)s) + "\n"; }

extern "C" {

const char* fake_log() { return g_log.c_str(); }
void fake_clear() { g_log.clear(); }
void fake_identity(int handle, unsigned long long id) { g_id[handle & 15] = id; }
void fake_capturing(int handle, int on) { g_capturing[handle & 15] = on; }

cudaError_t cudaMalloc(void** p, size_t n) { return (*p = malloc(n)) ? cudaSuccess : cudaErrorMemoryAllocation; }
cudaError_t cudaFree(void* p) { free(p); g_log += "free\n"; return cudaSuccess; }
cudaError_t cudaHostAlloc(void** p, size_t n, unsigned) { return cudaMalloc(p, n); }
cudaError_t cudaFreeHost(void* p) { free(p); return cudaSuccess; }
cudaError_t cudaHostGetDevicePointer(void** d, void* h, unsigned) { *d = h; return cudaSuccess; }
cudaError_t cudaMemset(void* p, int v, size_t n) { memset(p, v, n); return cudaSuccess; }
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t s) { memset(p, v, n); say("memset", s); return cudaSuccess; }
cudaError_t cudaGetDeviceCount(int* n) { *n = 1; return cudaSuccess; }
cudaError_t cudaGetDevice(int* d) {
  std::unique_lock<std::mutex> l(g_mu);
  if (g_blocking) {
    g_blocking = false;  // the one call
    g_inside = true;
    g_cv.notify_all();
    g_cv.wait(l, [] { return !g_inside; });
  }
  *d = 0;
  return cudaSuccess;
}
// 1: the next call stays inside the library until 0; 2: waits until it is there
void fake_block(int what) {
  std::unique_lock<std::mutex> l(g_mu);
  if (what == 2) g_cv.wait(l, [] { return g_inside; });
  else if (what == 1) g_blocking = true;
  else g_inside = false;
  g_cv.notify_all();
}
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "an error"; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) { *e = reinterpret_cast<cudaEvent_t>(16); return cudaSuccess; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t s) { say("record", s); return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { g_log += "synchronize\n"; return cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t, unsigned) { say("wait", s); return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t s, cudaStreamCaptureStatus* st) {
  *st = g_capturing[slot(s)] ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
cudaError_t cudaStreamGetId(cudaStream_t s, unsigned long long* id) {
  *id = g_id[slot(s)];
  return g_capturing[slot(s)] ? cudaErrorStreamCaptureUnsupported : cudaSuccess;  // and it ends the capture
}

// a translation unit of CUDA registers its (here empty) device code when it is loaded
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
char __cudaInitModule(void**) { return 1; }

}  // extern "C"
