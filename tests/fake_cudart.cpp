// A stand-in for the CUDA runtime, linked with the library's own objects, so that the host side
// of every entry point (checks, plans, bookkeeping, what it allocates and launches, what it does
// when a call or an allocation fails) runs and is tested without a GPU.  Device memory is
// reserved address space that nothing writes, launches are recorded and run nothing, and the
// test says which call fails.
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <sys/mman.h>

#include <cstdlib>
#include <cstring>
#include <map>
#include <new>
#include <string>
#include <vector>

namespace {

struct Launch {
  std::string name;
  dim3 grid;
};

// Everything below lives in one object that is made before the library's static initialisers
// register its kernels, and outside of the counted allocations (`quiet`).
struct State {
  std::map<const void *, std::string> kernels;
  std::map<void *, size_t> live;
  std::vector<Launch> launches;
  long long live_bytes = 0;
  int fail_malloc = -1, fail_launch = -1, fail_new = -1;  // calls until the one that fails
  int news = 0;
  int capture_mode = cudaStreamCaptureModeGlobal;
  bool capturing = false;
  int bad_mallocs = 0;  // cudaMalloc in a capture without the relaxed mode
  dim3 grid, block;
  size_t smem = 0;
  cudaStream_t stream = nullptr;
};

int quiet = 0;
struct Quiet {
  Quiet() { ++quiet; }
  ~Quiet() { --quiet; }
};

State &st() {
  static State *s = [] {
    Quiet q;
    return new State;
  }();
  return *s;
}

bool hit(int &countdown) { return countdown >= 0 && countdown-- == 0; }

cudaError_t launch(const void *fn, dim3 grid) {
  Quiet q;
  if (hit(st().fail_launch)) return cudaErrorLaunchOutOfResources;
  const auto it = st().kernels.find(fn);
  st().launches.push_back({it == st().kernels.end() ? "?" : it->second, grid});
  return cudaSuccess;
}

CUresult encode(...) { return CUDA_SUCCESS; }

}  // namespace

// ------------------------------------------------------------------ host allocations
void *operator new(size_t n) {
  if (!quiet) {
    ++st().news;
    if (hit(st().fail_new)) throw std::bad_alloc();
  }
  if (void *p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, size_t) noexcept { std::free(p); }

// ------------------------------------------------------------------ what a test asks
extern "C" {

void fake_reset() {
  Quiet q;
  State &s = st();
  s.launches.clear();
  s.fail_malloc = s.fail_launch = s.fail_new = -1;
  s.news = s.bad_mallocs = 0;
  s.capturing = false;
}
long long fake_live_bytes() { return st().live_bytes; }
int fake_live_blocks() { return (int)st().live.size(); }
int fake_launches() { return (int)st().launches.size(); }
const char *fake_launch_name(int i) { return st().launches[i].name.c_str(); }
int fake_launch_grid(int i) { return (int)st().launches[i].grid.x; }
void fake_fail_malloc(int after) { st().fail_malloc = after; }
void fake_fail_launch(int after) { st().fail_launch = after; }
void fake_fail_new(int after) {
  st().news = 0;
  st().fail_new = after;
}
int fake_news() { return st().news; }
void fake_capturing(int on) { st().capturing = on != 0; }
int fake_bad_mallocs() { return st().bad_mallocs; }

// ------------------------------------------------------------------ registration
void **__cudaRegisterFatBinary(void *) {
  static void *handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, uint3 *,
                            uint3 *, dim3 *, dim3 *, int *) {
  Quiet q;
  st().kernels[host] = name;
}

// ------------------------------------------------------------------ launches
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
  State &s = st();
  s.grid = grid, s.block = block, s.smem = smem, s.stream = stream;
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3 *grid, dim3 *block, size_t *smem, void *stream) {
  State &s = st();
  *grid = s.grid, *block = s.block, *smem = s.smem;
  *static_cast<cudaStream_t *>(stream) = s.stream;
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *fn) {
  *k = (cudaKernel_t)fn;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 grid, dim3, void **, size_t, cudaStream_t) {
  return launch((const void *)k, grid);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *fn, void **) {
  return launch(fn, c->gridDim);
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }

// ------------------------------------------------------------------ memory
cudaError_t cudaMalloc(void **p, size_t n) {
  Quiet q;
  State &s = st();
  *p = nullptr;
  if (s.capturing && s.capture_mode != cudaStreamCaptureModeRelaxed) {
    ++s.bad_mallocs;
    return cudaErrorStreamCaptureUnsupported;
  }
  if (hit(s.fail_malloc)) return cudaErrorMemoryAllocation;
  void *m = mmap(nullptr, n ? n : 1, PROT_READ | PROT_WRITE,
                 MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0);
  if (m == MAP_FAILED) return cudaErrorMemoryAllocation;
  s.live[m] = n;
  s.live_bytes += (long long)n;
  *p = m;
  return cudaSuccess;
}
cudaError_t cudaFree(void *p) {
  Quiet q;
  State &s = st();
  if (!p) return cudaSuccess;
  const auto it = s.live.find(p);
  if (it == s.live.end()) return cudaErrorInvalidValue;
  munmap(p, it->second ? it->second : 1);
  s.live_bytes -= (long long)it->second;
  s.live.erase(it);
  return cudaSuccess;
}
cudaError_t cudaMemset(void *, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpy(void *, const void *, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void *, const void *, size_t, cudaMemcpyKind, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes *a, const void *) {
  std::memset(a, 0, sizeof *a);
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void **p, const void *) {
  *p = nullptr;
  return cudaErrorInvalidSymbol;
}

// ------------------------------------------------------------------ device, streams, events
cudaError_t cudaGetDevice(int *d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetDeviceCount(int *n) {
  *n = 1;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) {
  *v = 152;  // SMs, all that the library asks for
  return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *r) {
  *p = reinterpret_cast<void *>(encode);
  if (r) *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus *c) {
  *c = st().capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode *m) {
  const int was = st().capture_mode;
  st().capture_mode = *m;
  *m = (cudaStreamCaptureMode)was;
  return cudaSuccess;
}
cudaError_t cudaEventCreate(cudaEvent_t *e) {
  *e = (cudaEvent_t)1;
  return cudaSuccess;
}
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventElapsedTime(float *ms, cudaEvent_t, cudaEvent_t) {
  *ms = 0;
  return cudaSuccess;
}

// ------------------------------------------------------------------ graphs
cudaError_t cudaGraphCreate(cudaGraph_t *g, unsigned) {
  *g = (cudaGraph_t)1;
  return cudaSuccess;
}
cudaError_t cudaGraphDestroy(cudaGraph_t) { return cudaSuccess; }
cudaError_t cudaGraphAddKernelNode(cudaGraphNode_t *n, cudaGraph_t, const cudaGraphNode_t *, size_t,
                                   const cudaKernelNodeParams *) {
  *n = (cudaGraphNode_t)1;
  return cudaSuccess;
}
cudaError_t cudaGraphAddDependencies(cudaGraph_t, const cudaGraphNode_t *, const cudaGraphNode_t *,
                                     const cudaGraphEdgeData *, size_t) {
  return cudaSuccess;
}
cudaError_t cudaGraphInstantiate(cudaGraphExec_t *e, cudaGraph_t, unsigned long long) {
  *e = (cudaGraphExec_t)1;
  return cudaSuccess;
}
cudaError_t cudaGraphExecKernelNodeSetParams(cudaGraphExec_t, cudaGraphNode_t,
                                             const cudaKernelNodeParams *) {
  return cudaSuccess;
}
cudaError_t cudaGraphExecDestroy(cudaGraphExec_t) { return cudaSuccess; }
cudaError_t cudaGraphLaunch(cudaGraphExec_t, cudaStream_t) { return cudaSuccess; }

}  // extern "C"
