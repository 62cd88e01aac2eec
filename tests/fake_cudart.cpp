// A CUDA runtime without a device, for tests of the library's host code on the CPU:
// the library's objects are linked with this file instead of libcudart. Device memory
// is host memory; no kernel runs, launches are recorded. A copy to the device is held
// back until something waits for it, as the real one may be: a cudaMemcpy from pageable
// memory returns once its bytes are staged.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <vector>

namespace {
struct Copy {
  void *dst;
  std::vector<uint8_t> bytes;
};
struct Launch {
  std::string name;
  std::vector<uint64_t> args;  // of kernels whose parameters are pointers and 8-byte values, else empty
};
std::vector<Copy> g_pending;
std::map<const void *, std::string> g_names;
std::vector<Launch> g_launches;
int g_regs = 168;

void arrive() {
  for (const Copy &c : g_pending) std::memcpy(c.dst, c.bytes.data(), c.bytes.size());
  g_pending.clear();
}
cudaError_t copy(void *dst, const void *src, size_t n, cudaMemcpyKind kind) {
  if (kind == cudaMemcpyHostToDevice) {
    const uint8_t *p = static_cast<const uint8_t *>(src);
    g_pending.push_back({dst, std::vector<uint8_t>(p, p + n)});
    return cudaSuccess;
  }
  arrive();
  std::memcpy(dst, src, n);
  return cudaSuccess;
}
cudaError_t launch(const void *f, void **args) {
  Launch l{g_names[f], {}};
  // the gather kernels' leading parameters: the tests look at their pointers
  const int n = l.name.find("lora_gather_set_kernel") != std::string::npos    ? 6
                : l.name.find("lora_gather_rows_kernel") != std::string::npos ? 3
                                                                              : 0;
  for (int i = 0; i < n; ++i) {
    uint64_t v = 0;
    std::memcpy(&v, args[i], i == 4 ? 4 : 8);  // (the set kernel's fifth is an int)
    l.args.push_back(v);
  }
  g_launches.push_back(l);
  return cudaSuccess;
}
CUresult encode(CUtensorMap *m, CUtensorMapDataType, cuuint32_t, void *base, const cuuint64_t *, const cuuint64_t *,
                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  if (reinterpret_cast<uintptr_t>(base) & 15u) return CUDA_ERROR_INVALID_VALUE;
  std::memset(m, 0, sizeof(*m));
  return CUDA_SUCCESS;
}
}  // namespace

extern "C" {
// ---- what the tests set and read
void fake_set_regs(int n) { g_regs = n; }
int fake_pending() { return static_cast<int>(g_pending.size()); }
int fake_launches() { return static_cast<int>(g_launches.size()); }
const char *fake_launch_name(int i) { return g_launches[i].name.c_str(); }
int fake_launch_args(int i) { return static_cast<int>(g_launches[i].args.size()); }
uint64_t fake_launch_arg(int i, int k) { return g_launches[i].args[k]; }
void fake_clear() { g_launches.clear(); }

// ---- registration, as nvcc's host code calls it
void **__cudaRegisterFatBinary(void *) {
  static void *handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *host, char *, const char *name, int, void *, void *, void *, void *,
                            int *) {
  g_names[host] = name;
}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
static dim3 g_grid, g_block;
static size_t g_shared;
static cudaStream_t g_stream;
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t shared, cudaStream_t stream) {
  g_grid = grid, g_block = block, g_shared = shared, g_stream = stream;
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3 *grid, dim3 *block, size_t *shared, void *stream) {
  *grid = g_grid, *block = g_block, *shared = g_shared, *static_cast<cudaStream_t *>(stream) = g_stream;
  return cudaSuccess;
}

// ---- the runtime calls of the library
cudaError_t cudaGetDevice(int *d) { return *d = 0, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrMultiProcessorCount ? 148 : 0;
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPoint(const char *, void **fn, unsigned long long, cudaDriverEntryPointQueryResult *q) {
  *fn = reinterpret_cast<void *>(&encode);
  if (q) *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes *a, const void *) {
  std::memset(a, 0, sizeof(*a));
  a->numRegs = g_regs;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *) { return *n = 1, cudaSuccess; }
cudaError_t cudaMalloc(void **p, size_t n) { return posix_memalign(p, 256, n ? n : 1) ? cudaErrorMemoryAllocation : cudaSuccess; }
cudaError_t cudaFree(void *p) { return arrive(), std::free(p), cudaSuccess; }
cudaError_t cudaHostAlloc(void **p, size_t n, unsigned) { return cudaMalloc(p, n); }
cudaError_t cudaFreeHost(void *p) { return std::free(p), cudaSuccess; }
cudaError_t cudaMemcpy(void *d, const void *s, size_t n, cudaMemcpyKind k) { return copy(d, s, n, k); }
cudaError_t cudaMemcpyAsync(void *d, const void *s, size_t n, cudaMemcpyKind k, cudaStream_t) { return copy(d, s, n, k); }
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void *d, const void *, size_t n, size_t, cudaMemcpyKind) { return std::memset(d, 0, n), cudaSuccess; }
cudaError_t cudaMemcpyToSymbol(const void *, const void *, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void **p, const void *) {
  static uint64_t symbol[2];
  return *p = symbol, cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return arrive(), cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus *s) { return *s = cudaStreamCaptureStatusNone, cudaSuccess; }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t *e, unsigned) { return *e = reinterpret_cast<cudaEvent_t>(std::malloc(1)), cudaSuccess; }
cudaError_t cudaEventDestroy(cudaEvent_t e) { return std::free(e), cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return arrive(), cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaLaunchKernel(const void *f, dim3, dim3, void **args, size_t, cudaStream_t) { return launch(f, args); }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *f, void **args) { return launch(f, args); }
}
