// Stand-ins for the CUDA runtime calls of the operators around the routed experts, so that
// their host code runs without a GPU: several devices that remember which kernel was allowed
// how much shared memory on which of them, and a log of what was launched and copied.
#include <cuda_runtime_api.h>

#include <cstdio>
#include <cstring>
#include <map>
#include <set>
#include <string>
#include <utility>
#include <vector>

namespace {
struct Launch {
  int device;
  std::string kernel;
  unsigned grid[3];
  int cluster;
  size_t smem;
};
int device = 0;
int status_word = 0;  // what the products' status reads
std::map<const void*, std::string> names;
std::map<std::pair<int, const void*>, int> allowed;
std::vector<Launch> launches;
std::vector<std::string> calls;
int word[64];

cudaError_t launch(const void* f, dim3 grid, size_t smem, int cluster) {
  const int most = allowed.count({device, f}) ? allowed[{device, f}] : 48 * 1024;
  if (smem > static_cast<size_t>(most)) return cudaErrorInvalidValue;
  launches.push_back({device, names[f], {grid.x, grid.y, grid.z}, cluster, smem});
  return cudaSuccess;
}
}  // namespace

namespace moe {
int report_error(int code, const char* msg) {
  std::fprintf(stderr, "%d: %s\n", code, msg);
  return code;
}
}  // namespace moe

extern "C" {
// ---- the tests' side
void fake_device(int d) { device = d; }
void fake_status(int v) { status_word = v; }
int fake_launches() { return static_cast<int>(launches.size()); }
void fake_launch(int i, int* dev, char* name, int room, unsigned* grid, int* cluster) {
  const Launch& l = launches[i];
  *dev = l.device, *cluster = l.cluster;
  std::snprintf(name, room, "%s", l.kernel.c_str());
  std::memcpy(grid, l.grid, sizeof(l.grid));
}
int fake_calls(const char* name) {
  int n = 0;
  for (const std::string& c : calls) n += c == name;
  return n;
}
void fake_clear() {
  launches.clear();
  calls.clear();
}

// ---- what compiled host code registers
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, void*, void*, void*, void*, int*) {
  names[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaErrorUnknown; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaErrorUnknown; }

// ---- the runtime
cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute attr, int value) {
  if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize) allowed[{device, f}] = value;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* cfg) {
  if (!allowed.count({device, f})) return cudaErrorInvalidValue;
  *n = 152 / static_cast<int>(cfg->attrs[0].val.clusterDim.x);
  calls.push_back("cudaOccupancyMaxActiveClusters");
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void* f, void**) {
  int cluster = 1;
  for (unsigned i = 0; i < cfg->numAttrs; ++i)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = cfg->attrs[i].val.clusterDim.x;
  return launch(f, cfg->gridDim, cfg->dynamicSmemBytes, cluster);
}
static int encode_nothing() { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* found) {
  *fn = reinterpret_cast<void*>(&encode_nothing);
  *found = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) {
  *p = &word[device];
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void* to, const void*, size_t n, cudaMemcpyKind, cudaStream_t) {
  std::memcpy(to, &status_word, n);
  calls.push_back("cudaMemcpyAsync");
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void*, int v, size_t, cudaStream_t) {
  status_word = v;
  calls.push_back("cudaMemsetAsync");
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "refused"; }
cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode*) { return cudaSuccess; }
cudaError_t cudaMemPoolCreate(cudaMemPool_t*, const cudaMemPoolProps*) { return cudaErrorNotSupported; }
cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t, cudaMemPoolAttr, void*) { return cudaErrorNotSupported; }
cudaError_t cudaMemPoolDestroy(cudaMemPool_t) { return cudaSuccess; }
cudaError_t cudaMallocFromPoolAsync(void**, size_t, cudaMemPool_t, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t cudaFreeAsync(void*, cudaStream_t) { return cudaSuccess; }
}
