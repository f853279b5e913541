// fake_runtime.cpp -- the part of the CUDA runtime that libgptq's host side
// calls, without a device: launches are written down instead of run, and
// refused where the real runtime would refuse them (more dynamic shared memory
// than the kernel's limit).  One device with 148 SMs of compute capability 10.
//
// With a hold set, cudaFuncSetAttribute lets two threads that set one kernel's
// limit run into each other: it waits (for that long at most) until both are
// inside, applies the larger value first and lets go of both when both are
// applied.
#include <cuda.h>
#include <cxxabi.h>
#include <driver_types.h>
#include <vector_types.h>

#include <algorithm>
#include <chrono>
#include <condition_variable>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

namespace {

constexpr int kDefaultLimit = 48 * 1024;

struct Kernel {
    std::string name;
    int limit = kDefaultLimit;
    std::vector<int> set;   // the values its limit was set to
};
struct Launch {
    std::string name;
    long long grid[3], threads, smem, cluster, early;
};

std::mutex m;
std::condition_variable cv;
std::map<const void*, Kernel>& kernels()
{
    static std::map<const void*, Kernel> k;
    return k;
}
std::vector<Launch> launches;
int hold_ms = 0;
std::map<const void*, std::vector<int>> pending;
int word = 0;

int launched(const void* f, dim3 grid, dim3 block, size_t smem, int cluster, int early)
{
    std::lock_guard<std::mutex> lk(m);
    const Kernel& k = kernels()[f];
    if (static_cast<long long>(smem) > k.limit) return cudaErrorInvalidValue;
    launches.push_back({k.name, {grid.x, grid.y, grid.z}, static_cast<long long>(block.x) * block.y * block.z,
                        static_cast<long long>(smem), cluster, early});
    return cudaSuccess;
}

CUresult encode(CUtensorMap* map, CUtensorMapDataType, cuuint32_t rank, void* p, const cuuint64_t* dims, const cuuint64_t* strides,
                const cuuint32_t* box, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                CUtensorMapFloatOOBfill)
{
    std::memset(map, 0, sizeof *map);
    if (reinterpret_cast<uintptr_t>(p) % 16) return CUDA_ERROR_INVALID_VALUE;
    for (cuuint32_t i = 0; i < rank; ++i)
        if (dims[i] < 1 || dims[i] > (cuuint64_t(1) << 32) || box[i] < 1 || box[i] > 256) return CUDA_ERROR_INVALID_VALUE;
    for (cuuint32_t i = 0; i + 1 < rank; ++i)
        if (strides[i] % 16 || strides[i] >= (cuuint64_t(1) << 40)) return CUDA_ERROR_INVALID_VALUE;
    return CUDA_SUCCESS;
}

struct Config {
    dim3 grid, block;
    size_t smem;
    void* stream;
};
thread_local std::vector<Config> configs;

}  // namespace

extern "C" {

void fake_hold(int ms) { hold_ms = ms; }
int fake_launches() { return static_cast<int>(launches.size()); }
void fake_forget()
{
    std::lock_guard<std::mutex> lk(m);
    launches.clear();
}
// Launch i: its kernel's name; v = grid x, y, z, threads, shared memory, cluster, early start.
void fake_launch(int i, char* name, int size, long long* v)
{
    std::lock_guard<std::mutex> lk(m);
    const Launch& l = launches[i];
    std::strncpy(name, l.name.c_str(), size - 1);
    name[size - 1] = 0;
    std::copy(l.grid, l.grid + 3, v);
    v[3] = l.threads;
    v[4] = l.smem;
    v[5] = l.cluster;
    v[6] = l.early;
}
// Compiled kernel i's name, or 0 where there is none.
int fake_kernel(int i, char* name, int size)
{
    std::lock_guard<std::mutex> lk(m);
    for (auto& [f, k] : kernels())
        if (i-- == 0) {
            std::strncpy(name, k.name.c_str(), size - 1);
            name[size - 1] = 0;
            return 1;
        }
    return 0;
}
// How many different values a kernel's limit was set to, the most over all.
int fake_most_limits()
{
    std::lock_guard<std::mutex> lk(m);
    size_t most = 0;
    for (auto& [f, k] : kernels()) {
        std::vector<int> v = k.set;
        std::sort(v.begin(), v.end());
        most = std::max<size_t>(most, std::unique(v.begin(), v.end()) - v.begin());
    }
    return static_cast<int>(most);
}

void** __cudaRegisterFatBinary(void*)
{
    static void* handle = nullptr;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, void*, void*, void*, void*, int*)
{
    int status = 0;
    char* plain = abi::__cxa_demangle(name, nullptr, nullptr, &status);
    kernels()[host].name = status == 0 ? plain : name;
    std::free(plain);
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, void* stream)
{
    configs.push_back({grid, block, smem, stream});
    return 0;
}
int __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* stream)
{
    const Config c = configs.back();
    configs.pop_back();
    *grid = c.grid;
    *block = c.block;
    *smem = c.smem;
    *static_cast<void**>(stream) = c.stream;
    return cudaSuccess;
}
int cudaLaunchKernel(const void* f, dim3 grid, dim3 block, void**, size_t smem, void*) { return launched(f, grid, block, smem, 1, 0); }
int cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**)
{
    int cluster = 1, early = 0;
    for (unsigned i = 0; i < c->numAttrs; ++i) {
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = static_cast<int>(c->attrs[i].val.clusterDim.x);
        if (c->attrs[i].id == cudaLaunchAttributeProgrammaticStreamSerialization)
            early = c->attrs[i].val.programmaticStreamSerializationAllowed;
    }
    if (c->gridDim.x % cluster) return cudaErrorInvalidValue;
    return launched(f, c->gridDim, c->blockDim, c->dynamicSmemBytes, cluster, early);
}
int cudaFuncSetAttribute(const void* f, int attr, int value)
{
    if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
    std::unique_lock<std::mutex> lk(m);
    if (value > 227 * 1024) return cudaErrorInvalidValue;
    const auto limit = std::chrono::milliseconds(hold_ms);
    std::vector<int>& mine = pending[f];
    if (hold_ms) {
        mine.push_back(value);
        cv.notify_all();
        cv.wait_for(lk, limit, [&] { return mine.size() >= 2; });
        cv.wait_for(lk, limit, [&] { return value >= *std::max_element(mine.begin(), mine.end()); });
    }
    kernels()[f].limit = value;
    kernels()[f].set.push_back(value);
    if (hold_ms) {
        mine.erase(std::find(mine.begin(), mine.end(), value));
        cv.notify_all();
        cv.wait_for(lk, limit, [&] { return mine.empty(); });
    }
    return cudaSuccess;
}
int cudaGetDriverEntryPoint(const char*, void** p, unsigned long long, int* result)
{
    *p = reinterpret_cast<void*>(encode);
    *result = 0;   // cudaDriverEntryPointSuccess
    return cudaSuccess;
}
int cudaDeviceGetAttribute(int* v, int attr, int)
{
    *v = attr == cudaDevAttrMultiProcessorCount ? 148 : attr == cudaDevAttrComputeCapabilityMajor ? 10 : 0;
    return cudaSuccess;
}
int cudaGetDevice(int* d)
{
    *d = 0;
    return cudaSuccess;
}
int cudaGetSymbolAddress(void** p, const void*)
{
    *p = &word;
    return cudaSuccess;
}
int cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorName(int) { return "fake"; }
const char* cudaGetErrorString(int) { return "refused by the fake runtime"; }

#define NOT_HERE(name) \
    int name() { return cudaErrorNotSupported; }
NOT_HERE(cudaDeviceGetStreamPriorityRange)
NOT_HERE(cudaDeviceSynchronize)
NOT_HERE(cudaEventCreate)
NOT_HERE(cudaEventCreateWithFlags)
NOT_HERE(cudaEventDestroy)
NOT_HERE(cudaEventElapsedTime)
NOT_HERE(cudaEventRecord)
NOT_HERE(cudaFreeHost)
NOT_HERE(cudaGraphDestroy)
NOT_HERE(cudaGraphExecDestroy)
NOT_HERE(cudaGraphInstantiate)
NOT_HERE(cudaGraphLaunch)
NOT_HERE(cudaHostAlloc)
NOT_HERE(cudaMemcpy)
NOT_HERE(cudaMemcpyAsync)
NOT_HERE(cudaMemcpyFromSymbol)
NOT_HERE(cudaMemset)
NOT_HERE(cudaMemsetAsync)
NOT_HERE(cudaOccupancyMaxActiveClusters)
NOT_HERE(cudaStreamBeginCapture)
NOT_HERE(cudaStreamCreateWithFlags)
NOT_HERE(cudaStreamCreateWithPriority)
NOT_HERE(cudaStreamEndCapture)
NOT_HERE(cudaStreamIsCapturing)
NOT_HERE(cudaStreamSynchronize)
NOT_HERE(cudaStreamWaitEvent)

}  // extern "C"
