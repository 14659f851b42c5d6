// watchdog.cu -- the device watchdog word and its test hook.
//
// Every spin-wait in this library's kernels is bounded (fc::mbar_wait_bounded).  A wait that runs
// out sets this word instead of trapping or hanging; the kernel then unwinds normally, so the
// context stays usable and the host learns of it through fuse_check() as FUSE_ETIMEOUT.
#include <mutex>

#include "fc_internal.cuh"
#include "fc_ptx.cuh"

// [0] the watchdog word, [1] the index word: set by a kernel that met a page, slot or position index
// (or a length) outside its range in device memory, where the host cannot check it.  The kernel leaves
// out what the index named and goes on; fuse_check() reports FUSE_EINDEX.
__device__ int g_fc_status[2];

namespace fc {

// Device address of the watchdog word on the current device (looked up once per device).
int* watchdog_flag() {
    static std::mutex mu;
    static int* cached[64] = {nullptr};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        (void)cudaGetLastError();
        return nullptr;
    }
    std::lock_guard<std::mutex> lock(mu);
    if (!cached[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_fc_status) != cudaSuccess) {
            (void)cudaGetLastError();
            return nullptr;
        }
        cached[dev] = static_cast<int*>(p);
    }
    return cached[dev];
}

int* index_flag() {
    int* p = watchdog_flag();
    return p ? p + 1 : nullptr;
}

namespace {
__device__ int g_fc_taken[2];
// Read and clear both words, each in one step: what another stream's kernel sets in between stays for the next check.
__global__ void status_take_kernel() {
    for (int i = 0; i < 2; ++i) g_fc_taken[i] = atomicExch(&g_fc_status[i], 0);
}
}  // namespace

int status_take(cudaStream_t stream) {
    int v[2] = {0, 0};
    if (cudaMemcpyFromSymbol(v, g_fc_status, sizeof(v)) != cudaSuccess) {
        (void)cudaGetLastError();
        return FUSE_OK;
    }
    if (!v[0] && !v[1]) return FUSE_OK;
    static std::mutex mu;      // one check at a time over g_fc_taken
    std::lock_guard<std::mutex> lock(mu);
    status_take_kernel<<<1, 1, 0, stream>>>();
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(v, g_fc_taken, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return record_cuda_error(e);
    return v[0] ? FUSE_ETIMEOUT : v[1] ? FUSE_EINDEX : FUSE_OK;
}

namespace {
// One thread waits on an mbarrier that nobody arrives on; the bounded wait gives up after
// `budget` cycles, raises the flag and the kernel returns.
__global__ void watchdog_probe_kernel(int* flag, long long budget) {
    __shared__ __align__(8) uint64_t bar;
    const uint32_t b = smem_addr(&bar);
    mbar_init(b, 1);
    fence_mbar_init();
    (void)mbar_wait_bounded(b, 0, flag, budget);
}
}  // namespace

}  // namespace fc

extern "C" int fuse_debug_expire_wait(int64_t budget_cycles, fuse_stream_t stream) {
    if (budget_cycles < 0 || budget_cycles >= (int64_t(1) << 31)) return FUSE_EINVAL;
    int* flag = fc::watchdog_flag();
    if (!flag) return FUSE_ECUDA;
    fc::watchdog_probe_kernel<<<1, 1, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        flag, static_cast<long long>(budget_cycles));
    return fc::check_launch();
}
