// The step planner's host code entered by two threads at once with different
// sizes, and the runtime calls that set a kernel's shared-memory limit and
// launch it stood in for: a limit that one call was given must hold until its
// launch, whatever the other asks for meanwhile.  Nothing touches a GPU.
#include <chrono>
#include <cstdio>
#include <map>
#include <mutex>
#include <thread>

#include "pa_step.cu"

static std::mutex lock_;
static std::map<const void*, int> limits;
static int launches, lowered, refused;

static void pause_ms(int ms) { std::this_thread::sleep_for(std::chrono::milliseconds(ms)); }

// the runtime's functions, by its names
extern "C" cudaError_t get_device(int* dev) asm("cudaGetDevice");
extern "C" cudaError_t set_attribute(const void*, cudaFuncAttribute, int) asm("cudaFuncSetAttribute");
extern "C" cudaError_t launch_kernel(const cudaLaunchConfig_t*, const void*, void**) asm("cudaLaunchKernelExC");

extern "C" cudaError_t get_device(int* dev) {
    *dev = 0;
    return cudaSuccess;
}

extern "C" cudaError_t set_attribute(const void* kernel, cudaFuncAttribute attr, int value) {
    if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize) return cudaSuccess;
    static thread_local int nth = 0;
    if (nth++ == 0) pause_ms(value < 60000 ? 300 : 0);           // a small request is slow to take effect
    const std::lock_guard<std::mutex> hold(lock_);
    if (value < limits[kernel]) ++lowered;
    limits[kernel] = value;
    return cudaSuccess;
}

extern "C" cudaError_t launch_kernel(const cudaLaunchConfig_t* cfg, const void* kernel, void**) {
    pause_ms(400);
    const std::lock_guard<std::mutex> hold(lock_);
    ++launches;
    const int limit = limits.count(kernel) ? limits[kernel] : 48 * 1024;
    if ((int)cfg->dynamicSmemBytes > limit) {
        ++refused;
        return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

template <class P>
static P* at(uintptr_t x) { return reinterpret_cast<P*>(x); }

static int plan(int seqs, int max_blocks, int rows) {
    const uintptr_t A = 0x100000;                                // never read
    return pa_plan_step(at<int32_t>(A), at<int32_t>(A), at<int32_t>(A), at<int32_t>(A), at<int64_t>(A), at<int32_t>(A),
                        at<int32_t>(A), at<int32_t>(A), at<int32_t>(A), at<int32_t>(A), at<int32_t>(A), at<int32_t>(A), 9, seqs,
                        rows, max_blocks, 4, 16, 64, nullptr, nullptr);
}

static int release(int released, int rows) {
    const uintptr_t A = 0x100000;
    return pa_release_rows(at<int32_t>(A), released, at<int32_t>(A), at<int32_t>(A), rows, 8, at<int32_t>(A), at<int32_t>(A),
                           9, nullptr, nullptr);
}

template <class F, class G>
static int both(F small, G large) {
    int a = 0, b = 0;
    std::thread first([&] { a = small(); });
    pause_ms(100);
    std::thread second([&] { b = large(); });
    first.join();
    second.join();
    return a | b;
}

int main() {
    int status = both([] { return plan(1024, 4, 180000); }, [] { return plan(2048, 4, 262144); });        // one cluster
    status |= both([] { return plan(2049, 256, 262144); }, [] { return plan(8192, 256, 262144); });       // two launches
    status |= both([] { return release(2049, 262144); }, [] { return release(8192, 262144); });
    if (status || lowered || refused || launches != 8) {
        std::printf("status %d, limits lowered %d times, %d of %d launches refused\n", status, lowered, refused, launches);
        return 1;
    }
    std::puts("ok");
    return 0;
}
