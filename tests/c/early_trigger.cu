// early_trigger.cu -- a kernel that lets the next one start at once and then
// takes its time: what stands before a programmatic launch may be slow.
#include <cuda_runtime.h>

__global__ void slow_kernel(long long ns, float *value)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    long long from, now;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(from));
    do {
        __nanosleep(1000);
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
    } while (now - from < ns);
    *value += 1.0f;
}

// One thread for up to 3 s, then value[0] += 1.
extern "C" int early_trigger(long long ms, float *value, void *stream)
{
    slow_kernel<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>((ms < 3000 ? ms : 3000) * 1000000LL, value);
    return static_cast<int>(cudaGetLastError());
}
