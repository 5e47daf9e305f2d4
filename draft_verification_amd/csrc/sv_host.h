// Host pieces that the library's source files share.
#ifndef SV_HOST_H
#define SV_HOST_H

#include <hip/hip_runtime.h>
#include <hip/hip_ext.h>

#include <stdint.h>

#include <tuple>

#include "spec_verify.h"

namespace sv {

// Checks the limits of a configuration (host only).
int check_config(const spec_verify_config* cfg);

// The configuration a handle was created with.
const spec_verify_config* handle_config(const spec_verify* h);

// Makes a device current for a scope.
struct DeviceGuard {
    int old = -1;
    explicit DeviceGuard(int dev)
    {
        if (hipGetDevice(&old) != hipSuccess) old = -1;
        if (old != dev) (void)hipSetDevice(dev);
    }
    ~DeviceGuard()
    {
        int cur = -1;
        if (old >= 0 && hipGetDevice(&cur) == hipSuccess && cur != old) (void)hipSetDevice(old);
    }
};

// Launches kernel on stream s with block threads per workgroup and returns the
// launch's own status.  With start and stop events the events are attached to
// the dispatch itself (hipExtLaunchKernel), so they time the kernel's
// execution and not the queue around it.
template <typename... KArgs, typename... Args>
hipError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, uint32_t shmem, hipStream_t s, hipEvent_t e0,
                         hipEvent_t e1, Args... args)
{
    std::tuple<KArgs...> t(args...);
    void* a[sizeof...(KArgs)];
    std::apply([&](auto&... x) {
        int i = 0;
        ((a[i++] = (void*)&x), ...);
    }, t);
    if (e0) return hipExtLaunchKernel((const void*)kernel, grid, block, a, shmem, s, e0, e1, 0);
    return hipLaunchKernel((const void*)kernel, grid, block, a, shmem, s);
}

} // namespace sv

#endif // SV_HOST_H
