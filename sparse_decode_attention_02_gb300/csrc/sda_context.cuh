// Driver calls from host threads that have made no CUDA call before.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace sda {

// fn(args...), a driver call that wants a context: a host thread has none until a
// runtime call has bound the current device's to it.
template <typename Fn, typename... Args>
inline CUresult with_context(Fn fn, Args... args)
{
    CUresult r = fn(args...);
    int dev = 0;
    if (r != CUDA_SUCCESS && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess)
        r = fn(args...);
    return r;
}

}  // namespace sda
