// sgmv_host.hpp -- host-side helpers shared by the C ABI's source files:
// kernel launches with their error bookkeeping, and pointer alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "sgmv.h"

namespace sgmv {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Threads along a grid's dimension are counted in 32 bits by the hardware.
inline bool grid_fits(long long blocks, int threads) { return blocks * threads <= 0xFFFFFFFFll; }

// Launch bookkeeping: every launch goes through hipLaunchKernel, whose
// return value describes that launch alone (hipGetLastError could also
// report an older, unrelated error of the caller's).  The first failure of a
// call is kept until launch_status() reads it; the last one stays readable
// through sgmv_last_hip_error().
inline thread_local hipError_t t_pending = hipSuccess;
inline thread_local hipError_t t_last = hipSuccess;

template <typename Tuple, size_t... I>
void arg_pointers(Tuple& t, void** out, std::index_sequence<I...>) {
    ((out[I] = (void*)&std::get<I>(t)), ...);
}

template <typename... KArgs, typename... Args>
void launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, hipStream_t st, Args&&... args) {
    static_assert(sizeof...(KArgs) == sizeof...(Args), "argument count mismatch");
    std::tuple<std::decay_t<KArgs>...> vals(static_cast<std::decay_t<KArgs>>(args)...);
    void* ptrs[sizeof...(KArgs) > 0 ? sizeof...(KArgs) : 1];
    arg_pointers(vals, ptrs, std::index_sequence_for<KArgs...>{});
    const hipError_t e = hipLaunchKernel((const void*)kernel, grid, block, ptrs, 0, st);
    if (e != hipSuccess && t_pending == hipSuccess) t_pending = e;
}

inline int launch_status() {
    const hipError_t e = t_pending;
    t_pending = hipSuccess;
    if (e == hipSuccess) return SGMV_OK;
    t_last = e;
    return SGMV_ERR_HIP;
}

}  // namespace sgmv
