// Accesses of kernels that read and write every value once. A call that moves more than the
// 256 MB Infinity Cache holds marks them as not used again soon; a smaller one leaves its results
// there for the kernel that follows. Residual norm of 65536 x 768 (403 MB) 73.5 and, so marked, 70.3 us, its
// backward 77 and 70, with the residual in fp32 (805 MB) 153 and 140; 8192 x 4096 (268 MB) 46 and 50,
// 65536 x 128 (67 MB) 16 and 19. Head norm of 65536 tokens of 12 heads of 128 (403 MB) 80.5 and 75.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hy {

constexpr int64_t kInfinityCache = int64_t(256) << 20;

template <bool STREAM, class T>
__device__ __forceinline__ T load_once(const T* p) {
    if constexpr (STREAM)
        return __builtin_nontemporal_load(p);
    else
        return *p;
}
template <bool STREAM, class T>
__device__ __forceinline__ void store_once(T v, T* p) {
    if constexpr (STREAM)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}

}  // namespace hy
