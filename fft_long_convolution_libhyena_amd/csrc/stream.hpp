// Accesses of kernels that read and write every value once. A call that moves more than the
// 256 MB Infinity Cache holds may mark them as not used again soon; a smaller one leaves its results
// there for the kernel that follows. Lines of 128 bytes that a marked instruction covers only in part do not stay for the
// one that takes the rest, and are moved again: marks are for accesses that cover whole lines. Head norm, 300 MiB, unmarked
// and marked: 128 bytes a head 65 and 60 us, 256 bytes 67 and 64; 64 bytes 67 and 76, 16 bytes 131 and 486; heads of 72 in
// bf16 91 and 114; 16 bytes of every 32 71 and 89. Residual norm of 65536 x 768 (403 MB) 73.5 and 70.3 us, its
// backward 77 and 70, with the residual in fp32 (805 MB) 153 and 140; 65536 x 128 (67 MB, which stay) 16 and 19.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hy {

constexpr int64_t kInfinityCache = int64_t(256) << 20;

constexpr int64_t kLine = 128;  // bytes
inline bool whole_lines(const void* p) { return (uintptr_t)p % kLine == 0; }

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
