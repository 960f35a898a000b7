// What the tensor-core kernels of the attention over a sliding window share.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "dn_tmap.h"
#include "dn_window.cuh"
#include "tc_ptx.cuh"
#include "dn_tc_sync.cuh"

namespace dn {

constexpr int kSinkCols = 32;  // keys of the narrow tile that holds the sinks alone, where they fit

__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {  // bits lo..hi of 32, where they are any
    lo = lo < 0 ? 0 : lo;
    hi = hi > 31 ? 31 : hi;
    return lo > hi ? 0u : (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo);
}

// Which of the keys k0 + 0..31 token t sees.
__device__ __forceinline__ uint32_t seen32(int t, int k0, const Sight &s) {
    const int hi = t - k0;
    const int lim = s.sinks - 1 - k0 < hi ? s.sinks - 1 - k0 : hi;
    return bit_range(hi - s.window + 1, hi) | bit_range(0, lim);
}

__device__ __forceinline__ void store32(void *dst, const uint32_t (&r)[8]) {  // 32 bytes at once
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

}  // namespace dn
