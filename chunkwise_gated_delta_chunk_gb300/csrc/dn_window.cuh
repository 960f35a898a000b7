// Device helpers of the attention over a sliding window: tiles of query and key
// tokens, which of them see each other.
#pragma once

#include <math_constants.h>

#include "dn_layer.cuh"
#include "dn_window.h"

namespace dn {

// Which keys token t of a sequence sees; positions are counted from the sequence's start.
struct Sight {
    int window, sinks;
    __device__ __forceinline__ bool sees(int t, int j) const { return j <= t && (t - j < window || j < sinks); }
};

// Key tiles of `len` tokens that the tokens [t0, t1) see: [first, last] by the window, and
// [0, sink_end) before them for the sinks alone.
struct KeyTiles {
    int first, last, sink_end;
    KeyTiles() = default;
    __device__ __forceinline__ KeyTiles(int t0, int t1, int len, const Sight &s) {
        const int lo = t0 - s.window + 1;  // window <= 2^30
        first = lo > 0 ? lo / len : 0;
        last = (t1 - 1) / len;
        const int want = (s.sinks + len - 1) / len;
        sink_end = first < want ? first : want;
    }
    __device__ __forceinline__ int count() const { return sink_end + last - first + 1; }
    __device__ __forceinline__ int tile(int i) const { return i < sink_end ? i : first + i - sink_end; }
};

// Query tiles of `len` tokens that see a key of [j0, j1), of a sequence of L tokens: [j0 / len, last],
// and those behind up to `end` see the sinks among them alone.
struct QueryTiles {
    int first, last, end;
    __device__ __forceinline__ QueryTiles(int j0, int j1, int L, int len, const Sight &s) {
        first = j0 / len;
        end = (L - 1) / len;
        const long long far = (long long)j1 - 1 + s.window - 1;
        const int lim = far < L - 1 ? (int)far : L - 1;
        last = lim / len;
    }
};

__device__ __forceinline__ float redo_mark() { return __uint_as_float(kRedoBits); }
__device__ __forceinline__ bool is_redo(float x) { return __float_as_uint(x) == kRedoBits; }

}  // namespace dn
