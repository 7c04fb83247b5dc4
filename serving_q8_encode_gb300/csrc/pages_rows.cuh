// What the paged cache's kernels over runs of rows share: 16-bit pairs, and which sequence an item belongs to.
#pragma once

#include "pages_internal.cuh"

namespace polykv {

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack_rn(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}
// The sequence that owns an append item (all lanes of the warp get it).
__device__ __forceinline__ int find_seq(const int32_t* starts, int A, int64_t item, int page, int lane) {
    int lo = 0, n = A;
    while (n > 1) {
        const int stride = (n + 31) / 32;
        const int i = lane * stride;
        const bool le = i < n && item_base(starts[lo + i], lo + i, page) <= item;
        const int cnt = max(1, __popc(__ballot_sync(0xffffffffu, le)));
        lo += (cnt - 1) * stride;
        n = min(stride, n - (cnt - 1) * stride);
    }
    return lo;
}

}  // namespace polykv
