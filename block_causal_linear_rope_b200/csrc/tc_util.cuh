// Small device helpers shared by the tensor-core kernels.
#pragma once

#include <cuda_bf16.h>

#include "ptx_sm100.cuh"

namespace blin {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s: far beyond any legitimate wait

// Byte offset of 16-byte chunk `j` of row `r` inside a swizzled tile whose base
// is 1024-byte aligned (64B swizzle: rows of 64 B; 128B swizzle: rows of 128 B).
template <int D>
__device__ __forceinline__ uint32_t swz_chunk(int r, int j) {
    if constexpr (D == 32)
        return static_cast<uint32_t>(r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
    else
        return static_cast<uint32_t>(r * 128 + ((j ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

// Rounds a pointer into the kernel's dynamic shared memory up to 1024 bytes by
// indexing from it (not through an integer cast), so the compiler keeps every
// derived access in the shared address space (LDS/STS, not generic loads).
__device__ __forceinline__ uint8_t *align1024(uint8_t *p) {
    const uint32_t a = ptx::smem_u32(p);
    return p + ((1024u - (a & 1023u)) & 1023u);
}

// mbar_wait_bounded for hand-overs that are usually a few hundred cycles away:
// the warp suspends on the barrier at once, and the clock is read only after a
// whole suspend time (10 ms) has passed, not on the way into every wait.
__device__ __forceinline__ bool mbar_wait_patient(uint32_t bar, uint32_t parity, int *watchdog, int code) {
    if (ptx::mbar_try_wait(bar, parity) || ptx::mbar_try_wait_suspend(bar, parity, ptx::kSuspendHintNs)) return true;
    return ptx::mbar_wait_bounded(bar, parity, watchdog, code, kWaitLimitNs);
}

// One mbarrier arrival for the whole warp, after every lane's shared-memory
// accesses (and tcgen05 loads, fenced by the caller) are ordered before it.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
}

// 4D tensor-map coordinates (feature, token, head, batch) in the map's own
// dimension order: dims 1 and 2 are ordered by stride, so `swap` puts the head
// before the token (a token-interleaved [B][N][H][d] layout).
struct MapCoord {
    int y, z;
};
__device__ __forceinline__ MapCoord map_coord(int n, int h, int swap) { return swap ? MapCoord{h, n} : MapCoord{n, h}; }

}  // namespace blin
