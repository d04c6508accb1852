// cba_attn.cuh -- what attention's two directions share: the tiles' geometry,
// 16-bit pairs, loads of tiles, rings of barriers, the strides of a call.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "cba_internal.cuh"
#include "cba_ptx.cuh"
#include "cba_types.cuh"

namespace cba {

constexpr uint64_t kAtLimitNs = 2000000000ull;
constexpr int kT = 128;                       // tile rows, of queries and of keys
constexpr uint32_t kBoxBytes = kT * 128u;     // 128 rows x 64 16-bit elements
constexpr float kLog2e = 1.4426950408889634f;

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
    if constexpr (BF16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&u));
    else return __half22float2(*reinterpret_cast<__half2 *>(&u));
}

// Loads a 128-row tile (DP / 64 boxes) into `dst`, completing `bar`'s phase.
// Where only `valid` of its rows are the sequence's own (packed sequences; the
// tensor map itself fills rows past a dense one with zeros), the tile arrives on
// the barrier `fix` first and the rows past them are zeroed: they are contracted
// over with P = dS = 0, which an infinity or NaN next door must not meet.
// Called by a whole warp.
template <int DP>
__device__ __forceinline__ bool load_tile(uint32_t dst, const CUtensorMap *tm, long long token,
                                          int head, int b, int valid, bool packed, uint32_t bar,
                                          uint32_t fix, uint32_t &fix_phase, volatile int *abort,
                                          unsigned *status) {
    const int lane = threadIdx.x & 31;
    const bool tail = packed && valid < kT;
    if (lane == 0) {
        const uint32_t on = tail ? fix : bar;
        ptx::mbar_arrive_expect_tx(on, DP / 64 * kBoxBytes);
#pragma unroll
        for (int j = 0; j < DP / 64; ++j)
            ptx::tma_load_4d(dst + j * kBoxBytes, tm, j * 64, (int)token, head, b, on);
    }
    if (tail) {
        bool ok = ptx::mbar_wait_bounded(fix, fix_phase, abort, status, kAtLimitNs);
        fix_phase ^= 1;
        if (!__all_sync(0xffffffffu, ok)) return false;
        for (int r = valid * 8 + lane; r < kT * 8; r += 32)
#pragma unroll
            for (int j = 0; j < DP / 64; ++j)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + j * kBoxBytes + r * 16),
                             "r"(0)
                             : "memory");
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar);
    }
    __syncwarp();
    return true;
}

__device__ __forceinline__ void at_init_bars(uint64_t *first, int n, uint32_t count) {
    for (int i = 0; i < n; ++i) ptx::mbar_init(ptx::smem_u32(first + i), count);
}

// A ring's stage and the parity of its phase.
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void step(int stages) {
        if (++s == stages) s = 0, ph ^= 1;
    }
};

// A warp's wait for two barriers at once, half of the lanes on each: a wait takes
// ~150 cycles even when its phase is over, in which the MMA warp issues none.  (Two
// warps that issue MMAs in turn hide that, but their MMAs then alternate between
// accumulators and run at half the rate: kv 666 -> 975 us on 1x8192 h32/8 d128.)
struct AtWait {
    uint64_t *bar;
    uint32_t parity;
};
__device__ __forceinline__ bool wait_both(AtWait x, AtWait y, volatile int *abort, unsigned *status) {
    const AtWait w = threadIdx.x & 1 ? y : x;
    const bool r = ptx::mbar_wait_bounded(ptx::smem_u32(w.bar), w.parity & 1u, abort, status, kAtLimitNs);
    ptx::tc_fence_after();
    return __all_sync(0xffffffffu, r) != 0;
}

// After a timeout the load warp waits (bounded) for the copies it has begun: the
// last `stages` of `count` phases of a ring.
__device__ __forceinline__ void drain_ring(uint64_t *bars, int stages, int count, unsigned *status) {
    int no = 0;
    for (int v = max(0, count - stages); v < count; ++v)
        ptx::mbar_wait_bounded(ptx::smem_u32(bars + v % stages), (uint32_t)(v / stages) & 1u, &no, status,
                               kAtLimitNs / 8);
}

// The strides that the kernels use; packed sequences have none from one to the next.
inline void fill_strides(const cba_attention_desc_t &d, const cba_attn_strides_t &s, int heads, long long len, long long *out) {
    if (s.batch == 0 && s.token == 0 && s.head == 0) {
        out[0] = len * heads * d.dim;
        out[1] = (long long)heads * d.dim;
        out[2] = d.dim;
    } else {
        out[0] = s.batch;
        out[1] = s.token;
        out[2] = s.head;
    }
    if (d.packed) out[0] = 0;
}

}  // namespace cba
