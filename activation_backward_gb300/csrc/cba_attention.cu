// cba_attention.cu -- attention's backward pass, which recomputes the
// probabilities from q, k and the rows' log-sum-exp.
//
//   S = scale q k^T,  P = exp(S - lse) on the allowed pairs, 0 elsewhere
//   D = rowsum(do o),  dP = do v^T,  dS = P (dP - D)
//   dv = P^T do,  dk = scale dS^T q,  dq = scale dS k
//   (dk and dv summed over the query heads that share a key/value head)
//
// Three launches:
//   attn_prep_kernel   D and lse in base 2 per query row, in rows padded to
//                      whole tiles (padding rows: lse = +inf, so P = 0)
//   attn_kv_kernel     one 128-row tile of keys per block, all its queries and
//                      query heads in turn: S^T and dP^T (keys on TMEM lanes),
//                      dv += P^T do, dk += dS^T q
//   attn_q_kernel      one 128-row tile of queries per block, all its keys in
//                      turn: S and dP (queries on TMEM lanes), dq += dS k
// S and dP are computed in both, 7 products of 128 x 128 x dim per tile pair
// where 5 would do: in exchange every gradient is a sum in a fixed order held
// in TMEM, with no fp32 dq buffer in memory and no atomics on it.
//
// P and dS are rounded to the inputs' 16-bit type for their products (the
// tensor cores take two operands of one type); they go from registers into
// TMEM, which the MMAs read as their A operand, and never to shared memory.
// In f16 both are scaled by powers of two first (P by 2^12, dS by a power that
// puts the bound 2 max|do| max|v| of |dP - D| at 2^15), so that their small
// values stay clear of f16's subnormals and none can overflow.
//
// Roles of a block: warp 0 issues the TMA loads (and zeroes the rows of a
// packed sequence's last tile that belong to its neighbour), warp 1 owns TMEM
// and issues the MMAs, warps 4-19 compute P and dS (four warpgroups, 32 columns
// of a tile each) and the epilogue.  Every wait is bounded (2 s); on a timeout
// the block sets the workspace status bit, stops, waits (bounded) for its
// copies in flight, frees its TMEM and returns.
#include <cuda.h>

#include <algorithm>
#include <cmath>

#include "cba_internal.cuh"
#include "cba_ptx.cuh"
#include "cba_types.cuh"

namespace cba {

namespace {

constexpr uint64_t kAtLimitNs = 2000000000ull;
constexpr int kAtThreads = 640;
constexpr int kAtWarps = 16;                  // that compute P and dS
constexpr int kT = 128;                       // tile rows, of queries and of keys
constexpr uint32_t kBoxBytes = kT * 128u;     // 128 rows x 64 16-bit elements
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 12.f;               // f16: P is held as 2^12 P

// A query- or key-side tensor on the host: bytes between batches, tokens, heads.
struct AtArgs {
    const int *cu_q, *cu_k;      // packed: sequence starts; dense: NULL
    int batch, hq, hkv, group, dim, len_q, len_k;  // packed: the lengths are upper bounds
    long long total_q, total_k;  // packed: tokens
    int causal, tiles, tile_slow;
    float scale;
    const float *lse;
    float *nlse, *ndsum;         // -lse / ln 2 and -D, [head][padded rows] (dense: [batch][head][padded rows])
    long long head_rows;         // padded rows of a head (dense: of a batch's head)
    unsigned *status, *maxima;   // maxima: bits of max |do|^2, max |v|^2 over rows (f16)
    const void *q, *o, *dout, *v;
    void *dq, *dk, *dv;
    long long sq[3], so[3], sdo[3], sv[3], sdq[3], sdk[3], sdv[3];  // batch, token, head (elements)
};

// The sequence b: its first query and key token, its lengths, and the first
// padded row of its statistics.  Values of cu are clamped into the tensors, so
// that wrong ones give wrong results but no access out of bounds.
struct AtSeq {
    long long q0, k0, row0;
    int lq, lk;
};

__device__ __forceinline__ AtSeq at_seq(const AtArgs &a, int b) {
    AtSeq s;
    if (a.cu_q == nullptr) {
        s.q0 = s.k0 = 0;
        s.lq = a.len_q;
        s.lk = a.len_k;
        s.row0 = (long long)b * a.hq * a.head_rows;
        return s;
    }
    const long long qa = min(max((long long)a.cu_q[b], 0LL), a.total_q);
    const long long qb = min(max((long long)a.cu_q[b + 1], qa), a.total_q);
    const long long ka = min(max((long long)a.cu_k[b], 0LL), a.total_k);
    const long long kb = min(max((long long)a.cu_k[b + 1], ka), a.total_k);
    s.q0 = qa;
    s.k0 = ka;
    s.lq = (int)min(qb - qa, (long long)a.len_q);
    s.lk = (int)min(kb - ka, (long long)a.len_k);
    s.row0 = (qa + kT - 1) / kT * kT + (long long)b * kT;
    return s;
}

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

// f16: the power of two by which dS is held, from the rows' largest norms.
__device__ __forceinline__ float ds_scale(const unsigned *maxima) {
    const float b = 2.f * sqrtf(__uint_as_float(__ldcg(maxima))) * sqrtf(__uint_as_float(__ldcg(maxima + 1)));
    if (!(b > 0.f) || !isfinite(b)) return 1.f;
    int e;
    frexpf(b, &e);  // b <= 2^e
    return exp2f((float)min(max(15 - e, -60), 60));
}

// ---- D, lse in base 2, and (f16) the largest row norms of do and v.  One block
// per 128-row tile of one head; 16 (DP = 128) or 8 lanes per row.
template <int DP, bool BF16>
__global__ void __launch_bounds__(256) attn_prep_kernel(const AtArgs a, int q_tiles, int v_blocks) {
    constexpr int LPR = DP / 8;
    const int t = threadIdx.x, lane = t % LPR;
    ptx::griddep_launch_dependents();
    float most = 0.f;
    int which = 0;
    if ((int)blockIdx.x >= v_blocks) {
        const int u = (int)blockIdx.x - v_blocks;
        const int tile = u % q_tiles, h = u / q_tiles % a.hq, b = u / q_tiles / a.hq;
        const AtSeq s = at_seq(a, b);
        if (u == 0 && t == 0 && BF16) *a.status = 0;  // f16: cleared with the maxima before
        if (tile * kT < s.lq) {
            const long long row0 = s.row0 + (long long)h * a.head_rows + tile * kT;
            constexpr int RPP = 256 / LPR, NR = 4;  // rows per pass; rows of a thread in flight
            for (int r0 = t / LPR; r0 < kT; r0 += NR * RPP) {
                uint4 x[NR], y[NR];
                float l[NR];
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    const int i = tile * kT + r0 + j * RPP;
                    x[j] = y[j] = make_uint4(0, 0, 0, 0);
                    l[j] = INFINITY;  // a padding row: P = 0
                    if (i < s.lq && lane * 8 < a.dim) {
                        x[j] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.o) + b * a.so[0] +
                                                                (s.q0 + i) * a.so[1] + h * a.so[2] + lane * 8);
                        y[j] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.dout) + b * a.sdo[0] +
                                                                (s.q0 + i) * a.sdo[1] + h * a.sdo[2] + lane * 8);
                    }
                    if (i < s.lq && lane == 0)
                        l[j] = a.lse[a.cu_q ? (long long)h * a.total_q + s.q0 + i
                                            : ((long long)b * a.hq + h) * a.len_q + i];
                }
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    float d = 0.f, n = 0.f;
                    const uint32_t xs[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                    const uint32_t ys[4] = {y[j].x, y[j].y, y[j].z, y[j].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 p = unpack2<BF16>(xs[e]), q = unpack2<BF16>(ys[e]);
                        d = fmaf(p.x, q.x, fmaf(p.y, q.y, d));
                        if (!BF16) n = fmaf(q.x, q.x, fmaf(q.y, q.y, n));
                    }
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) {
                        d += __shfl_xor_sync(0xffffffffu, d, o);
                        if (!BF16) n += __shfl_xor_sync(0xffffffffu, n, o);
                    }
                    most = fmaxf(most, n);
                    if (lane == 0) {
                        // a row whose keys are all masked has lse = -inf: P = 0 too
                        const long long at = row0 + r0 + j * RPP;
                        a.nlse[at] = l[j] == -INFINITY ? -INFINITY : (BF16 ? 0.f : kPShift) - l[j] * kLog2e;
                        a.ndsum[at] = -d;
                    }
                }
            }
        }
    } else if constexpr (!BF16) {
        // v's rows: [batch][token][head] flattened, strided over the blocks
        which = 1;
        const long long tokens = a.cu_k ? a.total_k : a.len_k;
        const long long rows = (a.cu_k ? 1 : (long long)a.batch) * tokens * a.hkv;
        const long long per = (rows + v_blocks - 1) / v_blocks;
        const long long r1 = min(rows, (blockIdx.x + 1LL) * per);
        for (long long r0 = blockIdx.x * per; r0 < r1; r0 += 256 / LPR) {
            const long long r = r0 + t / LPR;
            float n = 0.f;
            if (r < r1 && lane * 8 < a.dim) {
                const int h = (int)(r % a.hkv);
                const long long tok = r / a.hkv % tokens, b = r / a.hkv / tokens;
                const uint4 x = *reinterpret_cast<const uint4 *>(
                    static_cast<const uint16_t *>(a.v) + b * a.sv[0] + tok * a.sv[1] + h * a.sv[2] + lane * 8);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 p = unpack2<false>(xs[j]);
                    n = fmaf(p.x, p.x, fmaf(p.y, p.y, n));
                }
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            most = fmaxf(most, n);
        }
    }
    if constexpr (!BF16) {  // a maximum does not depend on the order
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        if ((t & 31) == 0) atomicMax(a.maxima + which, __float_as_uint(most));
    }
}

// ---- shared pieces of the two main kernels

template <int NA, int NB>
struct AtBars {
    uint64_t stat;                     // the block's own two tiles
    uint64_t a_full[NA], a_empty[NA];  // the ring used by the accumulating product
    uint64_t b_full[NB], b_empty[NB];
    uint64_t r_full[4], r_empty[4];    // row statistics (kv kernel)
    uint64_t s_full[2], p_ready;
    uint64_t dp_full[2], ds_ready;
    uint64_t fix, acc, drain;
    uint32_t tmem_base;
    int abort_flag;
};

// Loads a 128-row tile (DP / 64 boxes) into `dst`, completing `bar`'s phase.
// Where only `valid` of its rows are the sequence's own (packed sequences; the
// tensor map itself fills rows past a dense one with zeros), the tile arrives on
// the barrier `fix` first and the rows past them are zeroed: they are contracted
// over with P = dS = 0, which an infinity or NaN next door must not meet.
// Called by a whole warp.
template <int DP>
__device__ __forceinline__ bool load_tile(uint32_t dst, const CUtensorMap *tm, long long token,
                                          int head, int b, int valid, bool packed, uint32_t bar,
                                          uint32_t fix, uint32_t &fix_phase, uint32_t extra,
                                          volatile int *abort, unsigned *status) {
    const int lane = threadIdx.x & 31;
    const bool tail = packed && valid < kT;
    if (lane == 0) {
        const uint32_t on = tail ? fix : bar;
        ptx::mbar_arrive_expect_tx(on, DP / 64 * kBoxBytes + (tail ? 0u : extra));
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
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, extra);
    }
    __syncwarp();
    return true;
}

// D[128 x 128] = A[128 x dim] B[128 x dim]^T, both tiles row-major in 64-column
// boxes.  (A descriptor counts 16-byte units: steps are additions to it.)
template <int DP>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t sa, uint32_t sb, int steps,
                                         uint32_t idesc, uint64_t *done, uint64_t *done2 = nullptr) {
    const uint64_t da = ptx::smem_desc(sa, 16, 1024, 2), db = ptx::smem_desc(sb, 16, 1024, 2);
    if (ptx::elect_one()) {
        auto step = [&](int ks) {
            const uint32_t off = ((ks >> 2) * kBoxBytes + (ks & 3) * 32) >> 4;
            ptx::mma_f16(d, da + off, db + off, idesc, ks > 0);
        };
        if (steps == DP / 16) {  // a condition in each step doubles its issue time
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) step(ks);
        } else {
            for (int ks = 0; ks < steps; ++ks) step(ks);
        }
        ptx::mma_commit(ptx::smem_u32(done));
        if (done2) ptx::mma_commit(ptx::smem_u32(done2));
    }
    __syncwarp();
}

// D[128 x DP] (+)= A[128 x 128] B[128 x DP]: A in TMEM (16-bit; the 16 words of
// each 32 columns at ta, ta + 32, ...), B's rows contracted over.
__device__ __forceinline__ void mma_acc(uint32_t d, uint32_t ta, uint32_t sb, uint32_t idesc,
                                        bool accumulate, uint64_t *done) {
    const uint64_t db = ptx::smem_desc(sb, kBoxBytes, 1024, 2);
    if (ptx::elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kT / 16; ++ks)
            ptx::mma_f16_ts(d, ta + (ks >> 1) * 32 + (ks & 1) * 8, db + ks * (2048 >> 4), idesc,
                            accumulate || ks > 0);
        ptx::mma_commit(ptx::smem_u32(done));
    }
    __syncwarp();
}

// 2^(x cs + nlse) of 32 columns with an nlse of their own each.
__device__ __forceinline__ void probabilities(float2 (&p)[16], float cs, const float *nlse) {
    const float2 c2 = make_float2(cs, cs);
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
        const float4 l = *reinterpret_cast<const float4 *>(nlse + 2 * c);
        p[c] = ptx::fma2(p[c], c2, make_float2(l.x, l.y));
        p[c + 1] = ptx::fma2(p[c + 1], c2, make_float2(l.z, l.w));
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) p[c] = make_float2(ptx::ex2(p[c].x), ptx::ex2(p[c].y));
}

__device__ __forceinline__ void tmem_load(uint32_t t, float2 (&v)[16]) {
    float x[32];
    ptx::tmem_ld32(t, x);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] = make_float2(x[2 * c], x[2 * c + 1]);
}

template <bool BF16>
__device__ __forceinline__ void tmem_store(uint32_t t, const float2 (&v)[16]) {
    uint32_t w[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) w[c] = pack2<BF16>(v[c].x, v[c].y);
    ptx::tmem_st16(t, w);
    ptx::tmem_st_wait();
}

// One thread's row of a gradient tile: COLS fp32 columns of TMEM at `ta`,
// scaled, rounded and stored 16 bytes at a time.  Called by whole warps.
template <int COLS, bool BF16>
__device__ __forceinline__ void store_row(uint32_t ta, float scale, bool zero, bool live,
                                          uint16_t *out, int cols) {
#pragma unroll
    for (int c = 0; c < COLS; c += 16) {
        float v[16];
        __syncwarp();  // rows that are not stored skip the code below
        if (!zero) {
            ptx::tmem_ld16(ta + c, v);
            ptx::tmem_ld_wait();
        }
#pragma unroll
        for (int j = 0; j < 16; j += 8)
            if (live && c + j < cols) {
                uint4 w;
                uint32_t *u = &w.x;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    u[e] = zero ? 0u : pack2<BF16>(v[j + 2 * e] * scale, v[j + 2 * e + 1] * scale);
                *reinterpret_cast<uint4 *>(out + c + j) = w;
            }
    }
}

__device__ __forceinline__ void at_init_bars(uint64_t *first, int n, uint32_t count) {
    for (int i = 0; i < n; ++i) ptx::mbar_init(ptx::smem_u32(first + i), count);
}

// The MMA warp's wait for up to three barriers at once, some lanes on each: a wait
// takes ~150 cycles even when its phase is over, in which no MMA is issued.
struct AtWait {
    uint64_t *bar;
    uint32_t parity;
};
__device__ __forceinline__ bool wait_all(AtWait x, AtWait y, AtWait z, volatile int *abort, unsigned *status) {
    const int lane = threadIdx.x & 31;
    const AtWait w = lane < 10 ? x : lane < 20 ? y : z;
    const bool r = ptx::mbar_wait_bounded(ptx::smem_u32(w.bar), w.parity & 1u, abort, status, kAtLimitNs);
    ptx::tc_fence_after();
    return __all_sync(0xffffffffu, r) != 0;
}

// The end of the MMA warp's loop: the accumulators are handed over, and every
// MMA issued has finished before TMEM is released.
template <typename Bars>
__device__ __forceinline__ void finish_mmas(bool ok, Bars &sb, unsigned *status) {
    if (ptx::elect_one()) {
        if (ok) ptx::mma_commit(ptx::smem_u32(&sb.acc));
        else *reinterpret_cast<volatile int *>(&sb.abort_flag) = 1;
        ptx::mma_commit(ptx::smem_u32(&sb.drain));
    }
    __syncwarp();
    int no = 0;
    ptx::mbar_wait_bounded(ptx::smem_u32(&sb.drain), 0, &no, status, kAtLimitNs);
    __syncwarp();
}

// ---- dk, dv: one tile of keys, its queries in turn

// At dim 64 and less TMEM has room for two S tiles: S of the tile after next is
// computed once dv has used P, so that the compute warps find the next S ready.
// At larger dims S(i + 1) overwrites P(i) and the warps wait for it.
template <int DP>
struct Kv {
    static constexpr int NS = DP == 64 ? 2 : 1;               // S buffers
    // stages of q, of do, of the row statistics (dim 128 fills shared memory)
    static constexpr int QST = DP == 64 ? 4 : 3, DOST = DP == 64 ? 4 : 2, RST = DP == 64 ? 4 : 2;
    using Bars = AtBars<QST, DOST>;
    static constexpr uint32_t TILES = (2 + QST + DOST) * (DP / 64) * kBoxBytes;
    static constexpr uint32_t SMEM = TILES + RST * 1024 + sizeof(Bars);
};

template <int DP, bool BF16>
__global__ void __launch_bounds__(kAtThreads, 1)
    attn_kv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                   const AtArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr uint32_t TILE = DP / 64 * kBoxBytes;
    constexpr int NS = Kv<DP>::NS, kQStages = Kv<DP>::QST, kDoStages = Kv<DP>::DOST, kRStages = Kv<DP>::RST;
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t sK = sbase, sV = sK + TILE, sQ = sV + TILE, sDo = sQ + kQStages * TILE;
    float *rows = reinterpret_cast<float *>(smem + Kv<DP>::TILES);
    auto &sb = *reinterpret_cast<typename Kv<DP>::Bars *>(smem + Kv<DP>::TILES + kRStages * 1024);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (sbase & 1023) {  // the swizzled tiles need it
        if (tid == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    if (tid == 0) {
        at_init_bars(&sb.stat, 1, 1);
        at_init_bars(sb.a_full, kQStages, 1);
        at_init_bars(sb.a_empty, kQStages, 1);
        at_init_bars(sb.b_full, kDoStages, 1);
        at_init_bars(sb.b_empty, kDoStages, 1);
        at_init_bars(sb.r_full, kRStages, 1);
        at_init_bars(sb.r_empty, kRStages, kAtWarps);
        at_init_bars(sb.s_full, 2, 1);
        at_init_bars(&sb.p_ready, 1, kAtWarps);
        at_init_bars(sb.dp_full, 2, 1);
        at_init_bars(&sb.ds_ready, 1, kAtWarps);
        at_init_bars(&sb.fix, 3, 1);  // fix, acc, drain
        sb.abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&sb.tmem_base), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sb.tmem_base;
    ptx::griddep_wait();  // the row statistics and the maxima come from the kernel before
    ptx::griddep_launch_dependents();

    // this block's tile
    int u = (int)blockIdx.x, tile, h, b;
    if (a.tile_slow) {
        b = u % a.batch, u /= a.batch;
        h = u % a.hkv, tile = u / a.hkv;
    } else {
        tile = u % a.tiles, u /= a.tiles;
        h = u % a.hkv, b = u / a.hkv;
    }
    const AtSeq s = at_seq(a, b);
    const int k0 = tile * kT;
    const int off = s.lk - s.lq;  // causal: key j is seen by the queries i >= j - off
    const int qt_end = (s.lq + kT - 1) / kT;
    const int qt_begin = a.causal ? min(max(k0 - off, 0) / kT, qt_end) : 0;
    const int nq = qt_end - qt_begin;
    const bool live_tile = k0 < s.lk;
    const int n = live_tile ? nq * a.group : 0;
    const uint32_t tS = tmem, tDp = tmem + NS * 128, tDv = tDp + 128, tDk = tDv + DP;
    volatile int *ab = &sb.abort_flag;
    const int tb = a.cu_q ? 0 : b;  // the tensor maps' batch index

    if (warp == 0) {
        if (n > 0) {
            uint32_t fphase = 0;
            const uint32_t bfix = ptx::smem_u32(&sb.fix);
            if (lane == 0) {
                const uint32_t bar = ptx::smem_u32(&sb.stat);
                ptx::mbar_arrive_expect_tx(bar, 2 * TILE);
#pragma unroll
                for (int j = 0; j < DP / 64; ++j) {
                    ptx::tma_load_4d(sK + j * kBoxBytes, &tk, j * 64, (int)s.k0 + k0, h, tb, bar);
                    ptx::tma_load_4d(sV + j * kBoxBytes, &tv, j * 64, (int)s.k0 + k0, h, tb, bar);
                }
            }
            bool ok = true;
            int it = 0;
            for (; ok && it < n; ++it) {
                const int g = it / nq, q0 = (qt_begin + it - g * nq) * kT, hq = h * a.group + g;
                const int st = it % kQStages, sd = it % kDoStages, sr = it % kRStages;
                if (it >= kQStages)
                    ok = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.a_empty[st]),
                                                (uint32_t)(it / kQStages - 1) & 1u, ab, a.status, kAtLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const int valid = min(kT, s.lq - q0);
                ok = load_tile<DP>(sQ + st * TILE, &tq, s.q0 + q0, hq, tb, valid, a.cu_q != nullptr,
                                   ptx::smem_u32(&sb.a_full[st]), bfix, fphase, 0, ab, a.status);
                if (ok && it >= kRStages)
                    ok = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.r_empty[sr]), (uint32_t)(it / kRStages - 1) & 1u,
                                                ab, a.status, kAtLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    const uint32_t bar = ptx::smem_u32(&sb.r_full[sr]);
                    const long long r0 = s.row0 + (long long)hq * a.head_rows + q0;
                    ptx::mbar_arrive_expect_tx(bar, 2 * kT * 4);
                    ptx::bulk_load(ptx::smem_u32(rows + sr * 2 * kT), a.nlse + r0, kT * 4, bar);
                    ptx::bulk_load(ptx::smem_u32(rows + sr * 2 * kT + kT), a.ndsum + r0, kT * 4, bar);
                }
                if (it >= kDoStages)
                    ok = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.b_empty[sd]),
                                                (uint32_t)(it / kDoStages - 1) & 1u, ab, a.status, kAtLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ok = load_tile<DP>(sDo + sd * TILE, &tdo, s.q0 + q0, hq, tb, valid, a.cu_q != nullptr,
                                   ptx::smem_u32(&sb.b_full[sd]), bfix, fphase, 0, ab, a.status);
            }
            if (!ok) {
                // no copy may be in flight when the block exits: the barriers of
                // the last stages' phases that were begun
                int no = 0;
                ptx::mbar_wait_bounded(ptx::smem_u32(&sb.stat), 0, &no, a.status, kAtLimitNs);
                for (int v = max(0, it - kQStages); v <= it && v < n; ++v)
                    ptx::mbar_wait_bounded(ptx::smem_u32(&sb.a_full[v % kQStages]),
                                           (uint32_t)(v / kQStages) & 1u, &no, a.status, kAtLimitNs / 8);
                for (int v = max(0, it - kDoStages); v <= it && v < n; ++v)
                    ptx::mbar_wait_bounded(ptx::smem_u32(&sb.b_full[v % kDoStages]),
                                           (uint32_t)(v / kDoStages) & 1u, &no, a.status, kAtLimitNs / 8);
                for (int v = max(0, it - kRStages); v <= it && v < n; ++v)
                    ptx::mbar_wait_bounded(ptx::smem_u32(&sb.r_full[v % kRStages]), (uint32_t)(v / kRStages) & 1u, &no,
                                           a.status, kAtLimitNs / 8);
            }
        }
    } else if (warp == 1) {
        // The whole warp walks the loop and one elected lane issues: descriptors and
        // counters are then uniform over the warp, and an MMA takes a few cycles to
        // issue instead of ~100 (more than the 64 that one of 128 columns runs).
        if (n > 0) {
            constexpr uint32_t id_s = ptx::idesc_f16(128, 128, BF16, false);
            constexpr uint32_t id_a = ptx::idesc_f16(128, DP, BF16, true);
            const int steps = (a.dim + 15) / 16;
            auto wait = [&](AtWait x, AtWait y, AtWait z) { return wait_all(x, y, z, ab, a.status); };
            auto mma_s = [&](int it) {
                mma_rows<DP>(tS + it % NS * 128, sK, sQ + (it % kQStages) * TILE, steps, id_s, &sb.s_full[it & 1]);
            };
            auto mma_dp = [&](int it) {
                mma_rows<DP>(tDp, sV, sDo + (it % kDoStages) * TILE, steps, id_s, &sb.dp_full[0]);
            };
            auto full_q = [&](int it) { return AtWait{&sb.a_full[it % kQStages], (uint32_t)(it / kQStages)}; };
            auto full_do = [&](int it) { return AtWait{&sb.b_full[it % kDoStages], (uint32_t)(it / kDoStages)}; };
            const AtWait stat{&sb.stat, 0};
            bool ok = wait(stat, full_q(0), n > 1 ? full_q(NS - 1) : stat);
            if (ok) mma_s(0);
            if (ok && NS == 2 && n > 1) mma_s(1);
            ok = ok && wait(stat, stat, full_do(0));
            if (ok) mma_dp(0);
            for (int it = 0; ok && it < n; ++it) {
                const int ns = it + NS, nd = it + 1;  // the next tiles of S and of dP
                const AtWait pr{&sb.p_ready, (uint32_t)it}, dr{&sb.ds_ready, (uint32_t)it};
                if (!(ok = wait(pr, pr, ns < n ? full_q(ns) : pr))) break;
                mma_acc(tDv, tS + it % NS * 128, sDo + (it % kDoStages) * TILE, id_a, it > 0, &sb.b_empty[it % kDoStages]);
                // S overwrites P, dP overwrites dS: this thread's MMAs run in the order of issue
                if (ns < n) mma_s(ns);
                if (!(ok = wait(dr, dr, nd < n ? full_do(nd) : dr))) break;
                mma_acc(tDk, tDp, sQ + (it % kQStages) * TILE, id_a, it > 0, &sb.a_empty[it % kQStages]);
                if (nd < n) mma_dp(nd);
            }
            finish_mmas(ok, sb, a.status);
        }
    } else if (warp >= 4 && live_tile) {
        const int wg = (warp - 4) >> 2, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const int j = k0 + quarter * 32 + lane;  // this thread's key
        const float cs = a.scale * kLog2e;
        const float sds = BF16 ? 1.f : ds_scale(a.maxima);       // dS is held times sds
        const float pds = BF16 ? 1.f : sds * exp2f(-kPShift);    // from the held P
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            const bool r = ptx::mbar_wait_bounded(ptx::smem_u32(bar), parity & 1u, ab, a.status, kAtLimitNs);
            return __all_sync(0xffffffffu, r);
        };
        for (int it = 0; it < n; ++it) {
            const int g = it / nq, q0 = (qt_begin + it - g * nq) * kT, sr = it % kRStages;
            const float *nl = rows + sr * 2 * kT + wg * 32, *nd = nl + kT;
            float2 p[16];
            if (!(ok = wait(&sb.r_full[sr], (uint32_t)(it / kRStages)) && wait(&sb.s_full[it & 1], (uint32_t)(it / 2)))) break;
            ptx::tc_fence_after();
            const uint32_t ts = tS + it % NS * 128 + lanes + wg * 32;
            tmem_load(ts, p);
            probabilities(p, cs, nl);
            if (a.causal && k0 + kT - 1 > q0 + off) {
                const int first = j - off - q0 - wg * 32;  // columns before it do not see key j
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    if (2 * c < first) p[c].x = 0.f;
                    if (2 * c + 1 < first) p[c].y = 0.f;
                }
            }
            tmem_store<BF16>(ts, p);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.p_ready));
            if (!(ok = wait(&sb.dp_full[0], (uint32_t)it))) break;
            ptx::tc_fence_after();
            float2 x[16];
            tmem_load(tDp + lanes + wg * 32, x);
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
                const float4 d = *reinterpret_cast<const float4 *>(nd + 2 * c);
                x[c] = ptx::mul2(p[c], ptx::add2(x[c], make_float2(d.x, d.y)));
                x[c + 1] = ptx::mul2(p[c + 1], ptx::add2(x[c + 1], make_float2(d.z, d.w)));
                if constexpr (!BF16) {
                    x[c] = ptx::mul2(x[c], make_float2(pds, pds));
                    x[c + 1] = ptx::mul2(x[c + 1], make_float2(pds, pds));
                }
            }
            tmem_store<BF16>(tDp + lanes + wg * 32, x);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(ptx::smem_u32(&sb.ds_ready));
                ptx::mbar_arrive(ptx::smem_u32(&sb.r_empty[sr]));
            }
        }
        if (n > 0 && ok) ok = wait(&sb.acc, 0);
        if (ok) {
            ptx::tc_fence_after();
            // warpgroups 0 and 1 store dv, 2 and 3 dk, half of the columns each
            const bool isk = wg >= 2;
            const int c0 = (wg & 1) * (DP / 2);
            const long long *sg = isk ? a.sdk : a.sdv;
            uint16_t *out = static_cast<uint16_t *>(isk ? a.dk : a.dv) + tb * sg[0] + (s.k0 + j) * sg[1] + h * sg[2] + c0;
            const float f = isk ? a.scale / sds : (BF16 ? 1.f : exp2f(-kPShift));
            store_row<DP / 2, BF16>((isk ? tDk : tDv) + lanes + c0, f, n == 0, j < s.lk, out, a.dim - c0);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ---- dq: one tile of queries, its keys in turn

// The block's q and do rows are A operands of every tile's products, so they lie
// in TMEM (16-bit, 32 or 64 columns each): the products then read one operand
// from shared memory instead of two, whose 128 bytes per cycle are what an MMA
// of 128 columns with both operands there waits for (81 against 55 cycles each,
// dq of 1x8192 h32/8 d128 758 against 628 us).  At dim 128 that leaves room for one dP,
// below it for two, of which one is computed while the other's dS is used.
constexpr int kKStages = 4, kVStages = 3;
using QBars = AtBars<kKStages, kVStages>;

template <int DP>
constexpr uint32_t q_smem_bytes() {
    return (kKStages + kVStages) * (DP / 64) * kBoxBytes + sizeof(QBars);
}

// D[128 x 128] = A[128 x dim] B[128 x dim]^T, A in TMEM.
template <int DP>
__device__ __forceinline__ void mma_rows_ts(uint32_t d, uint32_t ta, uint32_t sb, int steps, uint32_t idesc,
                                            uint64_t *done, uint64_t *done2 = nullptr) {
    const uint64_t db = ptx::smem_desc(sb, 16, 1024, 2);
    if (ptx::elect_one()) {
        auto step = [&](int ks) {
            ptx::mma_f16_ts(d, ta + ks * 8, db + (((ks >> 2) * kBoxBytes + (ks & 3) * 32) >> 4), idesc, ks > 0);
        };
        if (steps == DP / 16) {
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) step(ks);
        } else {
            for (int ks = 0; ks < steps; ++ks) step(ks);
        }
        ptx::mma_commit(ptx::smem_u32(done));
        if (done2) ptx::mma_commit(ptx::smem_u32(done2));
    }
    __syncwarp();
}

// WORDS 32-bit words (pairs of elements) of a row into TMEM; zeros past `dim`.
template <int WORDS>
__device__ __forceinline__ void row_to_tmem(uint32_t t, const uint16_t *row, bool live, int dim, int first) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < WORDS; j += 4) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live && 2 * (first + j) < dim) v = *reinterpret_cast<const uint4 *>(row + 2 * (first + j));
        w[j] = v.x, w[j + 1] = v.y, w[j + 2] = v.z, w[j + 3] = v.w;
    }
    __syncwarp();
    if constexpr (WORDS == 16) ptx::tmem_st16(t + first, w);
    else ptx::tmem_st8(t + first, w);
}

template <int DP, bool BF16>
__global__ void __launch_bounds__(kAtThreads, 1)
    attn_q_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const AtArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr uint32_t TILE = DP / 64 * kBoxBytes;
    const uint32_t sbase = ptx::smem_u32(smem);
    constexpr int NB = DP == 64 ? 2 : 1;  // dP buffers
    const uint32_t sK = sbase, sV = sK + kKStages * TILE;
    QBars &sb = *reinterpret_cast<QBars *>(smem + (kKStages + kVStages) * TILE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (sbase & 1023) {
        if (tid == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    if (tid == 0) {
        at_init_bars(&sb.stat, 1, kAtWarps);  // the rows in TMEM
        at_init_bars(sb.a_full, kKStages, 1);
        at_init_bars(sb.a_empty, kKStages, 1);
        at_init_bars(sb.b_full, kVStages, 1);
        at_init_bars(sb.b_empty, kVStages, 1);
        at_init_bars(sb.s_full, 2, 1);
        at_init_bars(&sb.p_ready, 1, kAtWarps);
        at_init_bars(sb.dp_full, 2, 1);
        at_init_bars(&sb.ds_ready, 1, kAtWarps);
        at_init_bars(&sb.fix, 3, 1);
        sb.abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&sb.tmem_base), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sb.tmem_base;

    int u = (int)blockIdx.x, tile, h, b;
    if (a.tile_slow) {  // causal: the tiles with the most keys first
        b = u % a.batch, u /= a.batch;
        h = u % a.hq, tile = a.tiles - 1 - u / a.hq;
    } else {
        tile = u % a.tiles, u /= a.tiles;
        h = u % a.hq, b = u / a.hq;
    }
    const AtSeq s = at_seq(a, b);
    const int q0 = tile * kT, hk = h / a.group;
    const int off = s.lk - s.lq;
    const bool live_tile = q0 < s.lq;
    int n = live_tile ? (s.lk + kT - 1) / kT : 0;
    if (a.causal && live_tile) {
        const int last = min(q0 + kT, s.lq) - 1 + off;  // the last key any of its queries sees
        n = last < 0 ? 0 : min(n, last / kT + 1);
    }
    const uint32_t tS = tmem, tDp = tmem + 128, tDq = tDp + NB * 128, tQ = tDq + DP, tDo = tQ + DP / 2;
    volatile int *ab = &sb.abort_flag;
    const int tb = a.cu_q ? 0 : b;

    if (warp == 0) {
        if (n > 0) {
            uint32_t fphase = 0;
            const uint32_t bfix = ptx::smem_u32(&sb.fix);
            bool ok = true;
            int it = 0;
            for (; ok && it < n; ++it) {
                const int st = it % kKStages, sv = it % kVStages;
                const int valid = min(kT, s.lk - it * kT);
                if (it >= kKStages)
                    ok = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.a_empty[st]),
                                                (uint32_t)(it / kKStages - 1) & 1u, ab, a.status, kAtLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ok = load_tile<DP>(sK + st * TILE, &tk, s.k0 + it * kT, hk, tb, valid, a.cu_q != nullptr,
                                   ptx::smem_u32(&sb.a_full[st]), bfix, fphase, 0, ab, a.status);
                if (ok && it >= kVStages)
                    ok = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.b_empty[sv]),
                                                (uint32_t)(it / kVStages - 1) & 1u, ab, a.status, kAtLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ok = load_tile<DP>(sV + sv * TILE, &tv, s.k0 + it * kT, hk, tb, valid, a.cu_q != nullptr,
                                   ptx::smem_u32(&sb.b_full[sv]), bfix, fphase, 0, ab, a.status);
            }
            if (!ok) {
                int no = 0;
                for (int v = max(0, it - kKStages); v <= it && v < n; ++v)
                    ptx::mbar_wait_bounded(ptx::smem_u32(&sb.a_full[v % kKStages]),
                                           (uint32_t)(v / kKStages) & 1u, &no, a.status, kAtLimitNs / 8);
                for (int v = max(0, it - kVStages); v <= it && v < n; ++v)
                    ptx::mbar_wait_bounded(ptx::smem_u32(&sb.b_full[v % kVStages]),
                                           (uint32_t)(v / kVStages) & 1u, &no, a.status, kAtLimitNs / 8);
            }
        }
    } else if (warp == 1) {
        // The whole warp walks the loop and one elected lane issues: descriptors and
        // counters are then uniform over the warp, and an MMA takes a few cycles to
        // issue instead of ~100 (more than the 64 that one of 128 columns runs).
        if (n > 0) {
            constexpr uint32_t id_s = ptx::idesc_f16(128, 128, BF16, false);
            constexpr uint32_t id_a = ptx::idesc_f16(128, DP, BF16, true);
            const int steps = (a.dim + 15) / 16;
            auto wait = [&](AtWait x, AtWait y, AtWait z) { return wait_all(x, y, z, ab, a.status); };
            auto mma_s = [&](int it) {
                mma_rows_ts<DP>(tS, tQ, sK + (it % kKStages) * TILE, steps, id_s, &sb.s_full[it & 1]);
            };
            auto mma_dp = [&](int it) {
                mma_rows_ts<DP>(tDp + it % NB * 128, tDo, sV + (it % kVStages) * TILE, steps, id_s,
                                &sb.dp_full[it & 1], &sb.b_empty[it % kVStages]);
            };
            auto full_k = [&](int it) { return AtWait{&sb.a_full[it % kKStages], (uint32_t)(it / kKStages)}; };
            auto full_v = [&](int it) { return AtWait{&sb.b_full[it % kVStages], (uint32_t)(it / kVStages)}; };
            bool ok = wait({&sb.stat, 0}, full_k(0), full_v(0));
            if (ok) mma_s(0);
            if (ok) mma_dp(0);
            for (int it = 0; ok && it < n; ++it) {
                const int nx = it + 1;
                const bool more = nx < n;
                const AtWait pr{&sb.p_ready, (uint32_t)it}, dr{&sb.ds_ready, (uint32_t)it};  // pr: S is in registers
                if (!(ok = wait(pr, more ? full_k(nx) : pr, more && NB == 2 ? full_v(nx) : pr))) break;
                if (more) mma_s(nx);
                if (NB == 2 && more) mma_dp(nx);
                if (!(ok = wait(dr, dr, more && NB == 1 ? full_v(nx) : dr))) break;
                mma_acc(tDq, tDp + it % NB * 128, sK + (it % kKStages) * TILE, id_a, it > 0,
                        &sb.a_empty[it % kKStages]);
                // with one buffer dP overwrites dS: this thread's MMAs run in the order of issue
                if (NB == 1 && more) mma_dp(nx);
            }
            finish_mmas(ok, sb, a.status);
        }
    } else if (warp >= 4 && live_tile) {
        const int wg = (warp - 4) >> 2, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const int r = quarter * 32 + lane, i = q0 + r;  // this thread's query
        const long long row = s.row0 + (long long)h * a.head_rows + i;
        const float nl = __ldcg(a.nlse + row), nd = __ldcg(a.ndsum + row);
        const float cs = a.scale * kLog2e;
        const float sds = BF16 ? 1.f : ds_scale(a.maxima);
        const float pds = BF16 ? 1.f : sds * exp2f(-kPShift);
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            const bool w = ptx::mbar_wait_bounded(ptx::smem_u32(bar), parity & 1u, ab, a.status, kAtLimitNs);
            return __all_sync(0xffffffffu, w);
        };
        if (n > 0) {
            constexpr int WORDS = DP / 8;  // of each tensor's DP / 2 words, per warpgroup
            const uint16_t *qrow = static_cast<const uint16_t *>(a.q) + tb * a.sq[0] + (s.q0 + i) * a.sq[1] + h * a.sq[2];
            const uint16_t *drow = static_cast<const uint16_t *>(a.dout) + tb * a.sdo[0] + (s.q0 + i) * a.sdo[1] + h * a.sdo[2];
            row_to_tmem<WORDS>(tQ + lanes, qrow, i < s.lq, a.dim, wg * WORDS);
            row_to_tmem<WORDS>(tDo + lanes, drow, i < s.lq, a.dim, wg * WORDS);
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.stat));
        }
        for (int it = 0; it < n; ++it) {
            float2 p[16];
            if (!(ok = wait(&sb.s_full[it & 1], (uint32_t)(it / 2)))) break;
            ptx::tc_fence_after();
            tmem_load(tS + lanes + wg * 32, p);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.p_ready));
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                p[c] = ptx::fma2(p[c], make_float2(cs, cs), make_float2(nl, nl));
                p[c] = make_float2(ptx::ex2(p[c].x), ptx::ex2(p[c].y));
            }
            const int kb = it * kT;
            if (kb + kT > s.lk || (a.causal && kb + kT - 1 > q0 + off)) {
                int lim = s.lk - kb;  // columns from it on are masked
                if (a.causal) lim = min(lim, i + off - kb + 1);
                lim -= wg * 32;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    if (2 * c >= lim) p[c].x = 0.f;
                    if (2 * c + 1 >= lim) p[c].y = 0.f;
                }
            }
            if (!(ok = wait(&sb.dp_full[it & 1], (uint32_t)(it / 2)))) break;
            ptx::tc_fence_after();
            const uint32_t td = tDp + it % NB * 128 + lanes + wg * 32;
            float2 x[16];
            tmem_load(td, x);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                x[c] = ptx::mul2(p[c], ptx::add2(x[c], make_float2(nd, nd)));
                if constexpr (!BF16) x[c] = ptx::mul2(x[c], make_float2(pds, pds));
            }
            tmem_store<BF16>(td, x);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.ds_ready));
        }
        if (n > 0 && ok) ok = wait(&sb.acc, 0);
        if (ok) {
            ptx::tc_fence_after();
            // each warpgroup stores a quarter of the columns
            const int c0 = wg * (DP / 4);
            uint16_t *out = static_cast<uint16_t *>(a.dq) + tb * a.sdq[0] + (s.q0 + i) * a.sdq[1] + h * a.sdq[2] + c0;
            store_row<DP / 4, BF16>(tDq + lanes + c0, a.scale / sds, n == 0, i < s.lq, out, a.dim - c0);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
    // the launch before this one has written dk and dv: this grid completes
    // after it (its own reads depend only on what that one waited for)
    ptx::griddep_wait();
}

// ---- host side

struct AtPlan {
    int dp, q_tiles, k_tiles;
    long long head_rows;   // padded rows of one head
    size_t off_nlse, off_ndsum, total;
};

void fill_strides(const cba_attn_strides_t &s, int heads, int dim, long long len, long long *out) {
    if (s.batch == 0 && s.token == 0 && s.head == 0) {
        out[0] = len * heads * dim;
        out[1] = (long long)heads * dim;
        out[2] = dim;
    } else {
        out[0] = s.batch;
        out[1] = s.token;
        out[2] = s.head;
    }
}

int check_attn(const cba_attention_desc_t *d, AtPlan *p) {
    if (!d || d->batch < 1 || d->heads_q < 1 || d->heads_kv < 1 || d->dim < 1 || d->len_q < 0 ||
        d->len_k < 0 || d->heads_q % d->heads_kv != 0)
        return CBA_ERR_ARG;
    if (!dtype_ok(d->type) || (d->causal != 0 && d->causal != 1) || (d->packed != 0 && d->packed != 1) ||
        !std::isfinite(d->scale))
        return CBA_ERR_ARG;
    if (d->packed && (d->total_q < 0 || d->total_k < 0)) return CBA_ERR_ARG;
    if (d->type == CBA_F32 || d->dim > 128 || d->dim % 8 != 0) return CBA_ERR_UNSUPPORTED;
    const long long lim = 1LL << 30;
    if (d->len_q > lim || d->len_k > lim || (d->packed && (d->total_q > lim || d->total_k > lim)))
        return CBA_ERR_UNSUPPORTED;
    const cba_attn_strides_t *ss[] = {&d->q, &d->k, &d->v, &d->o, &d->dout, &d->dq, &d->dk, &d->dv};
    for (int i = 0; i < 8; ++i) {
        const auto *s = ss[i];
        if (s->batch == 0 && s->token == 0 && s->head == 0) continue;  // contiguous
        const bool kside = s == &d->k || s == &d->v || s == &d->dk || s == &d->dv;
        const long long v[] = {s->batch, s->token, s->head};
        const long long n[] = {d->packed ? 1 : d->batch,
                               d->packed ? (kside ? d->total_k : d->total_q) : (kside ? d->len_k : d->len_q),
                               kside ? d->heads_kv : d->heads_q};
        for (int j = 0; j < 3; ++j) {
            const long long x = v[j];
            if (x < 0 || (n[j] > 1 && x < d->dim)) return CBA_ERR_ARG;
            if (x % 8 != 0) return CBA_ERR_ALIGN;
            if (x >= (1LL << 38)) return CBA_ERR_UNSUPPORTED;
        }
    }
    p->dp = d->dim <= 64 ? 64 : 128;
    p->q_tiles = (d->len_q + kT - 1) / kT;
    p->k_tiles = (d->len_k + kT - 1) / kT;
    long long rows;
    if (d->packed) {
        p->head_rows = (d->total_q + kT - 1) / kT * kT + (long long)kT * (d->batch + 1);
        rows = p->head_rows * d->heads_q;
    } else {
        p->head_rows = (long long)p->q_tiles * kT;
        rows = p->head_rows * d->heads_q * d->batch;
    }
    const long long grid = std::max((long long)p->k_tiles * d->heads_kv, (long long)p->q_tiles * d->heads_q);
    if (grid * d->batch >= (1LL << 30) || rows >= (1LL << 40)) return CBA_ERR_UNSUPPORTED;
    p->off_nlse = 256;
    p->off_ndsum = p->off_nlse + ((size_t)rows * 4 + 255) / 256 * 256;
    p->total = p->off_ndsum + ((size_t)rows * 4 + 255) / 256 * 256;
    return CBA_OK;
}

// The map of one tensor: (dim, token, head, batch), boxes of 128 tokens x 64.
bool attn_map(CUtensorMap *m, const void *base, const cba_attention_desc_t &d, int heads, long long tokens,
              const long long *st) {
    const uint64_t dims[4] = {(uint64_t)d.dim, (uint64_t)tokens, (uint64_t)heads, (uint64_t)(d.packed ? 1 : d.batch)};
    uint64_t strides[3] = {(uint64_t)st[1] * 2, (uint64_t)st[2] * 2, (uint64_t)st[0] * 2};
    for (int i = 0; i < 3; ++i)  // an axis of one index has no stride of its own
        if (dims[i + 1] == 1) strides[i] = 16;
    const uint32_t box[4] = {64, kT, 1, 1};
    return tma_encode_16(m, base, d.type == CBA_BF16, 4, dims, strides, box);
}

template <int DP, bool BF16>
cudaError_t attn_launch(const cba_attention_desc_t &d, const AtPlan &p, AtArgs a, const CUtensorMap *tm,
                        cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (!BF16) e = cudaMemsetAsync(a.status, 0, 256, st);  // the status word and the maxima
    if (e != cudaSuccess) return e;
    // f16: the blocks that look for v's largest row
    const int vb = BF16 ? 0 : kNumSMs;
    const unsigned qgrid = (unsigned)((long long)p.q_tiles * d.heads_q * d.batch);
    attn_prep_kernel<DP, BF16><<<std::max(1u, qgrid) + vb, 256, 0, st>>>(a, std::max(1, p.q_tiles), vb);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attn_kv_kernel<DP, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Kv<DP>::SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attn_q_kernel<DP, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)q_smem_bytes<DP>());
    if (e != cudaSuccess) return e;
    if (p.k_tiles > 0) {
        a.tiles = p.k_tiles;
        e = launch_pdl(attn_kv_kernel<DP, BF16>, dim3((unsigned)((long long)p.k_tiles * d.heads_kv * d.batch)),
                       dim3(kAtThreads), Kv<DP>::SMEM, st, tm[0], tm[1], tm[2], tm[3], a);
        if (e != cudaSuccess) return e;
    }
    if (p.q_tiles > 0) {
        a.tiles = p.q_tiles;
        // without keys there is no launch between this one and the preparation
        if (p.k_tiles > 0)
            e = launch_pdl(attn_q_kernel<DP, BF16>, dim3(qgrid), dim3(kAtThreads), q_smem_bytes<DP>(), st, tm[1],
                           tm[2], a);
        else
            attn_q_kernel<DP, BF16><<<qgrid, kAtThreads, q_smem_bytes<DP>(), st>>>(tm[1], tm[2], a);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

}  // namespace

}  // namespace cba

using namespace cba;

extern "C" {

size_t cba_attention_workspace_bytes(const cba_attention_desc_t *d) {
    AtPlan p;
    return check_attn(d, &p) == CBA_OK ? p.total : 0;
}

int cba_attention_backward(const cba_attention_desc_t *d, const void *q, const void *k, const void *v,
                           const void *o, const float *lse, const void *dout, const int *cu_q,
                           const int *cu_k, void *dq, void *dk, void *dv, void *workspace,
                           size_t workspace_bytes, void *stream) {
    AtPlan p;
    const int rc = check_attn(d, &p);
    if (rc != CBA_OK) return rc;
    const long long tq = d->packed ? d->total_q : d->len_q, tk = d->packed ? d->total_k : d->len_k;
    if (tq > 0 && (!q || !o || !lse || !dout || !dq)) return CBA_ERR_ARG;
    if (tk > 0 && (!k || !v || !dk || !dv)) return CBA_ERR_ARG;
    if (d->packed ? (!cu_q || !cu_k) : (cu_q || cu_k)) return CBA_ERR_ARG;
    const void *ptrs[] = {q, k, v, o, dout, dq, dk, dv};
    for (const void *x : ptrs)
        if (!aligned_to(x, 16)) return CBA_ERR_ALIGN;
    if (!aligned_to(lse, 4) || !aligned_to(cu_q, 4) || !aligned_to(cu_k, 4)) return CBA_ERR_ALIGN;
    if (!workspace || workspace_bytes < p.total) return CBA_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return CBA_ERR_ALIGN;

    AtArgs a{};
    a.cu_q = cu_q; a.cu_k = cu_k;
    a.batch = d->batch; a.hq = d->heads_q; a.hkv = d->heads_kv; a.group = d->heads_q / d->heads_kv;
    a.dim = d->dim; a.len_q = d->len_q; a.len_k = d->len_k;
    a.total_q = d->total_q; a.total_k = d->total_k;
    a.causal = d->causal; a.tile_slow = d->causal; a.scale = d->scale;
    a.lse = lse;
    a.status = static_cast<unsigned *>(workspace);
    a.maxima = a.status + 4;
    a.nlse = ws_at<float>(workspace, p.off_nlse);
    a.ndsum = ws_at<float>(workspace, p.off_ndsum);
    a.head_rows = p.head_rows;
    a.q = q; a.o = o; a.dout = dout; a.v = v; a.dq = dq; a.dk = dk; a.dv = dv;
    long long sk[3];
    fill_strides(d->q, d->heads_q, d->dim, tq, a.sq);
    fill_strides(d->k, d->heads_kv, d->dim, tk, sk);
    fill_strides(d->v, d->heads_kv, d->dim, tk, a.sv);
    fill_strides(d->o, d->heads_q, d->dim, tq, a.so);
    fill_strides(d->dout, d->heads_q, d->dim, tq, a.sdo);
    fill_strides(d->dq, d->heads_q, d->dim, tq, a.sdq);
    fill_strides(d->dk, d->heads_kv, d->dim, tk, a.sdk);
    fill_strides(d->dv, d->heads_kv, d->dim, tk, a.sdv);
    // without queries (or keys) the main kernels load nothing of them
    CUtensorMap tm[4] = {};
    if (tq > 0 && tk > 0 &&
        (!attn_map(&tm[0], q, *d, d->heads_q, tq, a.sq) || !attn_map(&tm[1], k, *d, d->heads_kv, tk, sk) ||
         !attn_map(&tm[2], v, *d, d->heads_kv, tk, a.sv) || !attn_map(&tm[3], dout, *d, d->heads_q, tq, a.sdo)))
        return CBA_ERR_UNSUPPORTED;
    cudaGetLastError();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = select_device_of(workspace);
    if (e == cudaSuccess) {
        const bool bf = d->type == CBA_BF16;
        if (p.dp == 64) e = bf ? attn_launch<64, true>(*d, p, a, tm, st) : attn_launch<64, false>(*d, p, a, tm, st);
        else e = bf ? attn_launch<128, true>(*d, p, a, tm, st) : attn_launch<128, false>(*d, p, a, tm, st);
    }
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

}  // extern "C"
