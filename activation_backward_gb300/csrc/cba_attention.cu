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
// values stay clear of f16's subnormals and none can overflow.  The maxima are
// those of a sequence's rows under one key/value head, rows with infinities or
// NaN left out: neither another sequence's values nor an infinity among one's own
// costs the others bits.
//
// Measured (us; launches overlap, so a call takes less than their sum; rates count
// the formulas' 5 products):
//   8192 tokens, 32/8 heads of 128, causal, bf16   27 + 654 + 504, call 1125 after a pause and
//       1216 to 1242 where calls follow each other: 1.1 PFLOP/s, 1.56 with the 7 products that
//       run (1.7 after a pause).  The tensor cores bound it, at the clock that the power limit
//       leaves them
//   9 documents of 8192 tokens, 16/4 heads of 128  16 + 104 + 92, call 169: the longest tile
//   32 x 676 tokens, 8 heads of 64, f16            17 + 95 + 85, call 189: the compute warps,
//       whose two halves of a step (P, then dS) take 850 and 1000 cycles of latency; the tensor
//       cores are active for 38% of the cycles, the issue slots taken for 47%
//   2 x 169 tokens, 8 heads of 64, bf16            call 12.3 to 13.2: three launches, a tile or two each
// The preparation reads o and do at 5.1 TB/s in the first case.
//
// Roles of a block: warp 0 issues the TMA loads (and zeroes the rows of a
// packed sequence's last tile that belong to its neighbour) and hands out the
// work, warp 1 owns TMEM and issues the MMAs, warps 4-19 compute P and dS (four
// warpgroups, 32 columns of a tile each) and the epilogue.  Every wait is bounded (2 s); on a timeout
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
// Registers per thread: 96 at launch (of 640 threads), then moved from the load
// and MMA warps' warpgroup to the four that compute.
constexpr int kCtlRegs = 64, kCompRegs = 104;
static_assert(128 * kCtlRegs + 512 * kCompRegs <= 640 * 96);
constexpr int kT = 128;                       // tile rows, of queries and of keys
constexpr uint32_t kBoxBytes = kT * 128u;     // 128 rows x 64 16-bit elements
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 12.f;               // f16: P is held as 2^12 P

// What the kernels of a call get; strides in elements.
struct AtArgs {
    const int *cu_q, *cu_k;      // packed: sequence starts; dense: NULL
    int batch, hq, hkv, group, dim, len_q, len_k;  // packed: the lengths are upper bounds
    long long total_q, total_k;  // packed: tokens
    int causal, tiles, tile_slow;
    float scale;
    const float *lse;
    float *nlse, *ndsum;         // -lse / ln 2 and -D, [head][padded rows] (dense: [batch][head][padded rows])
    long long head_rows;         // padded rows of a head (dense: of a batch's head)
    unsigned *status;
    unsigned *maxima;            // f16: bits of max |do|^2, then of max |v|^2, over the finite rows
                                 // of each sequence and key/value head ([2][batch][hkv])
    unsigned *next;              // work items handed out, of the two main kernels
    int items;                   // this launch's
    int q_slots, k_slots;        // packed with loose bounds: see find_tile; 0: tiles are counted up to the bounds
    int chunk, chunks;           // steps of an item at most; items per tile at most
    int cnt_kv, cnt_q;           // tiles that have an arrival counter
    unsigned *arrived;           // this launch's counters (kv's lie before q's)
    float *part;                 // fp32 tiles of the items of a tile
    const void *o, *dout, *v;
    void *dq, *dk, *dv;
    long long so[3], sdo[3], sv[3], sdq[3], sdk[3], sdv[3];  // batch, token, head
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

// Tiles of packed sequences whose lengths are much below their bounds are numbered
// by the tokens instead: tile t of sequence b has the slot cu[b] / 128 + b + t.  The
// next sequence's first slot lies past its last, so there are total / 128 + batch of
// them at most, of which one per sequence may stand for no tile.
__device__ __forceinline__ long long slot_of(const int *cu, long long total, int b) {
    return min(max((long long)cu[b], 0LL), total) / kT + b;
}
// The sequence and tile of a slot, searched by a converged warp, 32 sequences at a
// time.  (A slot without a tile, or before the first sequence, gives one out of
// range; values of cu that fall give some in-range sequence.)
__device__ __forceinline__ void find_tile(const int *cu, long long total, int batch, int slot, int &b, int &tile) {
    int lo = 0, n = batch;  // the sequence is one of lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32, m = lo + ((int)(threadIdx.x & 31) + 1) * step;
        const bool past = m < lo + n && slot_of(cu, total, m) <= slot;
        const int k = __popc(__ballot_sync(0xffffffffu, past)) * step;
        n = min(step, n - k);
        lo += k;
    }
    b = lo;
    tile = slot - (int)slot_of(cu, total, lo);
}
// Slots up to the last sequence's end.
__device__ __forceinline__ int used_slots(const int *cu, long long total, int batch) {
    return (int)slot_of(cu, total, batch);
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

// f16: the power of two by which dS of sequence b under key/value head h is held:
// with its largest |do|^2 = x and |v|^2 = y (of finite rows: below 2^40, and above
// 2^-48 where they are not 0), the one that brings 2 sqrt(x y) to 2^14 .. 2^15.
__device__ __forceinline__ float ds_scale(const AtArgs &a, int b, int h) {
    const long long at = (long long)b * a.hkv + h;
    const float x = __uint_as_float(__ldcg(a.maxima + at)),
                y = __uint_as_float(__ldcg(a.maxima + (long long)a.batch * a.hkv + at));
    const float m = 4.f * x * y;
    if (!(m > 0.f)) return 1.f;
    const int e = (__float_as_int(m) >> 23) - 126;  // m < 2^e
    return __int_as_float((127 + min(max(15 - ((e + 1) >> 1), -60), 60)) << 23);
}

// ---- D, lse in base 2, and (f16) the largest row norms of do and v.  One block
// per 128-row tile of one head; 16 (DP = 128) or 8 lanes per row, four rows of a
// thread in flight.  Bound by memory: 134 MB of o and do in 26 us, 5.1 TB/s; with
// v for f16 66 MB in 17 us.
template <int DP, bool BF16, bool SLOTS>
__global__ void __launch_bounds__(256) attn_prep_kernel(const AtArgs a, int q_tiles, int k_tiles, int v_blocks) {
    constexpr int LPR = DP / 8;
    const int t = threadIdx.x, lane = t % LPR;
    ptx::griddep_launch_dependents();
    float most = 0.f;    // |row|^2 of the block's finite rows
    long long slot = 0;  // of its maximum
    if ((int)blockIdx.x >= v_blocks) {
        const int u = (int)blockIdx.x - v_blocks;
        int tile, h, b;
        if (SLOTS && a.q_slots) {
            h = u % a.hq;
            find_tile(a.cu_q, a.total_q, a.batch, u / a.hq, b, tile);
        } else {
            tile = u % q_tiles, h = u / q_tiles % a.hq, b = u / q_tiles / a.hq;
        }
        const AtSeq s = at_seq(a, b);
        slot = (long long)b * a.hkv + h / a.group;
        if (u == 0 && t == 0) {
            if (BF16) *a.status = 0;  // f16: cleared with the maxima before
            a.next[0] = a.next[1] = 0;
        }
        if (u == 0)
            for (int i = t; i < a.cnt_kv + a.cnt_q; i += 256) a.arrived[i] = 0;
        if (tile >= 0 && tile < (s.lq + kT - 1) / kT) {
            const long long row0 = s.row0 + (long long)h * a.head_rows + tile * kT;
            const int unseen = a.causal ? s.lq - s.lk : s.lk == 0 ? s.lq : 0;  // rows before it see no key
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
                        l[j] = i < unseen ? -INFINITY
                                          : a.lse[a.cu_q ? (long long)h * a.total_q + s.q0 + i
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
                    if (lane == 0) {
                        // a row that sees no key, by the mask or (lse = -inf) the caller's own: P = 0 and D = 0
                        // whatever the forward left in its o and lse (a softmax over nothing is NaN)
                        const bool none = l[j] == -INFINITY;
                        const long long at = row0 + r0 + j * RPP;
                        a.nlse[at] = none ? -INFINITY : (BF16 ? 0.f : kPShift) - l[j] * kLog2e;
                        a.ndsum[at] = none ? 0.f : -d;
                        if (!BF16 && !none && n < INFINITY) most = fmaxf(most, n);
                    }
                }
            }
        }
    } else if constexpr (!BF16) {
        // v, a block per 128 keys of one head
        const int u = (int)blockIdx.x;
        int tile, h, b;
        if (SLOTS && a.k_slots) {
            h = u % a.hkv;
            find_tile(a.cu_k, a.total_k, a.batch, u / a.hkv, b, tile);
        } else {
            tile = u % k_tiles, h = u / k_tiles % a.hkv, b = u / k_tiles / a.hkv;
        }
        const AtSeq s = at_seq(a, b);
        slot = (long long)(a.batch + b) * a.hkv + h;
        const uint16_t *v = static_cast<const uint16_t *>(a.v) + b * a.sv[0] + h * a.sv[2] + lane * 8;
        constexpr int RPP = 256 / LPR, NR = 4;
        if (tile >= 0 && tile < (s.lk + kT - 1) / kT)
            for (int r0 = t / LPR; r0 < kT; r0 += NR * RPP) {
                uint4 x[NR];
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    const int i = tile * kT + r0 + j * RPP;
                    x[j] = make_uint4(0, 0, 0, 0);
                    if (i < s.lk && lane * 8 < a.dim) x[j] = *reinterpret_cast<const uint4 *>(v + (s.k0 + i) * a.sv[1]);
                }
#pragma unroll
                for (int j = 0; j < NR; ++j) {
                    float n = 0.f;
                    const uint32_t xs[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 p = unpack2<false>(xs[e]);
                        n = fmaf(p.x, p.x, fmaf(p.y, p.y, n));
                    }
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
                    if (n < INFINITY) most = fmaxf(most, n);
                }
            }
    }
    if constexpr (!BF16) {  // a maximum does not depend on the order
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        __shared__ float warps[8];
        if ((t & 31) == 0) warps[t >> 5] = most;
        __syncthreads();
        if (t == 0) {
#pragma unroll
            for (int i = 1; i < 8; ++i) most = fmaxf(most, warps[i]);
            // many blocks on one word: most of them see that it is no less already
            if (__float_as_uint(most) > __ldcg(a.maxima + slot)) atomicMax(a.maxima + slot, __float_as_uint(most));
        }
    }
}

// ---- shared pieces of the two main kernels

// A barrier that the compute warps arrive on has two instances, used in turn,
// where a warp can be a tile ahead of another (the next S or dP is computed
// early): its arrival for the next tile must not count for this one.
template <int NA, int NB>
struct AtBars {
    uint64_t stat[2];                  // the item's own two tiles
    uint64_t a_full[NA], a_empty[NA];  // the ring used by the accumulating product
    uint64_t b_full[NB], b_empty[NB];
    uint64_t r_full[4], r_empty[4];    // row statistics (kv kernel)
    uint64_t s_full[2], p_ready[2];
    uint64_t dp_full[2], ds_ready[2];
    uint64_t fix, drain, acc, stat_empty[2];
    uint64_t i_full[2], i_empty[2];    // work items handed out
    uint64_t join;                     // the compute warps, around an arrival
    // The results of the items in turn have passed through q's ring (kv kernel, dim 128).  Two, as
    // the load warp may wait for an item's when the next item's are through as well.
    uint64_t staged[2];
    int last;
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

// D[128 x 128] = A[128 x dim] B[128 x dim]^T, both tiles row-major in 64-column
// boxes.  (A descriptor counts 16-byte units: steps are additions to it.)
template <int DP>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t sa, uint32_t sb, int steps,
                                         uint32_t idesc, uint64_t *done, uint64_t *done2 = nullptr) {
    const ptx::Desc da = ptx::desc_of(sa, 16, 1024, 2), db = ptx::desc_of(sb, 16, 1024, 2);
    if (ptx::elect_one()) {
        auto step = [&](int ks) {
            const uint32_t off = ((ks >> 2) * kBoxBytes + (ks & 3) * 32) >> 4;
            ptx::mma_f16(d, da, off, db, off, idesc, ks > 0);
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
    const ptx::Desc db = ptx::desc_of(sb, kBoxBytes, 1024, 2);
    if (ptx::elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kT / 16; ++ks)
            ptx::mma_f16_ts(d, ta + (ks >> 1) * 32 + (ks & 1) * 8, db, ks * (2048 >> 4), idesc,
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

// 32 rows x COLS columns of a warp's accumulators, stored through 2 KB of shared
// memory of its own, 32 columns at a time: row = lane, its 16-byte chunk j at
// j ^ ((row >> 1) & 3); then four lanes store a row's 64 bytes (16 bytes of 32 rows
// at a time, as store_row does, take 8300 cycles of an item at dim 128).
template <int COLS, bool BF16>
__device__ __forceinline__ void store_rows_staged(uint32_t ta, float scale, int live, uint16_t *out,
                                                  long long stride, int cols, uint8_t *stage) {
    const int lane = threadIdx.x & 31;
    auto slot = [&](int r, int j) { return stage + r * 64 + ((j ^ ((r >> 1) & 3)) << 4); };
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
        float v[32];
        ptx::tmem_ld32(ta + c, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 w;
            w.x = pack2<BF16>(v[8 * j] * scale, v[8 * j + 1] * scale);
            w.y = pack2<BF16>(v[8 * j + 2] * scale, v[8 * j + 3] * scale);
            w.z = pack2<BF16>(v[8 * j + 4] * scale, v[8 * j + 5] * scale);
            w.w = pack2<BF16>(v[8 * j + 6] * scale, v[8 * j + 7] * scale);
            *reinterpret_cast<uint4 *>(slot(lane, j)) = w;
        }
        __syncwarp();
        const int j = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2);
            if (r < live && c + j * 8 < cols)
                *reinterpret_cast<uint4 *>(out + r * stride + c + j * 8) = *reinterpret_cast<const uint4 *>(slot(r, j));
        }
        __syncwarp();
    }
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

// The end of the MMA warp's work: every MMA issued has finished before TMEM is
// released.
template <typename Bars>
__device__ __forceinline__ void finish_mmas(bool ok, Bars &sb, unsigned *status) {
    if (ptx::elect_one()) {
        if (!ok) *reinterpret_cast<volatile int *>(&sb.abort_flag) = 1;
        ptx::mma_commit(ptx::smem_u32(&sb.drain));
    }
    __syncwarp();
    int no = 0;
    ptx::mbar_wait_bounded(ptx::smem_u32(&sb.drain), 0, &no, status, kAtLimitNs);
    __syncwarp();
}

// ---- work items

// Both main kernels are persistent, one block per SM: a block takes its first
// item by its index and the others from a counter, in the order of falling work
// where the mask makes it fall.  The load warp takes the next item when it has
// begun the last loads of one (earlier, and the items would be dealt out before
// it is known who is done first); the loads and first products of the next item
// then run under the last products and the epilogue of the one before (of
// 32x676 h8 d64, six query tiles per item, more than half of a block's life was
// its start and end when it had one item).

// Few tiles with many steps each are cut into items of at most `chunk` steps.
// Such an item writes its fp32 sums to memory and arrives on the tile's counter;
// the one that arrives last adds all of them in the order of the steps, so the
// result does not depend on who that is.

// Load warp: hands item number k to the other warps (tile < 0: there is none).
template <typename Item, typename Bars>
__device__ __forceinline__ bool hand_out(const AtArgs &a, int k, const Item &w, Item *slots, Bars &sb, bool &ok) {
    if (k >= 2)
        ok = ok && ptx::mbar_wait_bounded(ptx::smem_u32(&sb.i_empty[k & 1]), (uint32_t)(k / 2 - 1) & 1u,
                                          &sb.abort_flag, a.status, kAtLimitNs);
    ok = __all_sync(0xffffffffu, ok) != 0;
    if (!ok) return false;
    if ((threadIdx.x & 31) == 0) {
        slots[k & 1] = w;
        ptx::mbar_arrive(ptx::smem_u32(&sb.i_full[k & 1]));
    }
    __syncwarp();
    return w.tile >= 0;
}
__device__ __forceinline__ int next_item(unsigned *next) {
    unsigned v = 0;
    if ((threadIdx.x & 31) == 0) v = atomicAdd(next, 1u);
    return (int)gridDim.x + (int)__shfl_sync(0xffffffffu, v, 0);
}

// The k-th item of this block, or NULL past the last (or on a timeout); it stays
// until all readers are done with it.  Called by whole warps.
template <typename Item, typename Bars>
__device__ __forceinline__ const Item *take_item(const AtArgs &a, int k, const Item *slots, Bars &sb, bool &ok) {
    ok = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.i_full[k & 1]), (uint32_t)(k / 2) & 1u, &sb.abort_flag, a.status,
                                kAtLimitNs);
    ok = __all_sync(0xffffffffu, ok) != 0;
    return ok && slots[k & 1].tile >= 0 ? slots + (k & 1) : nullptr;
}
template <typename Bars>
__device__ __forceinline__ void done_item(int k, Bars &sb) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.i_empty[k & 1]));
}
constexpr int kItemReaders = 1 + kAtWarps;  // the MMA and compute warps

// The first step and the number of steps of a tile's item c, of n in all; `used`:
// the items that the tile is cut into.
__device__ __forceinline__ void cut(const AtArgs &a, int c, int &it0, int &n, int &used) {
    used = 1;
    it0 = 0;
    if (a.chunks == 1) return;
    used = max(1, (n + a.chunk - 1) / a.chunk);
    const int each = (n + used - 1) / used;
    it0 = c * each;
    n = min(each, n - it0);
}

// The compute warps' arrival on a tile's counter with their sums in memory.  True
// in all of them if theirs was the last of `used` (ok: false on a timeout).
template <typename Bars>
__device__ __forceinline__ bool arrive_last(const AtArgs &a, int tile, int used, Bars &sb, uint32_t &phase, bool &ok) {
    auto meet = [&]() {
        __threadfence();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.join));
        const bool r = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.join), phase, &sb.abort_flag, a.status, kAtLimitNs);
        phase ^= 1;
        return ok = __all_sync(0xffffffffu, r) != 0;
    };
    if (!meet()) return false;
    if (threadIdx.x == 128)
        *const_cast<volatile int *>(&sb.last) = atomicAdd(a.arrived + tile, 1u) + 1 == (unsigned)used;
    if (!meet()) return false;
    return *const_cast<volatile int *>(&sb.last) != 0;
}

// COLS columns of a thread's row of accumulators in memory: 16 bytes of 32 rows
// side by side.  `at`: the item's sums plus the thread's row.
template <int COLS>
__device__ __forceinline__ void sums_to_memory(uint32_t ta, float4 *at) {
#pragma unroll
    for (int c = 0; c < COLS; c += 16) {
        float v[16];
        ptx::tmem_ld16(ta + c, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; j += 4)
            __stcg(at + (c + j) / 4 * kT, make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
    }
}
// The same of `used` items, `stride` float4 apart, added, scaled, rounded and
// stored 16 bytes at a time.
template <int COLS, bool BF16>
__device__ __forceinline__ void store_sums(const float4 *at, int used, long long stride, float scale, bool live,
                                           uint16_t *out, int cols) {
    constexpr int C = 16;  // columns at a time
    if (!live) return;
    for (int c = 0; c < COLS && c < cols; c += C) {
        float4 x[C / 4];
#pragma unroll
        for (int j = 0; j < C / 4; ++j) x[j] = __ldcg(at + (c / 4 + j) * kT);
        for (int i = 1; i < used; i += 2) {  // two items' loads in flight
            float4 y[2][C / 4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < C / 4; ++j) {
                    y[h][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i + h < used) y[h][j] = __ldcg(at + (i + h) * stride + (c / 4 + j) * kT);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < C / 4; ++j)
                    x[j] = make_float4(x[j].x + y[h][j].x, x[j].y + y[h][j].y, x[j].z + y[h][j].z, x[j].w + y[h][j].w);
        }
#pragma unroll
        for (int j = 0; j < C / 4; j += 2)
            if (c + 4 * j < cols) {
                uint4 w;
                w.x = pack2<BF16>(x[j].x * scale, x[j].y * scale);
                w.y = pack2<BF16>(x[j].z * scale, x[j].w * scale);
                w.z = pack2<BF16>(x[j + 1].x * scale, x[j + 1].y * scale);
                w.w = pack2<BF16>(x[j + 1].z * scale, x[j + 1].w * scale);
                *reinterpret_cast<uint4 *>(out + c + 4 * j) = w;
            }
    }
}

// The barriers that both main kernels have, by one thread.
template <typename Bars>
__device__ __forceinline__ void init_common(Bars &sb) {
    at_init_bars(sb.s_full, 2, 1);
    at_init_bars(sb.p_ready, 2, kAtWarps);
    at_init_bars(sb.dp_full, 2, 1);
    at_init_bars(sb.ds_ready, 2, kAtWarps);
    at_init_bars(&sb.fix, 3, 1);  // fix, drain, acc
    at_init_bars(&sb.join, 3, kAtWarps);  // join, staged
    at_init_bars(sb.i_full, 2, 1);
    at_init_bars(sb.i_empty, 2, kItemReaders);
    sb.abort_flag = 0;
}

// After a timeout the load warp waits (bounded) for the copies it has begun: the
// last `stages` of `count` phases of a ring.
__device__ __forceinline__ void drain_ring(uint64_t *bars, int stages, int count, unsigned *status) {
    int no = 0;
    for (int v = max(0, count - stages); v < count; ++v)
        ptx::mbar_wait_bounded(ptx::smem_u32(bars + v % stages), (uint32_t)(v / stages) & 1u, &no, status,
                               kAtLimitNs / 8);
}

// ---- dk, dv: one tile of keys, its queries in turn

// At dim 64 and less TMEM has room for two S tiles: S of the tile after next is
// computed once dv has used P, so that the compute warps find the next S ready.
// (Three tiles in turn for S and dP, both ready a step ahead: 97 us where 95.)
// At larger dims S(i + 1) overwrites P(i) and the warps wait for it.  Shared
// memory there is full with one K and V tile, and the results pass through a stage
// of q's ring that the load warp keeps free for them; below, the next item's K and
// V come while this one's are in use, and the results have a stage of their own.
template <int DP>
struct Kv {
    static constexpr int NS = DP == 64 ? 2 : 1;               // S buffers
    static constexpr int KVB = DP == 64 ? 2 : 1;              // K and V tiles
    // stages of q, of do, of the row statistics
    static constexpr int QST = DP == 64 ? 4 : 3, DOST = DP == 64 ? 3 : 2, RST = DP == 64 ? 4 : 2;
    using Bars = AtBars<QST, DOST>;
    static constexpr uint32_t TILES = (2 * KVB + QST + DOST) * (DP / 64) * kBoxBytes;
    static constexpr uint32_t STAGE = DP == 64 ? kAtWarps * 2048 : 0;
    static constexpr uint32_t ROWS = TILES + STAGE, BARS = ROWS + RST * 1024;
    static constexpr uint32_t SMEM = BARS + sizeof(Bars) + 2 * 128;  // and the items
};

struct KvItem {
    AtSeq s;
    int b, h, k0, off, qt_begin, nq;
    int it0, n;      // steps: query tiles, over the group's heads in turn
    int tile, c, used;
    float sds;       // dS is held times this
    bool live;       // there are keys, and steps or zeros to be stored
};
static_assert(sizeof(KvItem) <= 128);

template <bool SLOTS>
__device__ __forceinline__ KvItem kv_item(const AtArgs &a, int u) {
    KvItem w;
    w.c = 0;
    if (a.chunks > 1) w.c = u % a.chunks, u /= a.chunks;
    w.tile = u;
    int tile;
    if (SLOTS && a.k_slots) {
        w.h = u % a.hkv;
        find_tile(a.cu_k, a.total_k, a.batch, u / a.hkv, w.b, tile);
    } else if (a.tile_slow) {
        w.b = u % a.batch, u /= a.batch;
        w.h = u % a.hkv, tile = u / a.hkv;
    } else {
        tile = u % a.tiles, u /= a.tiles;
        w.h = u % a.hkv, w.b = u / a.hkv;
    }
    w.s = at_seq(a, w.b);
    const bool in = tile >= 0 && tile < (w.s.lk + kT - 1) / kT;
    w.k0 = in ? tile * kT : 0;
    w.off = w.s.lk - w.s.lq;  // causal: key j is seen by the queries i >= j - off
    const int qt_end = (w.s.lq + kT - 1) / kT;
    w.qt_begin = a.causal ? min(max(w.k0 - w.off, 0) / kT, qt_end) : 0;
    w.nq = qt_end - w.qt_begin;
    w.live = in;
    w.n = w.live ? w.nq * a.group : 0;
    cut(a, w.c, w.it0, w.n, w.used);
    w.live = w.live && w.c < w.used;
    if (!w.live) w.n = 0;
    return w;
}

template <int DP, bool BF16, bool SLOTS>
__global__ void __launch_bounds__(kAtThreads, 1)
    attn_kv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                   const AtArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr uint32_t TILE = DP / 64 * kBoxBytes;
    constexpr int NS = Kv<DP>::NS, KVB = Kv<DP>::KVB, kQStages = Kv<DP>::QST, kDoStages = Kv<DP>::DOST, kRStages = Kv<DP>::RST;
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t sK = sbase, sV = sK + KVB * TILE, sQ = sV + KVB * TILE, sDo = sQ + kQStages * TILE;
    float *rows = reinterpret_cast<float *>(smem + Kv<DP>::ROWS);
    auto &sb = *reinterpret_cast<typename Kv<DP>::Bars *>(smem + Kv<DP>::BARS);
    KvItem *slots = reinterpret_cast<KvItem *>(&sb + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (sbase & 1023) {  // the swizzled tiles need it
        if (tid == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    if (tid == 0) {
        at_init_bars(sb.stat, KVB, 1);
        at_init_bars(sb.stat_empty, KVB, 1);
        at_init_bars(sb.a_full, kQStages, 1);
        at_init_bars(sb.a_empty, kQStages, 1);
        at_init_bars(sb.b_full, kDoStages, 1);
        at_init_bars(sb.b_empty, kDoStages, 1);
        at_init_bars(sb.r_full, kRStages, 1);
        at_init_bars(sb.r_empty, kRStages, kAtWarps);
        init_common(sb);
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
    const uint32_t tS = tmem, tDp = tmem + NS * 128, tDv = tDp + 128, tDk = tDv + DP;
    volatile int *ab = &sb.abort_flag;
    const bool packed = a.cu_q != nullptr;
    bool ok = true;

    if (warp < 4) {
    ptx::regs_dec<kCtlRegs>();
    if (warp == 0) {
        uint32_t fphase = 0;
        const uint32_t bfix = ptx::smem_u32(&sb.fix);
        int gt = 0, nq_begun = 0, nr_begun = 0, ndo_begun = 0, staged = 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = ok && ptx::mbar_wait_bounded(ptx::smem_u32(bar), parity & 1u, ab, a.status, kAtLimitNs);
            ok = __all_sync(0xffffffffu, ok) != 0;
            return ok;
        };
        // the next item from `item` on with anything to do
        const int items = !SLOTS || !a.k_slots ? a.items
                                     : min(a.items, used_slots(a.cu_k, a.total_k, a.batch) * a.hkv * a.chunks);
        auto live = [&](int item) {
            KvItem w{};
            w.tile = -1;
            for (; item < items; item = next_item(a.next)) {
                w = kv_item<SLOTS>(a, item);
                if (w.live) break;
                w.tile = -1;
            }
            w.sds = BF16 || w.tile < 0 ? 1.f : ds_scale(a, w.b, w.h);
            return w;
        };
        KvItem w = live((int)blockIdx.x);
        for (int k = 0; hand_out(a, k, w, slots, sb, ok); ++k, w = live(next_item(a.next))) {
            const int tb = packed ? 0 : w.b;
            for (int it = 0; ok && it < w.n; ++it) {
                const int t = w.it0 + it, g = t / w.nq, q0 = (w.qt_begin + t - g * w.nq) * kT, hq = w.h * a.group + g;
                const int valid = min(kT, w.s.lq - q0);
                const int st = nq_begun % kQStages, sd = ndo_begun % kDoStages, sr = nr_begun % kRStages;
                // dim 128: the stage after an item's first q holds the results of the item before
                // until they are stored (gt: items whose K and V have been asked for)
                if (Kv<DP>::STAGE == 0 && it < 2 && staged < gt - 1) {
                    if (!wait(&sb.staged[staged & 1], (uint32_t)(staged >> 1))) break;
                    ++staged;
                }
                if (nq_begun >= kQStages && !wait(&sb.a_empty[st], (uint32_t)(nq_begun / kQStages - 1))) break;
                ++nq_begun;
                ok = load_tile<DP>(sQ + st * TILE, &tq, w.s.q0 + q0, hq, tb, valid, packed,
                                   ptx::smem_u32(&sb.a_full[st]), bfix, fphase, ab, a.status);
                if (!ok) break;
                if (nr_begun >= kRStages && !wait(&sb.r_empty[sr], (uint32_t)(nr_begun / kRStages - 1))) break;
                ++nr_begun;
                if (lane == 0) {
                    const uint32_t bar = ptx::smem_u32(&sb.r_full[sr]);
                    const long long r0 = w.s.row0 + (long long)hq * a.head_rows + q0;
                    ptx::mbar_arrive_expect_tx(bar, 2 * kT * 4);
                    ptx::bulk_load(ptx::smem_u32(rows + sr * 2 * kT), a.nlse + r0, kT * 4, bar);
                    ptx::bulk_load(ptx::smem_u32(rows + sr * 2 * kT + kT), a.ndsum + r0, kT * 4, bar);
                }
                if (ndo_begun >= kDoStages && !wait(&sb.b_empty[sd], (uint32_t)(ndo_begun / kDoStages - 1))) break;
                ++ndo_begun;
                ok = load_tile<DP>(sDo + sd * TILE, &tdo, w.s.q0 + q0, hq, tb, valid, packed,
                                   ptx::smem_u32(&sb.b_full[sd]), bfix, fphase, ab, a.status);
                if (!ok) break;
                if (it == 0) {  // K and V, once the item that used their tiles before is through with them:
                                // the last to be free
                    const int sk = gt % KVB;
                    if (gt >= KVB && !wait(&sb.stat_empty[sk], (uint32_t)(gt / KVB - 1))) break;
                    ++gt;
                    if (lane == 0) {
                        const uint32_t bar = ptx::smem_u32(&sb.stat[sk]);
                        ptx::mbar_arrive_expect_tx(bar, 2 * TILE);
#pragma unroll
                        for (int j = 0; j < DP / 64; ++j) {
                            const uint32_t to = sk * TILE + j * kBoxBytes;
                            ptx::tma_load_4d(sK + to, &tk, j * 64, (int)w.s.k0 + w.k0, w.h, tb, bar);
                            ptx::tma_load_4d(sV + to, &tv, j * 64, (int)w.s.k0 + w.k0, w.h, tb, bar);
                        }
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
        }
        if (!ok) {
            drain_ring(sb.stat, KVB, gt, a.status);
            drain_ring(sb.a_full, kQStages, nq_begun, a.status);
            drain_ring(sb.b_full, kDoStages, ndo_begun, a.status);
            drain_ring(sb.r_full, kRStages, nr_begun, a.status);
        }
    } else if (warp == 1) {
        // The whole warp walks the loop and one elected lane issues: descriptors and
        // counters are then uniform over the warp, and an MMA takes ~50 cycles to
        // issue instead of ~100 (more than the 64 that one of 128 columns runs).
        constexpr uint32_t id_s = ptx::idesc_f16(128, 128, BF16, false);
        constexpr uint32_t id_a = ptx::idesc_f16(128, DP, BF16, true);
        const int steps = (a.dim + 15) / 16;
        auto wait = [&](AtWait x, AtWait y) { return ok = wait_both(x, y, ab, a.status); };
        auto full_q = [&](Ring r) { return AtWait{&sb.a_full[r.s], r.ph}; };
        auto full_do = [&](Ring r) { return AtWait{&sb.b_full[r.s], r.ph}; };
        Ring rs, rk, rp, rv;   // q's ring for S and for dk, do's for dP and for dv
        int gt = 0, js = 0, jp = 0;  // items; tiles of S, tiles of dv so far
        auto mma_s = [&]() {
            mma_rows<DP>(tS + js % NS * 128, sK + gt % KVB * TILE, sQ + rs.s * TILE, steps, id_s, &sb.s_full[js & 1]);
            rs.step(kQStages);
            ++js;
        };
        auto mma_dp = [&](bool last) {  // the item's last product of K's and V's tiles
            mma_rows<DP>(tDp, sV + gt % KVB * TILE, sDo + rp.s * TILE, steps, id_s, &sb.dp_full[0],
                         last ? &sb.stat_empty[gt % KVB] : nullptr);
            rp.step(kDoStages);
        };
        const KvItem *w;
        for (int k = 0; (w = take_item(a, k, slots, sb, ok)) != nullptr; ++k) {
            const int n = w->n;
            done_item(k, sb);
            if (n == 0) continue;
            const AtWait stat{&sb.stat[gt % KVB], (uint32_t)(gt / KVB)};
            if (!wait(stat, full_q(rs))) break;
            mma_s();
            if (NS == 2 && n > 1) {
                if (!wait(full_q(rs), full_q(rs))) break;
                mma_s();
            }
            if (!wait(full_do(rp), stat)) break;
            mma_dp(n == 1);
            for (int it = 0; it < n; ++it, ++jp) {
                const bool ms = it + NS < n, md = it + 1 < n;  // more S, more dP to come
                const AtWait pr{&sb.p_ready[jp & 1], (uint32_t)(jp / 2)}, dr{&sb.ds_ready[jp & 1], (uint32_t)(jp / 2)};
                if (!wait(pr, ms ? full_q(rs) : pr)) break;
                mma_acc(tDv, tS + jp % NS * 128, sDo + rv.s * TILE, id_a, it > 0, &sb.b_empty[rv.s]);
                rv.step(kDoStages);
                // S overwrites P, dP overwrites dS: this warp's MMAs run in the order of issue.
                // (The first dv and dk overwrite the item before's, which the compute warps
                // have stored before the P that they follow.)
                if (ms) mma_s();
                if (!wait(dr, md ? full_do(rp) : dr)) break;
                mma_acc(tDk, tDp, sQ + rk.s * TILE, id_a, it > 0, &sb.a_empty[rk.s]);
                rk.step(kQStages);
                if (md) mma_dp(it + 2 == n);
            }
            if (!ok) break;
            if (ptx::elect_one()) ptx::mma_commit(ptx::smem_u32(&sb.acc));
            __syncwarp();
            ++gt;
        }
        finish_mmas(ok, sb, a.status);
    }
    } else {
        ptx::regs_inc<kCompRegs>();
        const int wg = (warp - 4) >> 2, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const float cs = a.scale * kLog2e;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            const bool r = ptx::mbar_wait_bounded(ptx::smem_u32(bar), parity & 1u, ab, a.status, kAtLimitNs);
            return ok = __all_sync(0xffffffffu, r) != 0;
        };
        int gt = 0, g0 = 0;
        uint32_t joined = 0;
        const KvItem *w;
        for (int k = 0; (w = take_item(a, k, slots, sb, ok)) != nullptr; ++k) {
            const int n = w->n;
            const float sds = BF16 ? 1.f : w->sds, pds = BF16 ? 1.f : sds * exp2f(-kPShift);  // pds: from the held P
            {
                const int begin = w->qt_begin * kT, end = begin + w->nq * kT;
                // this thread's key is seen by the queries from here on, the tile's last one by those from `all` on
                const int sees = w->k0 + quarter * 32 + lane - w->off, all = w->k0 + kT - 1 - w->off;
                // the step's first query, over the group's heads in turn
                int q0 = n > 0 ? begin + w->it0 % w->nq * kT : 0;
                for (int it = 0; it < n; ++it) {
                    const int i = g0 + it, sr = i % kRStages;
                    const float *nl = rows + sr * 2 * kT + wg * 32, *nd = nl + kT;
                    float2 p[16];
                    if (!(ok = wait_both({&sb.r_full[sr], (uint32_t)(i / kRStages)},
                                         {&sb.s_full[i & 1], (uint32_t)(i / 2)}, ab, a.status)))
                        break;
                    const uint32_t ts = tS + i % NS * 128 + lanes + wg * 32;
                    tmem_load(ts, p);
                    probabilities(p, cs, nl);
                    if (a.causal && q0 < all) {
                        const int first = sees - q0 - wg * 32;  // columns before it do not see the key
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            if (2 * c < first) p[c].x = 0.f;
                            if (2 * c + 1 < first) p[c].y = 0.f;
                        }
                    }
                    q0 += kT;
                    if (q0 == end) q0 = begin;
                    tmem_store<BF16>(ts, p);
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.p_ready[i & 1]));
                    if (!wait(&sb.dp_full[0], (uint32_t)i)) break;
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
                        ptx::mbar_arrive(ptx::smem_u32(&sb.ds_ready[i & 1]));
                        ptx::mbar_arrive(ptx::smem_u32(&sb.r_empty[sr]));
                    }
                }
            }
            if (!ok) break;
            if (n > 0 && !wait(&sb.acc, (uint32_t)gt)) break;
            ptx::tc_fence_after();
            {
                // warpgroups 0 and 1 store dv, 2 and 3 dk, half of the columns each
                const bool isk = wg >= 2;
                const int c0 = (wg & 1) * (DP / 2), row = w->k0 + quarter * 32;  // the warp's first key
                const long long *sg = isk ? a.sdk : a.sdv;
                uint16_t *out = static_cast<uint16_t *>(isk ? a.dk : a.dv) + (packed ? 0 : w->b) * sg[0] +
                                (w->s.k0 + row) * sg[1] + w->h * sg[2] + c0;
                const float f = isk ? a.scale / sds : (BF16 ? 1.f : exp2f(-kPShift));
                const uint32_t acc = (isk ? tDk : tDv) + lanes + c0;
                constexpr long long ITEM = 2 * DP * kT / 4;  // float4 of an item's sums
                float4 *at = reinterpret_cast<float4 *>(a.part) + w->tile * a.chunks * ITEM + wg * (DP / 2) / 4 * kT +
                             quarter * 32 + lane;
                const int live = w->s.lk - row;  // of the warp's rows
                if (w->used > 1)
                    sums_to_memory<DP / 2>(acc, at + w->c * ITEM);
                else if (n == 0)
                    store_row<DP / 2, BF16>(acc, f, true, lane < live, out + lane * sg[1], a.dim - c0);
                else
                    store_rows_staged<DP / 2, BF16>(acc, f, live, out, sg[1], a.dim - c0,
                                                    smem + (Kv<DP>::STAGE ? Kv<DP>::TILES
                                                                          : (2 * KVB + (g0 + n + 1) % kQStages) * TILE) +
                                                        (warp - 4) * 2048);
                ptx::tc_fence_before();
                if (n > 0) ++gt;
                if (Kv<DP>::STAGE == 0 && n > 0) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.staged[(gt - 1) & 1]));  // of item gt - 1
                }
                if (w->used > 1) {
                    const bool last = arrive_last(a, w->tile, w->used, sb, joined, ok);
                    if (!ok) break;
                    if (last)
                        store_sums<DP / 2, BF16>(at, w->used, ITEM, f, lane < live, out + lane * sg[1], a.dim - c0);
                }
            }
            done_item(k, sb);
            g0 += n;
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

// The item's q and do rows are A operands of every tile's products, so they lie
// in TMEM (16-bit, 32 or 64 columns each): the products then read one operand
// from shared memory instead of two, whose 128 bytes per cycle are what an MMA
// of 128 columns with both operands there waits for.  They come there through
// shared memory, where the next item's wait while this one runs.  At dim 128 TMEM
// has room for one dP, below it for two, of which one is computed while the
// other's dS is used.
template <int DP>
struct Qk {
    static constexpr int NB = DP == 64 ? 2 : 1;   // dP buffers
    static constexpr int KST = DP == 64 ? 4 : 3, VST = DP == 64 ? 3 : 2;
    using Bars = AtBars<KST, VST>;
    static constexpr uint32_t TILES = (2 + KST + VST) * (DP / 64) * kBoxBytes;
    static constexpr uint32_t SMEM = TILES + sizeof(Bars) + 2 * 128;  // and the items
};

// D[128 x 128] = A[128 x dim] B[128 x dim]^T, A in TMEM.
template <int DP>
__device__ __forceinline__ void mma_rows_ts(uint32_t d, uint32_t ta, uint32_t sb, int steps, uint32_t idesc,
                                            uint64_t *done, uint64_t *done2 = nullptr) {
    const ptx::Desc db = ptx::desc_of(sb, 16, 1024, 2);
    if (ptx::elect_one()) {
        auto step = [&](int ks) {
            ptx::mma_f16_ts(d, ta + ks * 8, db, ((ks >> 2) * kBoxBytes + (ks & 3) * 32) >> 4, idesc, ks > 0);
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

struct QItem {
    AtSeq s;
    int b, h, q0, off;
    int it0, n;      // steps: key tiles that any of the tile's queries sees
    int tile, c, used;
    float sds;       // dS is held times this
    bool live;       // there are queries, and steps or zeros to be stored
};
static_assert(sizeof(QItem) <= 128);

template <bool SLOTS>
__device__ __forceinline__ QItem q_item(const AtArgs &a, int u) {
    QItem w;
    w.c = 0;
    if (a.chunks > 1) w.c = u % a.chunks, u /= a.chunks;
    w.tile = u;
    int tile;
    if (SLOTS && a.q_slots) {  // causal: a sequence's tiles with the most keys first
        w.h = u % a.hq, u /= a.hq;
        find_tile(a.cu_q, a.total_q, a.batch, a.causal ? used_slots(a.cu_q, a.total_q, a.batch) - 1 - u : u, w.b, tile);
    } else if (a.tile_slow) {  // causal: the tiles with the most keys first
        w.b = u % a.batch, u /= a.batch;
        w.h = u % a.hq, tile = a.tiles - 1 - u / a.hq;
    } else {
        tile = u % a.tiles, u /= a.tiles;
        w.h = u % a.hq, w.b = u / a.hq;
    }
    w.s = at_seq(a, w.b);
    w.live = tile >= 0 && tile < (w.s.lq + kT - 1) / kT;
    w.q0 = w.live ? tile * kT : 0;
    w.off = w.s.lk - w.s.lq;
    w.n = w.live ? (w.s.lk + kT - 1) / kT : 0;
    if (a.causal && w.live) {
        const int last = min(w.q0 + kT, w.s.lq) - 1 + w.off;  // the last key any of its queries sees
        w.n = last < 0 ? 0 : min(w.n, last / kT + 1);
    }
    cut(a, w.c, w.it0, w.n, w.used);
    w.live = w.live && w.c < w.used;
    if (!w.live) w.n = 0;
    return w;
}

template <int DP, bool BF16, bool SLOTS>
__global__ void __launch_bounds__(kAtThreads, 1)
    attn_q_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                  const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                  const AtArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr uint32_t TILE = DP / 64 * kBoxBytes;
    const uint32_t sbase = ptx::smem_u32(smem);
    constexpr int NB = Qk<DP>::NB, kKStages = Qk<DP>::KST, kVStages = Qk<DP>::VST;
    const uint32_t sQ = sbase, sDo = sQ + TILE, sK = sDo + TILE, sV = sK + kKStages * TILE;
    auto &sb = *reinterpret_cast<typename Qk<DP>::Bars *>(smem + Qk<DP>::TILES);
    QItem *slots = reinterpret_cast<QItem *>(&sb + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (sbase & 1023) {
        if (tid == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    if (tid == 0) {
        at_init_bars(&sb.stat[0], 1, kAtWarps);  // the rows in TMEM
        at_init_bars(&sb.stat[1], 1, 1);         // in shared memory
        at_init_bars(sb.stat_empty, 1, kAtWarps);
        at_init_bars(sb.a_full, kKStages, 1);
        at_init_bars(sb.a_empty, kKStages, 1);
        at_init_bars(sb.b_full, kVStages, 1);
        at_init_bars(sb.b_empty, kVStages, 1);
        init_common(sb);
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
    const uint32_t tS = tmem, tDp = tmem + 128, tDq = tDp + NB * 128, tQ = tDq + DP, tDo = tQ + DP / 2;
    volatile int *ab = &sb.abort_flag;
    const bool packed = a.cu_q != nullptr;
    bool ok = true;

    if (warp < 4) {
    ptx::regs_dec<kCtlRegs>();
    if (warp == 0) {
        uint32_t fphase = 0;
        const uint32_t bfix = ptx::smem_u32(&sb.fix);
        int nk_begun = 0, nv_begun = 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = ok && ptx::mbar_wait_bounded(ptx::smem_u32(bar), parity & 1u, ab, a.status, kAtLimitNs);
            ok = __all_sync(0xffffffffu, ok) != 0;
            return ok;
        };
        const int items = !SLOTS || !a.q_slots ? a.items
                                     : min(a.items, used_slots(a.cu_q, a.total_q, a.batch) * a.hq * a.chunks);
        auto live = [&](int item) {
            QItem w{};
            w.tile = -1;
            for (; item < items; item = next_item(a.next + 1)) {
                w = q_item<SLOTS>(a, item);
                if (w.live) break;
                w.tile = -1;
            }
            w.sds = BF16 || w.tile < 0 ? 1.f : ds_scale(a, w.b, w.h / a.group);
            return w;
        };
        QItem w = live((int)blockIdx.x);
        int gt = 0;
        for (int k = 0; hand_out(a, k, w, slots, sb, ok); ++k, w = live(next_item(a.next + 1))) {
            const int tb = packed ? 0 : w.b, hk = w.h / a.group;
            if (w.n == 0) continue;
            // rows past a packed sequence's last are its neighbour's: their results are not stored
            if (gt > 0 && !wait(sb.stat_empty, (uint32_t)(gt - 1))) break;
            ++gt;
            if (lane == 0) {
                const uint32_t bar = ptx::smem_u32(&sb.stat[1]);
                ptx::mbar_arrive_expect_tx(bar, 2 * TILE);
#pragma unroll
                for (int j = 0; j < DP / 64; ++j) {
                    ptx::tma_load_4d(sQ + j * kBoxBytes, &tq, j * 64, (int)w.s.q0 + w.q0, w.h, tb, bar);
                    ptx::tma_load_4d(sDo + j * kBoxBytes, &tdo, j * 64, (int)w.s.q0 + w.q0, w.h, tb, bar);
                }
            }
            __syncwarp();
            for (int it = 0; ok && it < w.n; ++it) {
                const int st = nk_begun % kKStages, sv = nv_begun % kVStages;
                const int key = (w.it0 + it) * kT, valid = min(kT, w.s.lk - key);
                if (nk_begun >= kKStages && !wait(&sb.a_empty[st], (uint32_t)(nk_begun / kKStages - 1))) break;
                ++nk_begun;
                ok = load_tile<DP>(sK + st * TILE, &tk, w.s.k0 + key, hk, tb, valid, packed,
                                   ptx::smem_u32(&sb.a_full[st]), bfix, fphase, ab, a.status);
                if (!ok) break;
                if (nv_begun >= kVStages && !wait(&sb.b_empty[sv], (uint32_t)(nv_begun / kVStages - 1))) break;
                ++nv_begun;
                ok = load_tile<DP>(sV + sv * TILE, &tv, w.s.k0 + key, hk, tb, valid, packed,
                                   ptx::smem_u32(&sb.b_full[sv]), bfix, fphase, ab, a.status);
            }
            if (!ok) break;
        }
        if (!ok) {
            drain_ring(&sb.stat[1], 1, gt, a.status);
            drain_ring(sb.a_full, kKStages, nk_begun, a.status);
            drain_ring(sb.b_full, kVStages, nv_begun, a.status);
        }
    } else if (warp == 1) {
        constexpr uint32_t id_s = ptx::idesc_f16(128, 128, BF16, false);
        constexpr uint32_t id_a = ptx::idesc_f16(128, DP, BF16, true);
        const int steps = (a.dim + 15) / 16;
        auto wait = [&](AtWait x, AtWait y) { return ok = wait_both(x, y, ab, a.status); };
        auto full_k = [&](Ring r) { return AtWait{&sb.a_full[r.s], r.ph}; };
        auto full_v = [&](Ring r) { return AtWait{&sb.b_full[r.s], r.ph}; };
        Ring rs, rv, rq;  // k's ring for S and for dq, v's
        int gt = 0, js = 0, jp = 0;  // items; tiles of S and dP, tiles of dq so far
        auto mma_s = [&]() {
            mma_rows_ts<DP>(tS, tQ, sK + rs.s * TILE, steps, id_s, &sb.s_full[js & 1]);
            rs.step(kKStages);
        };
        auto mma_dp = [&]() {
            mma_rows_ts<DP>(tDp + js % NB * 128, tDo, sV + rv.s * TILE, steps, id_s, &sb.dp_full[js & 1],
                            &sb.b_empty[rv.s]);
            rv.step(kVStages);
            ++js;
        };
        const QItem *w;
        for (int k = 0; (w = take_item(a, k, slots, sb, ok)) != nullptr; ++k) {
            const int n = w->n;
            done_item(k, sb);
            if (n == 0) continue;
            const AtWait stat{&sb.stat[0], (uint32_t)gt};
            if (!wait(stat, full_k(rs))) break;
            mma_s();
            if (!wait(full_v(rv), stat)) break;
            mma_dp();
            for (int it = 0; it < n; ++it, ++jp) {
                const bool more = it + 1 < n;
                const AtWait pr{&sb.p_ready[jp & 1], (uint32_t)(jp / 2)}, dr{&sb.ds_ready[jp & 1], (uint32_t)(jp / 2)};
                if (!wait(pr, more ? full_k(rs) : pr)) break;  // S is in registers
                if (more) mma_s();
                if (NB == 2 && more) {
                    if (!wait(full_v(rv), full_v(rv))) break;
                    mma_dp();
                }
                if (!wait(dr, more && NB == 1 ? full_v(rv) : dr)) break;
                mma_acc(tDq, tDp + jp % NB * 128, sK + rq.s * TILE, id_a, it > 0, &sb.a_empty[rq.s]);
                rq.step(kKStages);
                // with one buffer dP overwrites dS: this warp's MMAs run in the order of issue.
                // (The first dq overwrites the item before's, stored before the dS it follows.)
                if (NB == 1 && more) mma_dp();
            }
            if (!ok) break;
            if (ptx::elect_one()) ptx::mma_commit(ptx::smem_u32(&sb.acc));
            __syncwarp();
            ++gt;
        }
        finish_mmas(ok, sb, a.status);
    }
    } else {
        ptx::regs_inc<kCompRegs>();
        const int wg = (warp - 4) >> 2, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const int r = quarter * 32 + lane;
        const float cs = a.scale * kLog2e;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            const bool x = ptx::mbar_wait_bounded(ptx::smem_u32(bar), parity & 1u, ab, a.status, kAtLimitNs);
            return ok = __all_sync(0xffffffffu, x) != 0;
        };
        int gt = 0, g0 = 0, k = 0;
        uint32_t joined = 0;
        int gr = 0;  // rows put into TMEM so far
        // the warpgroup's DP / 8 words of this thread's rows of q and do, from the
        // swizzled tiles (chunk j of row r at j ^ (r & 7)) into TMEM
        auto put_rows = [&]() {
            if (!wait(&sb.stat[1], (uint32_t)gr)) return;
            ++gr;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint8_t *tile = smem + half * TILE + r * 128;
                uint32_t x[DP / 8];
#pragma unroll
                for (int j = 0; j < DP / 32; ++j) {
                    const int c = wg * (DP / 32) + j;  // 16-byte chunk of the row
                    const uint4 v = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * kBoxBytes + (((c & 7) ^ (r & 7)) << 4));
                    x[4 * j] = v.x, x[4 * j + 1] = v.y, x[4 * j + 2] = v.z, x[4 * j + 3] = v.w;
                }
                const uint32_t to = (half ? tDo : tQ) + lanes + wg * (DP / 8);
                if constexpr (DP == 128) ptx::tmem_st16(to, x);
                else ptx::tmem_st8(to, x);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.stat[0]));
        };
        // the tiles may be filled again
        auto free_rows = [&]() {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(sb.stat_empty));
        };
        const QItem *w = take_item(a, k, slots, sb, ok);
        if (w && w->n > 0) {
            put_rows();
            free_rows();
        }
        while (ok && w) {
            const int n = w->n;
            const float sds = BF16 ? 1.f : w->sds, pds = BF16 ? 1.f : sds * exp2f(-kPShift);
            if (n > 0) {
                const long long row = w->s.row0 + (long long)w->h * a.head_rows + w->q0 + r;
                const float nl = __ldcg(a.nlse + row), nd = __ldcg(a.ndsum + row) * pds;
                // counted from the first step: this thread's query sees the keys before `sees`; tiles
                // that end by `all` need no mask
                const int lk = w->s.lk - w->it0 * kT, diag = w->q0 + w->off + 1 - w->it0 * kT;
                const int sees = a.causal ? min(lk, diag + r) : lk, all = a.causal ? min(lk, diag) : lk;
                for (int it = 0; it < n; ++it) {
                    const int i = g0 + it;
                    float2 p[16];
                    if (!wait(&sb.s_full[i & 1], (uint32_t)(i / 2))) break;
                    ptx::tc_fence_after();
                    tmem_load(tS + lanes + wg * 32, p);
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.p_ready[i & 1]));
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        p[c] = ptx::fma2(p[c], make_float2(cs, cs), make_float2(nl, nl));
                        p[c] = make_float2(ptx::ex2(p[c].x), ptx::ex2(p[c].y));
                    }
                    if (it * kT + kT > all) {
                        const int lim = sees - it * kT - wg * 32;  // columns from it on are masked
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            if (2 * c >= lim) p[c].x = 0.f;
                            if (2 * c + 1 >= lim) p[c].y = 0.f;
                        }
                    }
                    if (!wait(&sb.dp_full[i & 1], (uint32_t)(i / 2))) break;
                    ptx::tc_fence_after();
                    const uint32_t td = tDp + i % NB * 128 + lanes + wg * 32;
                    float2 x[16];
                    tmem_load(td, x);
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        if constexpr (BF16) x[c] = ptx::add2(x[c], make_float2(nd, nd));
                        else x[c] = ptx::fma2(x[c], make_float2(pds, pds), make_float2(nd, nd));
                        x[c] = ptx::mul2(p[c], x[c]);
                    }
                    tmem_store<BF16>(td, x);
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.ds_ready[i & 1]));
                }
                if (!ok) break;
            }
            const QItem *next = take_item(a, k + 1, slots, sb, ok);
            if (!ok || (n > 0 && !wait(&sb.acc, (uint32_t)gt))) break;
            ptx::tc_fence_after();
            // the products that read this item's rows are done
            const bool more = next && next->n > 0;
            if (more) {
                put_rows();
                // at dim 128 the results pass through the tile of q: all warps have read it
                if (ok && DP == 128) wait(&sb.stat[0], (uint32_t)(gr - 1));
                if (!ok) break;
                if (DP == 64) free_rows();
            }
            {
                // each warpgroup stores a quarter of the columns
                const int c0 = wg * (DP / 4), first = w->q0 + quarter * 32, live = w->s.lq - first;
                uint16_t *out = static_cast<uint16_t *>(a.dq) + (packed ? 0 : w->b) * a.sdq[0] +
                                (w->s.q0 + first) * a.sdq[1] + w->h * a.sdq[2] + c0;
                constexpr long long ITEM = DP * kT / 4;
                float4 *at = reinterpret_cast<float4 *>(a.part) + w->tile * a.chunks * ITEM + c0 / 4 * kT + r;
                // The staged store needs the tile of q, which is free once the next item's rows have been
                // read from it, or where no item follows.  An item without keys in between leaves in it
                // (now or soon) the rows of the one after.
                if (w->used == 1 && (DP == 64 || n == 0 || (next && !more)))
                    store_row<DP / 4, BF16>(tDq + lanes + c0, a.scale / sds, n == 0, lane < live, out + lane * a.sdq[1],
                                            a.dim - c0);
                else if (w->used == 1)
                    store_rows_staged<DP / 4, BF16>(tDq + lanes + c0, a.scale / sds, live, out, a.sdq[1], a.dim - c0,
                                                    smem + (warp - 4) * 2048);
                else
                    sums_to_memory<DP / 4>(tDq + lanes + c0, at + w->c * ITEM);
                if (DP == 128 && more) free_rows();
                ptx::tc_fence_before();
                if (n > 0) ++gt;
                if (w->used > 1) {
                    const bool last = arrive_last(a, w->tile, w->used, sb, joined, ok);
                    if (!ok) break;
                    if (last)
                        store_sums<DP / 4, BF16>(at, w->used, ITEM, a.scale / sds, lane < live, out + lane * a.sdq[1],
                                                 a.dim - c0);
                }
            }
            done_item(k, sb);
            ++k;
            g0 += n;
            w = next;
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

// Packed: tiles are counted by the tokens where counting up to the bounds would look
// at more than this many times as many.  A block passes a tile that does not exist in
// about a microsecond.  (us, by the tokens / up to the bounds: 64 documents of 700 to
// 1024 tokens, 32 heads of 128, tight bounds, 1.2 times as many 1906 / 2097, with all
// tokens as the bound 1907 / 11193; 4 long and 100 short ones, 3 times as many 251 /
// 367; 200 of up to 128 tokens, where every sequence is one tile and a third of the
// slots are none, 231 / 204.)
constexpr long long kLoose = 2;

struct AtCut {
    int chunk, chunks, tiles;  // steps per item, items per tile, tiles with a counter (0: not cut)
};
struct AtPlan {
    int dp, q_tiles, k_tiles;  // tiles of the longest sequence
    int q_slots, k_slots;      // tiles counted by the tokens (find_tile), 0: as below
    long long q_units, k_units;  // tiles of one head that are looked at: of every sequence, as many as
                                 // the longest has, or slots
    long long head_rows;   // padded rows of one head
    AtCut kv, q;
    size_t off_max, max_bytes, off_nlse, off_ndsum, off_arrived, off_part, total;
};

// Whether tiles of `steps` steps at most, `tiles` of them with `all` steps
// together, are cut into items: where the longest is more than 12 steps above
// `most` times an SM's share, into items of about half of it, but of 8 steps at
// least.  (A step takes 1 to 1.5 us; an item that is joined costs 4 us, and its
// tile 1.5 us more per item.  Causal, dim 128, whole / cut: 4096 tokens with 4
// heads 59 / 80 us, 2048 with 8 / 1 heads 186 / 47, 1024 with 32 / 4 heads 111 / 50,
// 8192 with 8 / 2 heads 413 / 302.  Items of 0.4 or 0.9 of the share: 3 to 8% slower
// on the last and on 3 documents of 8192 tokens; of 4 steps at least: 74 us where 50.)
AtCut plan_cut(long long tiles, long long steps, double all, double most) {
    const double share = all / kNumSMs;
    const long long chunk = std::max(8LL, (long long)(0.6 * share) + 1);
    AtCut c{(int)std::max(1LL, steps), 1, 0};
    if (steps <= most * share + 12 || steps < chunk + chunk / 4 || tiles > 1024) return c;
    c.chunk = (int)chunk;
    c.chunks = (int)((steps + chunk - 1) / chunk);
    c.tiles = (int)tiles;
    return c;
}

// The strides that the kernels use; packed sequences have none from one to the next.
void fill_strides(const cba_attention_desc_t &d, const cba_attn_strides_t &s, int heads, long long len, long long *out) {
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
    auto count = [&](long long len, long long total, int *tiles, int *slots, long long *units) {
        if (d->packed) len = std::min(len, total);
        *tiles = (int)((len + kT - 1) / kT);
        *units = (long long)*tiles * d->batch;
        const long long by_tokens = total / kT + d->batch;
        *slots = d->packed && *units > kLoose * by_tokens ? (int)by_tokens : 0;
        if (*slots) *units = by_tokens;
    };
    count(d->len_q, d->total_q, &p->q_tiles, &p->q_slots, &p->q_units);
    count(d->len_k, d->total_k, &p->k_tiles, &p->k_slots, &p->k_units);
    long long rows;
    if (d->packed) {
        p->head_rows = (d->total_q + kT - 1) / kT * kT + (long long)kT * (d->batch + 1);
        rows = p->head_rows * d->heads_q;
    } else {
        p->head_rows = (long long)p->q_tiles * kT;
        rows = p->head_rows * d->heads_q * d->batch;
    }
    if (std::max(p->k_units * d->heads_kv, p->q_units * d->heads_q) >= (1LL << 30) || rows >= (1LL << 40))
        return CBA_ERR_UNSUPPORTED;
    {
        // steps of all tiles together; packed: as if all sequences were the longest
        auto by_length = [](long long total, long long len) {
            return (double)total / std::max(1LL, std::min(len, total));
        };
        const double seqs = !d->packed ? d->batch
                                       : std::min((double)d->batch, std::max(by_length(d->total_q, d->len_q),
                                                                             by_length(d->total_k, d->len_k)));
        const double all = seqs * d->heads_q * p->q_tiles * p->k_tiles * (d->causal ? 0.5 : 1.0);
        // SMs that are done with dk and dv go on to dq, so a tile of dk and dv may take the time
        // of both shares, and where those are whole a tile of dq that of what is left beside them
        // (packed 8192 h16/4: 176 us with its longest tile at 1.2 times the share whole, 184 us cut;
        // dq cut beside whole dk and dv, 4096 tokens, 4 heads: 75 us, whole 59)
        p->kv = plan_cut(p->k_units * d->heads_kv,
                         (long long)p->q_tiles * (d->heads_q / d->heads_kv), all, 1.75);
        p->q = plan_cut(p->q_units * d->heads_q, p->k_tiles, all, p->kv.tiles ? 1.25 : 2.3);
    }
    p->off_max = 256;  // behind the status word's 256 bytes, with which they are cleared
    p->max_bytes = d->type == CBA_F16 ? (size_t)2 * d->batch * d->heads_kv * sizeof(unsigned) : 0;
    p->off_nlse = p->off_max + (p->max_bytes + 255) / 256 * 256;
    p->off_ndsum = p->off_nlse + ((size_t)rows * 4 + 255) / 256 * 256;
    p->off_arrived = p->off_ndsum + ((size_t)rows * 4 + 255) / 256 * 256;
    p->off_part = p->off_arrived + ((size_t)(p->kv.tiles + p->q.tiles) * 4 + 255) / 256 * 256;
    // the two kernels run at the same time where one ends: sums of their own
    p->total = p->off_part + (size_t)kT * p->dp * 4 *
                                 (2 * (size_t)p->kv.tiles * p->kv.chunks + (size_t)p->q.tiles * p->q.chunks);
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

// The search for slots is in kernels of its own: with it the preparation of f16 takes 69
// registers for 60, a block less on each SM (32x676 20.4 us, 16.4), and the main kernels
// of a small call 0.3 to 0.4 us more each (2x169: 14.3 us, 12.3).
template <int DP, bool BF16, bool SLOTS>
cudaError_t attn_launch(const cba_attention_desc_t &d, const AtPlan &p, AtArgs a, const CUtensorMap *tm,
                        cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (!BF16) e = cudaMemsetAsync(a.status, 0, p.off_max + p.max_bytes, st);  // the status word and the maxima
    if (e != cudaSuccess) return e;
    // f16: the blocks that look for v's largest rows
    const int vb = BF16 ? 0 : (int)(p.k_units * d.heads_kv);
    const unsigned qgrid = (unsigned)(p.q_units * d.heads_q);
    attn_prep_kernel<DP, BF16, SLOTS><<<std::max(1u, qgrid) + vb, 256, 0, st>>>(a, std::max(1, p.q_tiles), p.k_tiles, vb);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = allow_smem<attn_kv_kernel<DP, BF16, SLOTS>>((int)Kv<DP>::SMEM);
    if (e == cudaSuccess) e = allow_smem<attn_q_kernel<DP, BF16, SLOTS>>((int)Qk<DP>::SMEM);
    if (e != cudaSuccess) return e;
    if (p.k_tiles > 0) {
        a.tiles = p.k_tiles;
        a.chunk = p.kv.chunk;
        a.chunks = p.kv.chunks;
        a.items = (int)(p.k_units * d.heads_kv) * a.chunks;
        e = launch_pdl(attn_kv_kernel<DP, BF16, SLOTS>, dim3((unsigned)std::min(a.items, kNumSMs)),
                       dim3(kAtThreads), Kv<DP>::SMEM, st, tm[0], tm[1], tm[2], tm[3], a);
        if (e != cudaSuccess) return e;
    }
    if (p.q_tiles > 0) {
        a.tiles = p.q_tiles;
        a.chunk = p.q.chunk;
        a.chunks = p.q.chunks;
        a.items = (int)qgrid * a.chunks;
        a.arrived += p.kv.tiles;
        a.part += 2 * (size_t)kT * p.dp * p.kv.tiles * p.kv.chunks;
        const unsigned blocks = (unsigned)std::min(a.items, kNumSMs);
        // without keys there is no launch between this one and the preparation
        if (p.k_tiles > 0)
            e = launch_pdl(attn_q_kernel<DP, BF16, SLOTS>, dim3(blocks), dim3(kAtThreads), Qk<DP>::SMEM, st, tm[0],
                           tm[1], tm[2], tm[3], a);
        else
            attn_q_kernel<DP, BF16, SLOTS><<<blocks, kAtThreads, Qk<DP>::SMEM, st>>>(tm[0], tm[1], tm[2], tm[3], a);
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
    a.q_slots = p.q_slots; a.k_slots = p.k_slots;
    a.causal = d->causal; a.tile_slow = d->causal; a.scale = d->scale;
    a.lse = lse;
    a.status = static_cast<unsigned *>(workspace);
    a.next = a.status + 2;
    a.cnt_kv = p.kv.tiles;
    a.cnt_q = p.q.tiles;
    a.arrived = ws_at<unsigned>(workspace, p.off_arrived);
    a.part = ws_at<float>(workspace, p.off_part);
    a.maxima = ws_at<unsigned>(workspace, p.off_max);
    a.nlse = ws_at<float>(workspace, p.off_nlse);
    a.ndsum = ws_at<float>(workspace, p.off_ndsum);
    a.head_rows = p.head_rows;
    a.o = o; a.dout = dout; a.v = v; a.dq = dq; a.dk = dk; a.dv = dv;
    long long sq[3], sk[3];
    fill_strides(*d, d->q, d->heads_q, tq, sq);
    fill_strides(*d, d->k, d->heads_kv, tk, sk);
    fill_strides(*d, d->v, d->heads_kv, tk, a.sv);
    fill_strides(*d, d->o, d->heads_q, tq, a.so);
    fill_strides(*d, d->dout, d->heads_q, tq, a.sdo);
    fill_strides(*d, d->dq, d->heads_q, tq, a.sdq);
    fill_strides(*d, d->dk, d->heads_kv, tk, a.sdk);
    fill_strides(*d, d->dv, d->heads_kv, tk, a.sdv);
    // without queries (or keys) the main kernels load nothing of them
    CUtensorMap tm[4] = {};
    if (tq > 0 && tk > 0 &&
        (!attn_map(&tm[0], q, *d, d->heads_q, tq, sq) || !attn_map(&tm[1], k, *d, d->heads_kv, tk, sk) ||
         !attn_map(&tm[2], v, *d, d->heads_kv, tk, a.sv) || !attn_map(&tm[3], dout, *d, d->heads_q, tq, a.sdo)))
        return CBA_ERR_UNSUPPORTED;
    cudaGetLastError();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = select_device_of(workspace);
    if (e == cudaSuccess) {
        const bool bf = d->type == CBA_BF16, slots = p.q_slots || p.k_slots;
        auto launch = [&](auto dp, auto b, auto sl) { return attn_launch<dp(), b(), sl()>(*d, p, a, tm, st); };
        auto typed = [&](auto dp, auto b) { return slots ? launch(dp, b, std::true_type{}) : launch(dp, b, std::false_type{}); };
        auto sized = [&](auto dp) { return bf ? typed(dp, std::true_type{}) : typed(dp, std::false_type{}); };
        e = p.dp == 64 ? sized(std::integral_constant<int, 64>{}) : sized(std::integral_constant<int, 128>{});
    }
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

}  // extern "C"
