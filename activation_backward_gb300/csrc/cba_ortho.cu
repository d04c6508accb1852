// cba_ortho.cu -- orthogonalising a matrix by Newton-Schulz products.
//
//   X_0 = G / (|G|_F + eps);  S = X X^T,  X <- (a I + b S + c S^2) X
// (rows <= cols; otherwise S = X^T X and X <- X (a I + b S + c S^2), the same
// polynomial of the singular values from the short side).  m = min(rows, cols), n = max.
//
// Per step three products, each one launch of ns_gemm_kernel:
//   S = X X^T                m x m, contraction n   (both operands are X)
//   C = a I + b S + c S S    m x m, contraction m   (S is symmetric: S S = S S^T)
//   X' = C X                 m x n, contraction m
// (a I inside C: one matrix less to read, and C's diagonal, a - |b| + c near the
// end, is smaller than B's, so its rounding costs no more than B's would).
// X is kept in the caller's orientation.  An operand whose contraction runs
// along its rows' elements is loaded K-major, one whose contraction runs across
// its rows M/N-major; the tensor cores take both, so nothing is transposed.
//
// Operands are f16, products accumulate in fp32: 11 significant bits where
// bf16, the usual choice for this iteration, has 8.  f16's short range is met
// with powers of two: X is held times 2^round(log2(n)/2) (its elements are of
// order 1/sqrt(n) or 1/sqrt(m n)), S times 2^12 and C times a power chosen from the
// coefficients, both with room for singular values of X up to 2 (1.2 is what
// coefficients that converge keep).
//
// The product kernel: TMA-fed tcgen05 tiles of 128 rows per block; with CG = 2
// a pair of blocks computes 256 x 256 tiles (each holds half of A's and of B's
// rows, which halves the traffic of both per product), with CG = 1 a block
// computes 128 x BN.  Persistent: two accumulators in TMEM, so the epilogue of
// one tile runs under the products of the next.  Where S has too few tiles for
// the SMs, a cluster of blocks shares a tile's contraction (ns_split_kernel).
// Warp 0 issues the TMA loads, warp 1 the MMAs, warps 2-9 the epilogue.  Every wait
// is bounded (2 s); on a timeout the block sets the workspace status bit, stops,
// waits (bounded) for copies and MMAs in flight, frees its TMEM and returns.
//
// Measured, 5 steps (us):
//   2 of 8192 x 2048  858 after a pause, 900 to 935 where calls follow each other; per step S 58,
//       C 23, X' 82: X' at 1.67 PFLOP/s, 0.98 of what cuBLAS sustains under the power limit;
//       S and C are one round of tiles over the SMs, whose beginning and end nothing covers
//   512 x 2304        106: 15 dependent launches of 5 to 9, latency
//   50 x 500          25 (a call 27), one launch: 2 in reading G, 4 to 5 a step, 2 in writing O
#include <cuda.h>

#include <algorithm>
#include <cmath>

#include "cba_internal.cuh"
#include "cba_ptx.cuh"
#include "cba_types.cuh"

namespace cba {

namespace {

constexpr uint64_t kNsLimitNs = 2000000000ull;
constexpr int kNsEpiWarps = 8;                 // two per quarter of a tile's rows
constexpr int kNsThreads = 64 + 32 * kNsEpiWarps;
constexpr int kNsStages = 6;
constexpr int kNsBK = 64;                      // contraction elements per stage (128 bytes)
constexpr float kNsSym = 4096.f;               // S is held times 2^12: room for singular values up to 2 (and 3.9)
constexpr int kNormBlocks = 512;               // partial sums of |G|^2 per matrix (at most)

struct NsArgs {
    int M, N, K;            // output rows, columns, contraction
    int mt, nt, units;      // tiles; units = batch * mt * nt
    int a_major, b_major;   // 0: K-major, 1: M- / N-major
    int sym;                // the output is symmetric: only tiles on and above the
                            // diagonal are computed, the others stored transposed
    float alpha, beta;      // out = alpha * product + beta * aux + diag * I
    float diag;
    const __half *aux;      // same shape as out, or NULL
    long long aux_ld, aux_batch;
    void *out;
    int out_type;
    long long out_ld, out_batch;
    int vec;                // 16-byte accesses to out (and aux)
    unsigned *status;
};

struct NsBars {
    uint64_t full[kNsStages], empty[kNsStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};

template <int CG, int BN>
struct NsTile {
    static constexpr int ROWS_B = BN / CG;  // B rows a block loads
    static constexpr uint32_t A_BYTES = 128u * 128u, B_BYTES = ROWS_B * 128u;
    static constexpr uint32_t STAGE = A_BYTES + B_BYTES;
    static constexpr uint32_t STAGED = kNsStages * STAGE;  // 32 rows x 32 columns of 16 bits per epilogue warp
    static constexpr uint32_t BARS = STAGED + kNsEpiWarps * 2048;
    static constexpr uint32_t SMEM = BARS + 1024 + sizeof(NsBars);
    static constexpr int TM = 128 * CG;     // tile rows
    static constexpr uint32_t TMEM_COLS = 2 * BN;
};

// `rows` rows (a multiple of 64) of one operand's stage: K-major, one box of 64
// contraction elements x rows; M/N-major, boxes of 64 rows x 64 contraction
// elements.
template <int CG>
__device__ __forceinline__ void ns_load(uint32_t dst, const CUtensorMap *tm, int major, int rows,
                                        int row0, int k0, int b, uint32_t bar) {
    auto box = [&](uint32_t to, int x, int y) {
        if constexpr (CG == 2) ptx::tma_load_3d_pair(to, tm, x, y, b, bar);
        else ptx::tma_load_3d(to, tm, x, y, b, bar);
    };
    if (major == 0) {
        box(dst, k0, row0);
    } else {
        for (int i = 0; i < rows / 64; ++i) box(dst + i * 8192, row0 + i * 64, k0);
    }
}

template <typename T, int N>
__device__ __forceinline__ void ns_store(void *out, long long at, const float (&v)[N], int n, int vec) {
    T *o = static_cast<T *>(out) + at;
    if (vec && n >= N) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < N; i += V) {
            Pack<T, V> p;
#pragma unroll
            for (int j = 0; j < V; ++j) p.v[j] = from_f32<T>(v[i + j]);
            *reinterpret_cast<Pack<T, V> *>(o + i) = p;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) o[i] = from_f32<T>(v[i]);
    }
}

// Tile u of the triangle on and above the diagonal: column j holds rows 0 .. j.
__device__ __forceinline__ void triangle(int u, int &i, int &j) {
    j = (int)((sqrtf(8.f * u + 1.f) - 1.f) * 0.5f);
    while (j * (j + 1) / 2 > u) --j;
    while ((j + 1) * (j + 2) / 2 <= u) ++j;
    i = u - j * (j + 1) / 2;
}

// 32 columns of a warp's 32 rows, through its 2 KB of shared memory, so that four
// lanes store 64 bytes of a row side by side: 32 lanes that store 16 bytes of their
// own rows take a line each (5 of 700x700 208, 264 us; 3500x4000 811, 839; 2048x2048
// alike).  `at`: of the first row; n columns, `live` rows exist.
template <typename T>
__device__ __forceinline__ void ns_store_staged(void *out, long long at, long long ld, const float (&v)[32], int live,
                                                int n, bool vec, uint8_t *stage) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        Pack<T, 8> p;
#pragma unroll
        for (int e = 0; e < 8; ++e) p.v[e] = from_f32<T>(v[8 * j + e]);
        *reinterpret_cast<Pack<T, 8> *>(stage + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)) = p;
    }
    __syncwarp();
    if (!vec) {  // rows on any address: 32 lanes store 32 elements of one (1000x2001 203 -> 180 us)
#pragma unroll 8
        for (int r = 0; r < 32; ++r) {
            const T x = *reinterpret_cast<const T *>(stage + r * 64 + (((lane >> 3) ^ (r >> 1 & 3)) << 4) + (lane & 7) * 2);
            if (r < live && lane < n) static_cast<T *>(out)[at + r * ld + lane] = x;
        }
        __syncwarp();
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + lane / 4, c = lane & 3;
        const Pack<T, 8> p = *reinterpret_cast<const Pack<T, 8> *>(stage + r * 64 + ((c ^ (r >> 1 & 3)) << 4));
        T *o = static_cast<T *>(out) + at + r * ld + 8 * c;
        if (r >= live) continue;
        if (8 * c + 8 <= n) *reinterpret_cast<Pack<T, 8> *>(o) = p;
        else
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (8 * c + e < n) o[e] = p.v[e];
    }
    __syncwarp();  // read before the next columns are written
}

// N aux values of a row, 16 bytes at a time.
template <int N>
__device__ __forceinline__ void aux_load(Pack<__half, 8> (&p)[N / 8], const __half *aux, int n) {
#pragma unroll
    for (int j = 0; j < N / 8; ++j)
        if (8 * j < n) p[j] = *reinterpret_cast<const Pack<__half, 8> *>(aux + 8 * j);  // rows are 16-byte multiples
}

// N results of one row from column `col` on (n of them in the matrix; live: the
// row is): out = alpha v + beta aux + diag I, stored, and on tiles above the
// diagonal of a symmetric matrix (mirror) also as a column.  Called by whole warps
// whose lanes hold neighbouring rows, an even one in an even lane.  `stage`: the
// warp's shared memory for 32 columns, or NULL.
template <int N>
__device__ __forceinline__ void ns_result(const NsArgs &a, float (&v)[N], const Pack<__half, 8> *aux, int b, int row,
                                          int col, bool mirror, uint8_t *stage) {
    const int n = a.N - col;
    if (n <= 0) return;
    const bool live = row < a.M;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        v[j] *= a.alpha;
        if (a.aux) v[j] = fmaf(a.beta, __half2float(aux[j / 8].v[j & 7]), v[j]);
        if (a.diag != 0.f && col + j == row) v[j] += a.diag;
    }
    if (mirror) {
        // two rows of a column are 4 bytes side by side: even lanes store even
        // columns, odd lanes odd ones (a row past M falls on the pitch's padding)
        __half *o = static_cast<__half *>(a.out) + b * a.out_batch + (row & ~1);
        const bool odd = row & 1;
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
            const __half2 h = odd ? __floats2half2_rn(got, v[j + 1]) : __floats2half2_rn(v[j], got);
            if ((row & ~1) < a.M && j + odd < n) *reinterpret_cast<__half2 *>(o + (col + j + odd) * a.out_ld) = h;
        }
    }
    if constexpr (N == 32) {
        if (stage && a.out_type != CBA_F32) {
            const int first = row - (int)(threadIdx.x & 31);
            const long long at = b * a.out_batch + first * a.out_ld + col;
            if (a.out_type == CBA_F16) ns_store_staged<__half>(a.out, at, a.out_ld, v, a.M - first, n, a.vec, stage);
            else ns_store_staged<__nv_bfloat16>(a.out, at, a.out_ld, v, a.M - first, n, a.vec, stage);
            return;
        }
    }
    if (!live) return;
    const long long at = b * a.out_batch + row * a.out_ld + col;
    if (a.out_type == CBA_F16) ns_store<__half>(a.out, at, v, n, a.vec);
    else if (a.out_type == CBA_BF16) ns_store<__nv_bfloat16>(a.out, at, v, n, a.vec);
    else ns_store<float>(a.out, at, v, n, a.vec);
}

template <int CG, int BN>
__global__ void __launch_bounds__(kNsThreads, 1)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                   const NsArgs a) {
    using L = NsTile<CG, BN>;
    extern __shared__ uint8_t smem_dyn[];
    // both blocks of a pair round up alike: the same kernel, the same layout
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    NsBars &sb = *reinterpret_cast<NsBars *>(smem + L::BARS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? ptx::cluster_ctarank() : 0;
    if (tid == 0) {
        for (int i = 0; i < kNsStages; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sb.full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sb.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sb.acc_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sb.acc_empty[i]), kNsEpiWarps * CG);
        }
        ptx::mbar_init(ptx::smem_u32(&sb.drain), 1);
        sb.abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            ptx::tmem_alloc_pair(ptx::smem_u32(&sb.tmem_base), L::TMEM_COLS);
        } else {
            ptx::tmem_alloc(ptx::smem_u32(&sb.tmem_base), L::TMEM_COLS);
            ptx::tmem_relinquish();
        }
    }
    ptx::tc_fence_before();
    if constexpr (CG == 2) ptx::cluster_sync();
    else __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sb.tmem_base;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const int g0 = (int)blockIdx.x / CG, gstep = (int)gridDim.x / CG;
    const int nk = (a.K + kNsBK - 1) / kNsBK;
    const int mine = a.units > g0 ? (a.units - 1 - g0) / gstep + 1 : 0;
    volatile int *ab = &sb.abort_flag;
    // unit -> batch, tile row, tile column; tile rows fastest, so that blocks
    // running together share B's rows in L2
    auto where = [&](int i, int &b, int &m0, int &n0) {
        int u = g0 + i * gstep;
        if (a.sym) {
            const int tri = a.mt * (a.mt + 1) / 2;
            b = u / tri;
            u -= b * tri;
            int ti, tj;
            triangle(u, ti, tj);
            m0 = ti * L::TM;
            n0 = tj * BN;
            return;
        }
        m0 = u % a.mt * L::TM;
        u /= a.mt;
        n0 = u % a.nt * BN;
        b = u / a.nt;
    };

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            int gs = 0;
            for (int i = 0; ok && i < mine; ++i) {
                int b, m0, n0;
                where(i, b, m0, n0);
                const int ar = m0 + (int)rank * 128, br = n0 + (int)rank * L::ROWS_B;
                for (int kb = 0; kb < nk; ++kb, ++gs) {
                    const int s = gs % kNsStages;
                    if (gs >= kNsStages)
                        ok = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.empty[s]),
                                                    (uint32_t)(gs / kNsStages - 1) & 1u, ab, a.status, kNsLimitNs);
                    if (!ok) break;
                    uint32_t bar = ptx::smem_u32(&sb.full[s]);
                    // the pair's copies all complete on the even block's barrier
                    if (rank == 0) ptx::mbar_arrive_expect_tx(bar, CG * L::STAGE);
                    if constexpr (CG == 2) bar = ptx::mapa(bar, 0);
                    const uint32_t to = ptx::smem_u32(smem + s * L::STAGE);
                    ns_load<CG>(to, &ta, a.a_major, 128, ar, kb * kNsBK, b, bar);
                    ns_load<CG>(to + L::A_BYTES, &tb, a.b_major, L::ROWS_B, br, kb * kNsBK, b, bar);
                }
            }
            if (!ok && rank == 0) {  // no copy may be in flight when the block exits
                int no = 0;
                for (int v = max(0, gs - kNsStages); v < gs; ++v)
                    ptx::mbar_wait_bounded(ptx::smem_u32(&sb.full[v % kNsStages]),
                                           (uint32_t)(v / kNsStages) & 1u, &no, a.status, kNsLimitNs / 8);
            }
        }
    } else if (warp == 1) {
        // the whole warp walks the loop and one elected lane issues (descriptors and
        // counters are then uniform over the warp: half the issue time per MMA)
        if (rank == 0) {
            const uint32_t idesc = ptx::idesc_f16(L::TM, BN, false, a.b_major != 0, a.a_major != 0);
            // 16-byte units of one K = 16 step
            const uint32_t sa = a.a_major ? 2048 >> 4 : 32 >> 4, sbk = a.b_major ? 2048 >> 4 : 32 >> 4;
            auto commit = [&](uint64_t *bar) {
                if constexpr (CG == 2) ptx::mma_commit_pair(ptx::smem_u32(bar));
                else ptx::mma_commit(ptx::smem_u32(bar));
            };
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                const bool r = ptx::mbar_wait_bounded(ptx::smem_u32(bar), parity, ab, a.status, kNsLimitNs);
                ptx::tc_fence_after();
                return __all_sync(0xffffffffu, r) != 0;
            };
            bool ok = true;
            int s = 0;
            uint32_t ph = 0;
            for (int i = 0; ok && i < mine; ++i) {
                const int ac = i & 1;
                if (i >= 2 && !(ok = wait(&sb.acc_empty[ac], (uint32_t)(i / 2 - 1) & 1u))) break;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!(ok = wait(&sb.full[s], ph))) break;
                    const uint32_t at = ptx::smem_u32(smem + s * L::STAGE);
                    const ptx::Desc da = ptx::desc_of(at, a.a_major ? 8192 : 16, 1024, 2);
                    const ptx::Desc db = ptx::desc_of(at + L::A_BYTES, a.b_major ? 8192 : 16, 1024, 2);
                    if (ptx::elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < kNsBK / 16; ++ks) {
                            const uint32_t acc = (kb > 0 || ks > 0) ? 1u : 0u;
                            if constexpr (CG == 2)
                                ptx::mma_f16_pair(tmem + ac * BN, da, ks * sa, db, ks * sbk, idesc, acc);
                            else
                                ptx::mma_f16(tmem + ac * BN, da, ks * sa, db, ks * sbk, idesc, acc);
                        }
                        commit(&sb.empty[s]);
                        if (kb + 1 == nk) commit(&sb.acc_full[ac]);
                    }
                    __syncwarp();
                    if (++s == kNsStages) s = 0, ph ^= 1;
                }
            }
            // every MMA issued has finished before TMEM is released
            if (ptx::elect_one()) {
                if (!ok) *ab = 1;
                commit(&sb.drain);
            }
            __syncwarp();
            int no = 0;
            ptx::mbar_wait_bounded(ptx::smem_u32(&sb.drain), 0, &no, a.status, kNsLimitNs);
            __syncwarp();
        }
    } else {
        const int quarter = warp & 3, c0 = (warp - 2) / 4 * (BN / 2);
        bool ok = true;
        for (int i = 0; ok && i < mine; ++i) {
            const int ac = i & 1;
            int b, m0, n0;
            where(i, b, m0, n0);
            const int row = m0 + (int)rank * 128 + quarter * 32 + lane;
            const __half *aux = a.aux ? a.aux + b * a.aux_batch + min(row, a.M - 1) * a.aux_ld + n0 + c0 : nullptr;
            Pack<__half, 8> ax[4];  // 32 columns ahead (all of them while the products run: C 1 us slower)
            if (aux) aux_load<32>(ax, aux, a.N - n0 - c0);
            ok = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.acc_full[ac]), (uint32_t)(i / 2) & 1u, ab, a.status,
                                        kNsLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t t0 = tmem + ((uint32_t)(quarter * 32) << 16) + ac * BN + c0;
#pragma unroll 1
            for (int c = 0; c < BN / 2; c += 32) {
                float v[32];
                __syncwarp();  // rows past M skip the stores
                ptx::tmem_ld32(t0 + c, v);
                ptx::tmem_ld_wait();
                if (c + 32 == BN / 2) {  // the accumulator is read: the MMAs may reuse it
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 2)
                            ptx::mbar_arrive_cluster(ptx::mapa(ptx::smem_u32(&sb.acc_empty[ac]), 0));
                        else
                            ptx::mbar_arrive(ptx::smem_u32(&sb.acc_empty[ac]));
                    }
                }
                ns_result<32>(a, v, ax, b, row, n0 + c0 + c, a.sym && m0 < n0, smem + L::STAGED + (warp - 2) * 2048);
                if (aux && c + 32 < BN / 2) aux_load<32>(ax, aux + c + 32, a.N - n0 - c0 - c - 32);
            }
        }
    }
    ptx::tc_fence_before();
    if constexpr (CG == 2) ptx::cluster_sync();  // the peer's arrivals on this block's barriers are done
    else __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        if constexpr (CG == 2) ptx::tmem_dealloc_pair(tmem, L::TMEM_COLS);
        else ptx::tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

// ---- a tile's contraction shared by a cluster

// D[128 x 128] of a symmetric product: block `rank` of a cluster of SK contracts
// every SK-th part, leaves its fp32 sums in its shared memory ([column / 4][row]
// float4), and adds up 128 / SK of the columns of all blocks, in the order of
// the ranks.  (S of 512 x 2304: ten tiles, whose 36 stages a block alone loads at
// ~100 GB/s in 9 us.)
template <int SK>
__global__ void __launch_bounds__(kNsThreads, 1)
    ns_split_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                    const NsArgs a) {
    using L = NsTile<1, 128>;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    NsBars &sb = *reinterpret_cast<NsBars *>(smem + kNsStages * L::STAGE);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)ptx::cluster_ctarank();
    if (tid == 0) {
        for (int i = 0; i < kNsStages; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sb.full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sb.empty[i]), 1);
        }
        ptx::mbar_init(ptx::smem_u32(&sb.acc_full[0]), 1);
        sb.abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&sb.tmem_base), 128);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sb.tmem_base;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    int u = (int)blockIdx.x / SK;
    const int tri = a.mt * (a.mt + 1) / 2, b = u / tri;
    int ti, tj;
    triangle(u - b * tri, ti, tj);
    const int m0 = ti * 128, n0 = tj * 128;
    const int nk = (a.K + kNsBK - 1) / kNsBK, k0 = nk * rank / SK, k1 = nk * (rank + 1) / SK;
    volatile int *ab = &sb.abort_flag;
    bool ok = true;
    int begun = 0;  // stages that lane 0 of the load warp has begun to fill
    if (warp == 0) {
        if (lane == 0)
            for (int kb = k0; kb < k1; ++kb, ++begun) {
                const int s = begun % kNsStages;
                if (begun >= kNsStages)
                    ok = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.empty[s]), (uint32_t)(begun / kNsStages - 1) & 1u, ab,
                                                a.status, kNsLimitNs);
                if (!ok) break;
                const uint32_t bar = ptx::smem_u32(&sb.full[s]), to = ptx::smem_u32(smem + s * L::STAGE);
                ptx::mbar_arrive_expect_tx(bar, L::STAGE);
                ns_load<1>(to, &ta, a.a_major, 128, m0, kb * kNsBK, b, bar);
                ns_load<1>(to + L::A_BYTES, &tb, a.b_major, 128, n0, kb * kNsBK, b, bar);
            }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t idesc = ptx::idesc_f16(128, 128, false, a.b_major != 0, a.a_major != 0);
        const uint32_t sa = a.a_major ? 2048 >> 4 : 32 >> 4, sbk = a.b_major ? 2048 >> 4 : 32 >> 4;
        int s = 0;
        uint32_t ph = 0;
        for (int kb = k0; kb < k1; ++kb) {
            const bool r = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.full[s]), ph, ab, a.status, kNsLimitNs);
            ptx::tc_fence_after();
            if (!(ok = __all_sync(0xffffffffu, r))) break;
            const uint32_t at = ptx::smem_u32(smem + s * L::STAGE);
            const ptx::Desc da = ptx::desc_of(at, a.a_major ? 8192 : 16, 1024, 2);
            const ptx::Desc db = ptx::desc_of(at + L::A_BYTES, a.b_major ? 8192 : 16, 1024, 2);
            if (ptx::elect_one()) {
#pragma unroll
                for (int ks = 0; ks < kNsBK / 16; ++ks)
                    ptx::mma_f16(tmem, da, ks * sa, db, ks * sbk, idesc, kb > k0 || ks > 0);
                ptx::mma_commit(ptx::smem_u32(&sb.empty[s]));
            }
            __syncwarp();
            if (++s == kNsStages) s = 0, ph ^= 1;
        }
        if (ptx::elect_one()) {
            if (!ok) *ab = 1;
            ptx::mma_commit(ptx::smem_u32(&sb.acc_full[0]));
        }
        __syncwarp();
    }
    // every thread: the products are done (and with them the copies), so that the
    // stages may hold the sums; a block that timed out leaves nothing to be added
    int no = 0;
    bool done = ptx::mbar_wait_bounded(ptx::smem_u32(&sb.acc_full[0]), 0, &no, a.status, kNsLimitNs);
    done = __syncthreads_and(done && *ab == 0) != 0;
    ptx::tc_fence_after();
    if (!done)  // copies that no product waited for
        for (int v = max(0, begun - kNsStages); v < begun; ++v)
            ptx::mbar_wait_bounded(ptx::smem_u32(&sb.full[v % kNsStages]), (uint32_t)(v / kNsStages) & 1u, &no, a.status,
                                   kNsLimitNs / 8);
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    float4 *sums = reinterpret_cast<float4 *>(smem);
    if (warp >= 2 && done) {
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
            float v[16];
            ptx::tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + half * 64 + c, v);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                sums[(half * 64 + c + j) / 4 * 128 + quarter * 32 + lane] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
    }
    ptx::cluster_sync();
    if (warp >= 2) {
        constexpr int COLS = 128 / SK, PER = COLS / 2 < 8 ? 8 : COLS / 2;  // of a rank, of a warp
        const int c0 = rank * COLS + half * PER, row = quarter * 32 + lane;
        if (half * PER < COLS) {
#pragma unroll
            for (int c = 0; c < PER; c += 8) {
                float v[8] = {};
#pragma unroll
                for (int q = 0; q < SK; ++q) {
                    const uint32_t from = ptx::mapa(ptx::smem_u32(sums + (c0 + c) / 4 * 128 + row), (uint32_t)q);
                    const float4 x = ptx::ld_cluster(from), y = ptx::ld_cluster(from + 128 * 16);
                    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                    v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
                }
                __syncwarp();
                ns_result<8>(a, v, nullptr, b, m0 + row, n0 + c0 + c, m0 < n0, nullptr);
            }
        }
    }
    ptx::cluster_sync();  // the others have read this block's sums
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 128);
    }
}

// ---- |G|^2 and the scaled f16 copy

// The sum of `v` over a block of 256 threads, in thread 0 (fixed order).
__device__ __forceinline__ double block_sum(double v, double *sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
#pragma unroll
        for (int i = 1; i < 8; ++i) v += sm[i];
    return v;
}

// Partial sums of squares: block (p, b) takes the p-th part of matrix b's 16-byte
// vectors (VEC elements; 1 where rows are not whole vectors), summed in a fixed
// order: 4 vectors in fp32 (in fp64 where that overflows), their sums in fp64.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
    ns_norm_kernel(const T *g, int rows, int cols, long long ld, long long batch_stride, double *part) {
    __shared__ double sm[8];
    ptx::griddep_launch_dependents();
    const T *gb = g + (long long)blockIdx.y * batch_stride;
    const bool flat = ld == cols;
    const long long per_row = cols / VEC, n = per_row * rows;
    const long long per = (n + gridDim.x - 1) / gridDim.x;
    const long long e1 = min(n, (blockIdx.x + 1) * per);
    double total = 0.0;
    for (long long e = blockIdx.x * per + threadIdx.x; e < e1; e += 4 * 256) {
        Pack<T, VEC> p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long i = e + j * 256;
            if (i < e1) {
                const long long r = flat ? 0 : i / per_row;
                p[j] = *reinterpret_cast<const Pack<T, VEC> *>(gb + (flat ? i * VEC : r * ld + (i - r * per_row) * VEC));
            }
        }
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e + j * 256 < e1)
#pragma unroll
                for (int k = 0; k < VEC; ++k) s = fmaf(to_f32(p[j].v[k]), to_f32(p[j].v[k]), s);
        if (s < INFINITY) {
            total += s;
        } else {  // elements past 1e19, or an infinity or NaN
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (e + j * 256 < e1)
#pragma unroll
                    for (int k = 0; k < VEC; ++k) total += (double)to_f32(p[j].v[k]) * to_f32(p[j].v[k]);
        }
    }
    total = block_sum(total, sm);
    if (threadIdx.x == 0) part[(long long)blockIdx.y * kNormBlocks + blockIdx.x] = total;
}

// X = G * (held / (|G| + eps)) in f16, rows `pitch` apart (the padding is never
// read: the maps end at cols).  One warp per row, strided.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
    ns_cast_kernel(const T *g, int rows, int cols, long long ld, long long batch_stride, const double *part,
                   int nparts, float eps, float held, __half *x, long long pitch, long long x_batch,
                   unsigned *status) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    __shared__ float f;
    const int b = blockIdx.y;
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (int i = threadIdx.x; i < nparts; i += 32) s += part[(long long)b * kNormBlocks + i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) f = (float)((double)held / (sqrt(s) + (double)eps));
    }
    if (blockIdx.x == 0 && b == 0 && threadIdx.x == 0) *status = 0;
    __syncthreads();
    const float k = f;
    const int lane = threadIdx.x & 31;
    for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += gridDim.x * 8) {
        const T *src = g + b * batch_stride + r * ld;
        __half *dst = x + b * x_batch + r * pitch;
        constexpr int N = VEC == 1 ? 8 : 4;  // loads ahead of the stores
        for (int c0 = lane * VEC; c0 < cols; c0 += N * 32 * VEC) {
            Pack<T, VEC> p[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = c0 + i * 32 * VEC;
                if (c < cols) p[i] = *reinterpret_cast<const Pack<T, VEC> *>(src + c);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = c0 + i * 32 * VEC;
                Pack<__half, VEC> o;
#pragma unroll
                for (int j = 0; j < VEC; ++j) o.v[j] = __float2half_rn(to_f32(p[i].v[j]) * k);
                if (c < cols) *reinterpret_cast<Pack<__half, VEC> *>(dst + c) = o;
            }
        }
    }
}

// ---- one block per matrix: all steps in shared memory

// For m <= 128, X [R][n] (R = 64 or 128 rows, zero padded) stays in shared
// memory in boxes of R rows x 64 columns with the 128-byte swizzle: as rows it
// is the K-major operand of S = X X^T, as columns the N-major operand of C X.
// Each 256-column chunk of X' depends on that chunk of X alone, so X is replaced
// chunk by chunk.  TMEM holds two accumulators of a chunk: the next chunk's product
// runs while one is read back, and the one that the last chunk leaves free takes
// the next step's S, begun over the finished chunks.  The MMAs have M = 128 rows;
// with R = 64 the upper 64 lanes compute with whatever lies behind the operand and
// are not read.  A tall matrix is transposed on its way in and out.
// Bound by the chain of small products and barriers, not by a rate: 50 x 500 takes
// 47,000 cycles (24 us), 7,000 of them to read G and 7,500 a step; 128 x 576
// 85,000 (44 us).  Before the products of chunks ran ahead: 77,000 and 118,000.
// (1024 threads: each phase is slower by its barriers.)
constexpr int kSmThreads = 512;
constexpr size_t kSmMax = 227 * 1024;

struct SmBars {
    uint64_t sq, x[2], drain;
    uint32_t tmem_base;
    int abort_flag;
    float factor;
    double part[kSmThreads / 32];
};

struct SmArgs {
    const void *G;
    void *O;
    int rows, cols, m, n, steps;
    int wide, R, nb;              // nb: 64-column boxes of X
    int in_type, out_type;
    long long ld_in, batch_in, ld_out, batch_out;
    float a, b, c;                // of C as held, from I, from S and S S as held
    float eps, scale, held, c_held;
    unsigned *status;
};

size_t small_smem(int R, int nb) {
    return (size_t)nb * R * 128 + 2 * (size_t)(R / 64) * R * 128 + (R == 64 ? 8192 : 0) + sizeof(SmBars) + 1024;
}

// Byte offset of elements 8 c8 .. 8 c8 + 7 of row r in boxes of R rows.
__device__ __forceinline__ uint32_t box_at(int R, int r, int c8) {
    return (uint32_t)((c8 >> 3) * R * 128 + r * 128 + (((c8 & 7) ^ (r & 7)) << 4));
}

// The sum of squares of a thread's share of `n` packs of VEC elements, `per_row`
// packs to a row (flat: one row), 8 loads in flight; in fp64 where fp32 overflows.
template <typename T, int VEC>
__device__ __forceinline__ double small_squares(const T *g, int n, int per_row, long long ld, bool flat) {
    float s = 0.f;
    for (int e = threadIdx.x; e < n; e += 8 * kSmThreads) {
        Pack<T, VEC> p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = e + j * kSmThreads;
#pragma unroll
            for (int k = 0; k < VEC; ++k) p[j].v[k] = from_f32<T>(0.f);
            if (i < n) {
                const int r = flat ? 0 : i / per_row;
                p[j] = *reinterpret_cast<const Pack<T, VEC> *>(g + r * ld + (long long)(i - r * per_row) * VEC);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int k = 0; k < VEC; ++k) s = fmaf(to_f32(p[j].v[k]), to_f32(p[j].v[k]), s);
    }
    if (s < INFINITY) return s;
    double big = 0.0;  // elements past 1e19, or an infinity or NaN
    for (int e = threadIdx.x; e < n; e += kSmThreads) {
        const int r = flat ? 0 : e / per_row;
        const T *x = g + r * ld + (long long)(e - r * per_row) * VEC;
        for (int k = 0; k < VEC; ++k) big += (double)to_f32(x[k]) * to_f32(x[k]);
    }
    return big;
}

// Rows of a wide G, scaled, as the boxes' rows: a warp per row, W elements a time,
// 8 loads in flight.
template <typename T, int W>
__device__ __forceinline__ void small_rows(const SmArgs &a, const T *g, uint8_t *sx, float k) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int c0 = lane * W; c0 < a.nb * 64; c0 += 64 * W)
        for (int r0 = warp; r0 < a.R; r0 += kSmThreads / 8) {
            Pack<T, W> v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = r0 + (i >> 1) * (kSmThreads / 32), c = c0 + (i & 1) * 32 * W;
#pragma unroll
                for (int j = 0; j < W; ++j) v[i].v[j] = from_f32<T>(0.f);
                if (r < a.m && c < a.n) v[i] = *reinterpret_cast<const Pack<T, W> *>(g + r * a.ld_in + c);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // R is a multiple of the 64 rows that a pass covers
                const int r = r0 + (i >> 1) * (kSmThreads / 32), c = c0 + (i & 1) * 32 * W;
                Pack<__half, W> p;
#pragma unroll
                for (int j = 0; j < W; ++j) p.v[j] = __float2half_rn(to_f32(v[i].v[j]) * k);
                if (c < a.nb * 64)
                    *reinterpret_cast<Pack<__half, W> *>(sx + box_at(a.R, r, c >> 3) + (c & 7) * 2) = p;
            }
        }
}

// |G|^2 and the scaled, zero-padded f16 copy.  G is read twice, the second time
// from L1 or L2.
template <typename T>
__device__ __forceinline__ void small_load(const SmArgs &a, const T *g, uint8_t *sx, SmBars &sb) {
    const int tid = threadIdx.x;
    const int n = a.rows * a.cols;
    const bool flat = a.ld_in == a.cols;
    constexpr int V = 16 / sizeof(T);
    double total = flat && n % V == 0 && aligned_to(g, 16) ? small_squares<T, V>(g, n / V, n / V, 0, true)
                                                           : small_squares<T, 1>(g, n, a.cols, a.ld_in, flat);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if ((tid & 31) == 0) sb.part[tid >> 5] = total;
    __syncthreads();
    if (tid < 32) {
        double s = tid < kSmThreads / 32 ? sb.part[tid] : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (tid == 0) sb.factor = (float)((double)a.held / (sqrt(s) + (double)a.eps));
    }
    __syncthreads();
    const float k = sb.factor;
    // neighbouring threads read neighbouring elements of G
    if (a.wide) {
        if (aligned_to(g, 4 * sizeof(T)) && a.ld_in % 4 == 0 && a.n % 4 == 0) small_rows<T, 4>(a, g, sx, k);
        else small_rows<T, 1>(a, g, sx, k);
        return;
    }
#pragma unroll 2
    for (int i = tid; i < a.R * a.nb * 8; i += kSmThreads) {  // 8 of a column of G
        const int r = i % a.R, c8 = i / a.R;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c8 * 8 + j;
            v[j] = r < a.m && c < a.n ? to_f32(g[c * a.ld_in + r]) : 0.f;
        }
        Pack<__half, 8> p;
#pragma unroll
        for (int j = 0; j < 8; ++j) p.v[j] = __float2half_rn(v[j] * k);
        *reinterpret_cast<Pack<__half, 8> *>(sx + box_at(a.R, r, c8)) = p;
    }
}

// 32 values of row r as elements c .. c + 31 of boxes of R rows.
template <typename H, int N>
__device__ __forceinline__ void box_put(uint8_t *to, int R, int r, int c, const float (&v)[N]) {
#pragma unroll
    for (int q = 0; q < N / 8; ++q) {
        Pack<H, 8> p;
#pragma unroll
        for (int e = 0; e < 8; ++e) p.v[e] = from_f32<H>(v[q * 8 + e]);
        *reinterpret_cast<Pack<H, 8> *>(to + box_at(R, r, c / 8 + q)) = p;
    }
}

// One thread's 32 results of row r: neighbouring threads hold neighbouring rows,
// which lie side by side in a tall O.
template <typename T>
__device__ __forceinline__ void small_store(const SmArgs &a, T *o, const float (&v)[32], int r, int c0) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (c0 + j < a.n) o[a.wide ? r * a.ld_out + c0 + j : (c0 + j) * a.ld_out + r] = from_f32<T>(v[j]);
}

// A wide O's rows from the finished chunk, which the threads put back into its
// boxes in O's 16-bit type: a warp per row, W elements at a time.
template <typename T, int W>
__device__ __forceinline__ void small_copy_by(const SmArgs &a, T *o, const uint8_t *sx, int c0, int cols) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = warp; r < a.m; r += kSmThreads / 32)
#pragma unroll 2
        for (int c = c0 + lane * W; c < c0 + cols; c += 32 * W)
            *reinterpret_cast<Pack<T, W> *>(o + r * a.ld_out + c) =
                *reinterpret_cast<const Pack<T, W> *>(sx + box_at(a.R, r, c >> 3) + (c & 7) * 2);
}
template <typename T>
__device__ __forceinline__ void small_copy(const SmArgs &a, T *o, const uint8_t *sx, int c0, int cols) {
    if (aligned_to(o, 8) && a.ld_out % 4 == 0 && cols % 4 == 0) small_copy_by<T, 4>(a, o, sx, c0, cols);
    else small_copy_by<T, 1>(a, o, sx, c0, cols);
}

__device__ __forceinline__ void tmem_ld(uint32_t t, float (&v)[32]) { ptx::tmem_ld32(t, v); }
__device__ __forceinline__ void tmem_ld(uint32_t t, float (&v)[16]) { ptx::tmem_ld16(t, v); }

template <int R>
__global__ void __launch_bounds__(kSmThreads, 1) ns_small_kernel(const SmArgs a) {
    extern __shared__ uint8_t smem_dyn[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    constexpr uint32_t box = R * 128;
    uint8_t *sx = smem, *ss = sx + a.nb * box, *sc = ss + (R / 64) * box;
    SmBars &sb = *reinterpret_cast<SmBars *>(sc + (R / 64) * box + (R == 64 ? 8192 : 0));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (uint64_t *b : {&sb.sq, &sb.x[0], &sb.x[1], &sb.drain}) ptx::mbar_init(ptx::smem_u32(b), 1);
        sb.abort_flag = 0;
        ptx::fence_mbar_init();
        if (gridDim.x == 1) *a.status = 0;
    }
    if (warp == 0) {
        ptx::tmem_alloc(ptx::smem_u32(&sb.tmem_base), 512);
        ptx::tmem_relinquish();
    }
    const long long b = blockIdx.x;
    if (a.in_type == CBA_F32) small_load(a, static_cast<const float *>(a.G) + b * a.batch_in, sx, sb);
    else if (a.in_type == CBA_F16) small_load(a, static_cast<const __half *>(a.G) + b * a.batch_in, sx, sb);
    else small_load(a, static_cast<const __nv_bfloat16 *>(a.G) + b * a.batch_in, sx, sb);
    // Everything that the tensor cores read was written by these threads.  A wait
    // that ran out shows at the next publish, to all threads at once.
    bool ok = true;
    auto publish = [&]() {
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ok = __syncthreads_and(ok) != 0;
        ptx::tc_fence_after();
        return ok;
    };
    publish();
    const uint32_t tmem = sb.tmem_base, uX = ptx::smem_u32(sx), uS = ptx::smem_u32(ss), uC = ptx::smem_u32(sc);
    constexpr uint32_t id_s = ptx::idesc_f16(128, R, false, false);
    const int km = (a.m + 15) / 16, kn = (a.n + 15) / 16;
    // 16 warps: the quarter of the rows that TMEM lets a warp read, and one of
    // four column parts
    const int quarter = warp & 3, part = warp >> 2, r = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const bool mine = quarter * 32 < R;  // this warp's rows exist
    constexpr int issuer = R == 64 ? 2 : 0;  // of the MMAs: a warp without rows, if there is one
    constexpr int CS = R / 4;            // S columns per thread
    const int c_s = part * CS, nchunks = (a.nb + 3) / 4;
    const uint32_t tS = tmem + (nchunks & 1) * 256, tQ = tS + 128;
    const float s_alpha = kNsSym / (a.held * a.held);
    volatile int *ab = &sb.abort_flag;
    uint32_t ph_x = 0;  // a bit for each chunk in flight
    auto wait = [&](uint64_t *bar, uint32_t phase) {
        ok = ptx::mbar_wait_bounded(ptx::smem_u32(bar), phase, ab, a.status, kNsLimitNs) && ok;
        ptx::tc_fence_after();
    };
    // D (+)= U U^T, R columns, the K steps k0 .. k1 - 1 of U's ksteps
    auto product = [&](uint32_t d, uint32_t u, int k0, int k1, int ksteps) {
        const ptx::Desc de = ptx::desc_of(u, 16, 1024, 2);
        if (ptx::elect_one()) {
#pragma unroll 4
            for (int ks = k0; ks < min(k1, ksteps); ++ks) {
                const uint32_t off = ((ks >> 2) * box + (ks & 3) * 32) >> 4;
                ptx::mma_f16(d, de, off, de, off, id_s, ks > 0);
            }
            if (k1 >= ksteps) ptx::mma_commit(ptx::smem_u32(&sb.sq));
        }
        __syncwarp();
    };
    auto apply = [&](int ch) {  // the 256 columns of X' from box 4 ch on
        const uint32_t id = ptx::idesc_f16(128, 64 * min(4, a.nb - 4 * ch), false, true);
        const ptx::Desc dc = ptx::desc_of(uC, 16, 1024, 2), dx = ptx::desc_of(uX + 4 * ch * box, box, 1024, 2);
        if (ptx::elect_one()) {
#pragma unroll 4
            for (int ks = 0; ks < km; ++ks)
                ptx::mma_f16(tmem + (ch & 1) * 256, dc, ((ks >> 2) * box + (ks & 3) * 32) >> 4, dx, ks * (2048 >> 4),
                             id, ks > 0);
            ptx::mma_commit(ptx::smem_u32(&sb.x[ch & 1]));
        }
        __syncwarp();
    };
    if (warp == issuer) product(tS, uX, 0, kn, kn);
    for (int step = 0; step < a.steps; ++step) {
        wait(&sb.sq, 0);
        float s[CS];
        if (mine) {
            tmem_ld(tS + lanes + c_s, s);
            ptx::tmem_ld_wait();
            // b S takes S as rounded too: C is then the polynomial of one matrix, and near 1 an
            // error of S moves it by b + 2 c = -0.7 of itself instead of b (50x500: 2.1e-3 -> 1e-3)
#pragma unroll
            for (int j = 0; j < CS; ++j) s[j] = __half2float(__float2half_rn(s[j] * s_alpha));
            box_put<__half>(ss, R, r, c_s, s);
        }
        if (!publish()) break;
        if (warp == issuer) product(tQ, uS, 0, km, km);
        wait(&sb.sq, 1);
        if (mine) {
            float q[CS];
            tmem_ld(tQ + lanes + c_s, q);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < CS; ++j) {
                q[j] = fmaf(a.c, q[j], a.b * s[j]);
                if (c_s + j == r) q[j] += a.a;
            }
            box_put<__half>(sc, R, r, c_s, q);
        }
        if (!publish()) break;
        const bool last = step + 1 == a.steps;
        const float alpha = (last ? a.scale / a.held : 1.f) / a.c_held;
        if (warp == issuer)
            for (int ch = 0; ch < min(2, nchunks); ++ch) apply(ch);
        for (int ch = 0; ch < nchunks; ++ch) {
            wait(&sb.x[ch & 1], ph_x >> (ch & 1) & 1);
            ph_x ^= 1u << (ch & 1);
            if (mine)
                for (int i = part; i < 2 * min(4, a.nb - 4 * ch); i += 4) {
                    const int c0 = ch * 256 + i * 32;
                    float v[32];
                    ptx::tmem_ld32(tmem + (ch & 1) * 256 + lanes + i * 32, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] *= alpha;
                    if (!last) {
                        box_put<__half>(sx, R, r, c0, v);
                    } else if (a.out_type == CBA_F32) {
                        if (r < a.m) small_store(a, static_cast<float *>(a.O) + b * a.batch_out, v, r, c0);
                    } else if (a.out_type == CBA_F16) {
                        if (a.wide) box_put<__half>(sx, R, r, c0, v);
                        else if (r < a.m) small_store(a, static_cast<__half *>(a.O) + b * a.batch_out, v, r, c0);
                    } else {
                        if (a.wide) box_put<__nv_bfloat16>(sx, R, r, c0, v);
                        else if (r < a.m) small_store(a, static_cast<__nv_bfloat16 *>(a.O) + b * a.batch_out, v, r, c0);
                    }
                }
            if (!publish()) break;
            if (warp == issuer) {
                if (ch + 2 < nchunks) apply(ch + 2);
                else if (!last) product(tS, uX, ch + 1 < nchunks || nchunks == 1 ? 0 : 16 * ch, 16 * ch + 16, kn);
            }
            if (last && a.wide && a.out_type != CBA_F32) {
                const int cols = min(256, a.n - 256 * ch);
                if (a.out_type == CBA_F16)
                    small_copy(a, static_cast<__half *>(a.O) + b * a.batch_out, sx, 256 * ch, cols);
                else
                    small_copy(a, static_cast<__nv_bfloat16 *>(a.O) + b * a.batch_out, sx, 256 * ch, cols);
            }
        }
        if (!ok) break;
    }
    // on a timeout MMAs may still be in flight: wait (bounded) for all of them
    if (!ok && tid == issuer * 32) {
        int no = 0;
        ptx::mma_commit(ptx::smem_u32(&sb.drain));
        ptx::mbar_wait_bounded(ptx::smem_u32(&sb.drain), 0, &no, a.status, kNsLimitNs);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ---- host side

// The power of two by which C = a I + b S + c S^2 is held in f16: its eigenvalues
// for singular values up to 2 stay below half of the largest f16.
float c_power(const cba_orthogonalize_desc_t &d) {
    auto p = [&](double t) { return std::fabs(d.a + t * ((double)d.b + t * d.c)); };
    double most = std::max(p(0.0), p(4.0));
    const double turn = d.c != 0.f ? -0.5 * d.b / d.c : 0.0;
    if (turn > 0.0 && turn < 4.0) most = std::max(most, p(turn));
    int e = 0;
    std::frexp(most, &e);  // most < 2^e
    return std::ldexp(1.f, std::min(12, std::max(15 - e, -64)));
}

struct NsPlan {
    int m, n;
    bool wide;                 // rows <= cols
    long long x_pitch, s_pitch;
    long long x_batch, s_batch;  // elements of one matrix
    size_t off_part, off_x0, off_x1, off_s, off_c, total;
};

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

int check_ns(const cba_orthogonalize_desc_t *d, NsPlan *p) {
    if (!d || d->batch < 1 || d->rows < 1 || d->cols < 1 || d->steps < 1) return CBA_ERR_ARG;
    if (!dtype_ok(d->in_type) || !dtype_ok(d->out_type)) return CBA_ERR_ARG;
    if (!std::isfinite(d->a) || !std::isfinite(d->b) || !std::isfinite(d->c) || !std::isfinite(d->scale) ||
        !(std::isfinite(d->eps) && d->eps >= 0.f))
        return CBA_ERR_ARG;
    const long long need = (long long)d->rows * d->cols;
    if ((d->ld_in != 0 && d->ld_in < d->cols) || (d->ld_out != 0 && d->ld_out < d->cols)) return CBA_ERR_ARG;
    const long long ldi = d->ld_in ? d->ld_in : d->cols, ldo = d->ld_out ? d->ld_out : d->cols;
    if (d->steps > 100 || d->rows > (1 << 20) || d->cols > (1 << 20) || d->batch > 65535 || need >= (1LL << 36) ||
        ldi >= (1LL << 31) || ldo >= (1LL << 31))
        return CBA_ERR_UNSUPPORTED;
    // a matrix's own rows fit its batch stride
    if (d->batch > 1) {
        if (d->batch_in != 0 && d->batch_in < (d->rows - 1) * ldi + d->cols) return CBA_ERR_ARG;
        if (d->batch_out != 0 && d->batch_out < (d->rows - 1) * ldo + d->cols) return CBA_ERR_ARG;
    }
    p->wide = d->rows <= d->cols;
    p->m = std::min(d->rows, d->cols);
    p->n = std::max(d->rows, d->cols);
    p->x_pitch = (d->cols + 7LL) / 8 * 8;
    p->s_pitch = (p->m + 7LL) / 8 * 8;
    p->x_batch = p->x_pitch * d->rows;
    p->s_batch = p->s_pitch * p->m;
    const size_t xb = up256((size_t)p->x_batch * d->batch * 2), sb = up256((size_t)p->s_batch * d->batch * 2);
    p->off_part = 256;
    p->off_x0 = p->off_part + up256((size_t)d->batch * kNormBlocks * sizeof(double));
    p->off_x1 = p->off_x0 + xb;
    p->off_s = p->off_x1 + xb;
    p->off_c = p->off_s + sb;
    p->total = p->off_c + sb;
    return CBA_OK;
}

// One operand: [batch][rows][cols] of f16, rows `pitch` apart, `tile` rows of the
// operand per load (K-major) or boxes of 64 x 64 (M/N-major).
bool ns_map(CUtensorMap *m, const __half *base, int batch, int rows, int cols, long long pitch, int major, int tile) {
    const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)batch};
    const uint64_t strides[2] = {(uint64_t)pitch * 2, (uint64_t)pitch * 2 * (uint64_t)rows};
    const uint32_t box[3] = {64, major ? 64u : (uint32_t)tile, 1};
    return tma_encode_16(m, base, false, 3, dims, strides, box);
}

struct NsOperand {
    const __half *base;
    int rows, cols;
    long long pitch;
    int major;
};

// A product's kernel and the tensor maps of its operands, made once per call and
// operand buffer.
struct NsProduct {
    int cg, bn, sk;  // blocks per tile (pair), tile columns, blocks that share a contraction
    CUtensorMap ta, tb;
};

// The tile whose rounds over the SMs take least: a round of 256 x 256 by pairs of
// blocks takes 1, of 128 x 128 0.8, of 128 x 64 0.55 of the time (a smaller tile
// moves more bytes per product); 128 x 64 computes all of a symmetric product.
// And where `split` (a symmetric product without aux) has a long contraction and
// few tiles, clusters share it.  Five steps in us, the rule's side first:
//   128 columns, not pairs   1024x2048 154, 168; symmetric ones of 2048x2048 256, 309, of 8 of 1024x1024 279, 368
//   pairs, not 128 columns   1024x4096 196, 205; symmetric ones of 2 of 8192x2048 857, 1033
//   64 columns, not 128      symmetric ones of 1024x1024 124, 152
//   128 columns, not 64      1024x2048 154, 166
//   contractions shared      512x2304 109, not 128; 256x8192 117, not 235; 1024x4096 196, not 215
//   by two only where long   1024x1024 124, also below 48 stages 132
bool ns_product(NsProduct *p, const NsOperand &oa, const NsOperand &ob, int M, int N, int K, bool sym, bool split,
                int batch) {
    auto tiles = [&](int tm, int tn, bool half) {
        const long long mt = (M + tm - 1) / tm, nt = (N + tn - 1) / tn;
        return (half ? mt * (mt + 1) / 2 : mt * nt) * batch;
    };
    auto cost = [](long long tiles, int at_once, int round) { return (tiles + at_once - 1) / at_once * round; };
    const long long c256 = cost(tiles(256, 256, sym), kNumSMs / 2, 20), c128 = cost(tiles(128, 128, sym), kNumSMs, 16),
                    c64 = cost(tiles(128, 64, false), kNumSMs, 11);
    if (c256 < c128 && c256 < c64) *p = NsProduct{2, 256, 1, {}, {}};
    else if (c128 <= c64) *p = NsProduct{1, 128, 1, {}, {}};
    else *p = NsProduct{1, 64, 1, {}, {}};
    const int nk = (K + kNsBK - 1) / kNsBK;
    if (split && p->cg == 1) {
        // 128 blocks in clusters of 8 fit the GPU at once; at least 4 stages each, and
        // more where few share: joining costs them as much as it saves otherwise
        const long long t128 = tiles(128, 128, true);
        for (int sk = 8; sk >= 2; sk /= 2)
            if (t128 * sk <= 128 && nk >= 4 * sk && nk * sk >= 96) {
                *p = NsProduct{1, 128, sk, {}, {}};
                break;
            }
    }
    return ns_map(&p->ta, oa.base, batch, oa.rows, oa.cols, oa.pitch, oa.major, 128) &&
           ns_map(&p->tb, ob.base, batch, ob.rows, ob.cols, ob.pitch, ob.major, p->bn / p->cg);
}

template <auto Kern>
cudaError_t ns_launch(unsigned grid, int cluster, uint32_t smem, const NsProduct &p, const NsArgs &a, cudaStream_t st) {
    cudaError_t e = allow_smem<Kern>((int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kNsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, Kern, p.ta, p.tb, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t ns_gemm(const NsProduct &p, NsArgs a, int batch, cudaStream_t st) {
    const int tm = 128 * p.cg;
    a.mt = (a.M + tm - 1) / tm;
    a.nt = (a.N + p.bn - 1) / p.bn;
    a.sym = a.sym && tm == p.bn;  // needs square tiles
    a.units = (a.sym ? a.mt * (a.mt + 1) / 2 : a.mt * a.nt) * batch;
    const unsigned grid = (unsigned)(p.cg * std::min(a.units, kNumSMs / p.cg)), parts = (unsigned)(a.units * p.sk);
    if (p.sk == 8) return ns_launch<ns_split_kernel<8>>(parts, 8, NsTile<1, 128>::SMEM, p, a, st);
    if (p.sk == 4) return ns_launch<ns_split_kernel<4>>(parts, 4, NsTile<1, 128>::SMEM, p, a, st);
    if (p.sk == 2) return ns_launch<ns_split_kernel<2>>(parts, 2, NsTile<1, 128>::SMEM, p, a, st);
    if (p.cg == 2) return ns_launch<ns_gemm_kernel<2, 256>>(grid, 2, NsTile<2, 256>::SMEM, p, a, st);
    if (p.bn == 128) return ns_launch<ns_gemm_kernel<1, 128>>(grid, 1, NsTile<1, 128>::SMEM, p, a, st);
    return ns_launch<ns_gemm_kernel<1, 64>>(grid, 1, NsTile<1, 64>::SMEM, p, a, st);
}

template <typename T, int VEC>
cudaError_t ns_start_vec(const cba_orthogonalize_desc_t &d, const NsPlan &p, const T *G, long long ld, long long bs,
                         void *ws, float held, cudaStream_t st) {
    const long long n = (long long)d.rows * d.cols;
    const int parts = (int)std::max(1LL, std::min<long long>(kNormBlocks, n / 8192));
    double *part = ws_at<double>(ws, p.off_part);
    ns_norm_kernel<T, VEC><<<dim3(parts, d.batch), 256, 0, st>>>(G, d.rows, d.cols, ld, bs, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int blocks = std::max(1, std::min((d.rows + 7) / 8, 8 * kNumSMs / std::min(d.batch, 8 * kNumSMs)));
    return launch_pdl(ns_cast_kernel<T, VEC>, dim3(blocks, d.batch), dim3(256), 0, st, G, d.rows, d.cols, ld, bs,
                      static_cast<const double *>(part), parts, d.eps, held, ws_at<__half>(ws, p.off_x0), p.x_pitch,
                      p.x_batch, static_cast<unsigned *>(ws));
}

template <typename T>
cudaError_t ns_start(const cba_orthogonalize_desc_t &d, const NsPlan &p, const void *G, void *ws, float held,
                     cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const long long ld = d.ld_in ? d.ld_in : d.cols, bs = d.batch_in ? d.batch_in : ld * d.rows;
    const T *g = static_cast<const T *>(G);
    if (aligned_to(G, 16) && d.cols % V == 0 && ld % V == 0 && bs % V == 0)
        return ns_start_vec<T, V>(d, p, g, ld, bs, ws, held, st);
    return ns_start_vec<T, 1>(d, p, g, ld, bs, ws, held, st);
}

// All steps of a matrix in one block, where it fits (in us, and as launches of their
// own: 50x500 24, 87; 128x576 44, 86; 64 of 64x256 25, 100; 304 of 128x512 86, 402).
bool small_fits(const NsPlan &p) {
    const int R = p.m <= 64 ? 64 : 128;
    return p.m <= 128 && small_smem(R, (p.n + 63) / 64) <= kSmMax;
}

cudaError_t ns_small(const cba_orthogonalize_desc_t &d, const NsPlan &p, const void *G, void *O, void *ws, float held,
                     cudaStream_t st) {
    SmArgs a{};
    a.G = G; a.O = O; a.rows = d.rows; a.cols = d.cols; a.m = p.m; a.n = p.n; a.steps = d.steps;
    a.wide = p.wide; a.R = p.m <= 64 ? 64 : 128; a.nb = (p.n + 63) / 64;
    a.in_type = d.in_type; a.out_type = d.out_type;
    a.ld_in = d.ld_in ? d.ld_in : d.cols;
    a.batch_in = d.batch_in ? d.batch_in : a.ld_in * d.rows;
    a.ld_out = d.ld_out ? d.ld_out : d.cols;
    a.batch_out = d.batch_out ? d.batch_out : a.ld_out * d.rows;
    a.c_held = c_power(d);
    a.a = d.a * a.c_held; a.b = d.b * (a.c_held / kNsSym); a.c = d.c * (a.c_held / (kNsSym * kNsSym));
    a.eps = d.eps; a.scale = d.scale; a.held = held;
    a.status = static_cast<unsigned *>(ws);
    const size_t smem = small_smem(a.R, a.nb);
    auto kern = a.R == 64 ? ns_small_kernel<64> : ns_small_kernel<128>;
    cudaError_t e = a.R == 64 ? allow_smem<ns_small_kernel<64>>((int)kSmMax) : allow_smem<ns_small_kernel<128>>((int)kSmMax);
    if (e != cudaSuccess) return e;
    // one block clears the status word itself, several must not undo each other's
    if (d.batch > 1) e = cudaMemsetAsync(ws, 0, 4, st);
    if (e != cudaSuccess) return e;
    kern<<<d.batch, kSmThreads, smem, st>>>(a);
    return cudaGetLastError();
}

cudaError_t ns_run(const cba_orthogonalize_desc_t &d, const NsPlan &p, const void *G, void *O, void *ws,
                   cudaStream_t st) {
    const float held = exp2f(roundf(0.5f * log2f((float)p.n)));
    if (small_fits(p)) return ns_small(d, p, G, O, ws, held, st);
    cudaError_t e = d.in_type == CBA_F32   ? ns_start<float>(d, p, G, ws, held, st)
                    : d.in_type == CBA_F16 ? ns_start<__half>(d, p, G, ws, held, st)
                                           : ns_start<__nv_bfloat16>(d, p, G, ws, held, st);
    if (e != cudaSuccess) return e;
    __half *x[2] = {ws_at<__half>(ws, p.off_x0), ws_at<__half>(ws, p.off_x1)};
    __half *S = ws_at<__half>(ws, p.off_s), *C = ws_at<__half>(ws, p.off_c);
    unsigned *status = static_cast<unsigned *>(ws);
    const NsOperand so{S, p.m, p.m, p.s_pitch, 0}, co{C, p.m, p.m, p.s_pitch, 0};
    // S: the contraction runs along X's rows (wide) or across them (tall); X': wide
    // C X, X's rows contracted over, tall X C
    NsProduct ps[2], pc, px[2];
    const int bufs = d.steps > 1 ? 2 : 1;
    bool ok = ns_product(&pc, so, so, p.m, p.m, p.m, true, false, d.batch);
    NsArgs as{}, ac{}, ax{};
    as.a_major = as.b_major = p.wide ? 0 : 1;
    ax.b_major = p.wide ? 1 : 0;
    for (int i = 0; i < bufs && ok; ++i) {
        const NsOperand xs{x[i], d.rows, d.cols, p.x_pitch, as.a_major}, xk{x[i], d.rows, d.cols, p.x_pitch, 0},
            xn{x[i], d.rows, d.cols, p.x_pitch, 1};
        ok = ns_product(&ps[i], xs, xs, p.m, p.m, p.n, true, true, d.batch) &&
             (p.wide ? ns_product(&px[i], co, xn, d.rows, d.cols, p.m, false, false, d.batch)
                     : ns_product(&px[i], xk, co, d.rows, d.cols, p.m, false, false, d.batch));
    }
    if (!ok) return cudaErrorInvalidValue;
    as.M = as.N = ac.M = ac.N = ac.K = ax.K = p.m;
    as.K = p.n;
    as.out_ld = ac.out_ld = ac.aux_ld = p.s_pitch;
    as.out_batch = ac.out_batch = ac.aux_batch = p.s_batch;
    as.out_type = ac.out_type = ax.out_type = CBA_F16;
    as.vec = ac.vec = ax.vec = 1;
    as.sym = ac.sym = 1;
    as.status = ac.status = ax.status = status;
    as.alpha = kNsSym / (held * held);
    as.out = S;
    const float c_held = c_power(d);
    ac.alpha = d.c * (c_held / (kNsSym * kNsSym));
    ac.beta = d.b * (c_held / kNsSym);
    ac.diag = d.a * c_held;
    ac.aux = S;
    ac.out = C;
    ax.M = d.rows;
    ax.N = d.cols;
    ax.alpha = 1.f / c_held;
    ax.out_ld = p.x_pitch;
    ax.out_batch = p.x_batch;
    for (int i = 0; i < d.steps; ++i) {
        e = ns_gemm(ps[i & 1], as, d.batch, st);
        if (e == cudaSuccess) e = ns_gemm(pc, ac, d.batch, st);
        if (e != cudaSuccess) return e;
        ax.out = x[~i & 1];
        if (i + 1 == d.steps) {  // the last product writes the caller's matrix
            ax.alpha *= d.scale / held;
            ax.out = O;
            ax.out_type = d.out_type;
            ax.out_ld = d.ld_out ? d.ld_out : d.cols;
            ax.out_batch = d.batch_out ? d.batch_out : ax.out_ld * d.rows;
            const long long v = 16 / (long long)dtype_bytes(d.out_type);
            ax.vec = aligned_to(O, 16) && ax.out_ld % v == 0 && ax.out_batch % v == 0;
        }
        e = ns_gemm(px[i & 1], ax, d.batch, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

}  // namespace cba

using namespace cba;

extern "C" {

size_t cba_orthogonalize_workspace_bytes(const cba_orthogonalize_desc_t *d) {
    NsPlan p;
    return check_ns(d, &p) == CBA_OK ? p.total : 0;
}

int cba_orthogonalize(const cba_orthogonalize_desc_t *d, const void *G, void *O, void *workspace,
                      size_t workspace_bytes, void *stream) {
    NsPlan p;
    const int rc = check_ns(d, &p);
    if (rc != CBA_OK) return rc;
    if (!G || !O) return CBA_ERR_ARG;
    if (!aligned_to(G, dtype_bytes(d->in_type)) || !aligned_to(O, dtype_bytes(d->out_type))) return CBA_ERR_ALIGN;
    if (!workspace || workspace_bytes < p.total) return CBA_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return CBA_ERR_ALIGN;
    cudaGetLastError();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = select_device_of(workspace);
    if (e == cudaSuccess) e = ns_run(*d, p, G, O, workspace, st);
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

}  // extern "C"
