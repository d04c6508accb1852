// cba_layernorm.cu -- layer norm over the last axis, forward and backward.
//
//   forward   mu = mean x, r = 1 / sqrt(mean (x - mu)^2 + eps)
//             y = (x - mu) r gamma + beta
//   backward  g = dy gamma, h = (x - mu) r
//             dx = r (g - mean g - h mean(g h)) (+ residual)
//             dgamma (= | +=) sum_rows dy h,   dbeta (= | +=) sum_rows dy
//
// Both are bound by memory: every element of x, dy and residual is read once
// and every element of y and dx written once.  A row is held in the registers
// of TPR threads (EPT elements each), so the centred variance and the two row
// means of the backward cost no second read.  All sums are fp32.
//
// Backward: a thread owns the same EPT columns of every row its group visits,
// so dgamma and dbeta are register accumulators over the rows; a block writes
// one partial row of each and colsum_kernel adds the partials in a fixed order
// (no atomics: the result does not depend on scheduling).
//
// Measured (us, and of the measured copy rate where memory bounds it):
//   forward 65536 x 2048 bf16                    103: 5.2 TB/s, 0.77 (96 after a pause)
//   backward 32768 x 4096 bf16 with a residual   193: 5.6 TB/s, 0.83 (187 + 3.5 of column sums)
//   backward 43264 x 255 fp32                    31: 4.3 TB/s, 0.63 (26 + 3.5; rows that are not
//       whole vectors move 4 bytes a thread)
//   169 x 512 fp32                               3 and 5.5 on the device; a call from Python takes
//       5.2 and 8.1, the time in which the host issues it
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "cba_internal.cuh"
#include "cba_kept.cuh"
#include "cba_ptx.cuh"
#include "cba_types.cuh"

namespace cba {

namespace {

constexpr int kLnMaxTpr = 512;          // threads of the widest in-register row (backward)
constexpr int kLnEpt = 16;              // elements per thread (backward)
constexpr int kWideCols = 2048;         // columns per block of the wide backward

struct LnArgs {
    const void *x, *dy, *gamma, *beta, *residual;
    void *y, *dx;
    float *mean, *rstd;         // forward: outputs (nullable)
    const float *mean_in, *rstd_in;
    float *part;                // backward partials [nblk][2][cols]
    float2 *rowc;               // wide backward: mean g, mean(g h) of each row
    long long rows, ld_x, ld_y, ld_dy, ld_dx, ld_res;
    int cols;
    float eps, inv_cols;
};

// Sum over the TPR threads of a row group (a warp, or warps of one block that
// meet at named barrier 1 + group); every thread gets it.  `buf` holds two
// halves used in turn, so one barrier per reduction is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&s)[N], float *buf, int &half, int group, int t) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        float *b = buf + (group * 2 + half) * (W * N);
        if ((t & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) b[(t >> 5) * N + i] = s[i];
        ptx::named_bar_sync(1 + group, TPR);
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] += b[w * N + i];
        half ^= 1;
    }
}

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, VEC> *>(p);
}

// ---- forward: one row per group of TPR threads

// (64 registers from 128 threads a row on, 1024 threads on an SM: 10000x9001 bf16
// 165 us, with the 69 that the compiler takes 305.)
template <typename T, typename P, int VEC, int TPR, int EPT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, TPR < 128 ? 0 : 1024 / TPR)
    ln_fwd_kernel(const LnArgs a) {
    constexpr int NV = EPT / VEC;
    constexpr int BLOCK = TPR < 128 ? 128 : TPR;
    __shared__ float buf[BLOCK / 32 * 2 * 1 + 1];
    const int group = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * (BLOCK / TPR) + group;
    if (row >= a.rows) return;  // whole groups leave: their barrier is theirs alone
    int half = 0;
    const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
    float v[EPT];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * VEC;
        if (c < a.cols) {
            const Pack<T, VEC> p = load_pack<T, VEC>(x + c);
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[0] += v[i * VEC + j] = to_f32(p.v[j]);
        }
    }
    row_sum<TPR, 1>(s, buf, half, group, t);
    const float mean = s[0] * a.inv_cols;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((i * TPR + t) * VEC < a.cols)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = v[i * VEC + j] - mean;
                s[0] = fmaf(d, d, s[0]);
            }
    row_sum<TPR, 1>(s, buf, half, group, t);
    const float rstd = 1.f / sqrtf(s[0] * a.inv_cols + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    T *y = static_cast<T *>(a.y) + row * a.ld_y;
    const P *ga = static_cast<const P *>(a.gamma), *be = static_cast<const P *>(a.beta);
    // 8 columns' parameters at a time: no load of theirs moves ahead of a store to y by itself
    // (20000x1001 bf16: 46 -> 32 us)
    constexpr int CH = VEC < 8 ? 8 / VEC : 1;
#pragma unroll
    for (int i0 = 0; i0 < NV; i0 += CH) {
        Pack<P, VEC> g[CH], b[CH];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = ((i0 + k) * TPR + t) * VEC;
            if (c < a.cols) {
                if (ga) g[k] = load_pack<P, VEC>(ga + c);
                if (be) b[k] = load_pack<P, VEC>(be + c);
            }
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int i = i0 + k, c = (i * TPR + t) * VEC;
            if (c < a.cols) {
                Pack<T, VEC> o;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    float h = (v[i * VEC + j] - mean) * rstd;
                    if (ga) h *= to_f32(g[k].v[j]);
                    if (be) h += to_f32(b[k].v[j]);
                    o.v[j] = from_f32<T>(h);
                }
                *reinterpret_cast<Pack<T, VEC> *>(y + c) = o;
            }
        }
    }
}

// Rows too long for registers: three sweeps, the second and third from L2.
template <typename T, typename P>
__global__ void __launch_bounds__(1024) ln_fwd_long_kernel(const LnArgs a) {
    __shared__ float buf[64];
    const long long row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
    T *y = static_cast<T *>(a.y) + row * a.ld_y;
    const P *ga = static_cast<const P *>(a.gamma), *be = static_cast<const P *>(a.beta);
    int half = 0;
    float s[1] = {0.f};
#pragma unroll 8
    for (int c = threadIdx.x; c < a.cols; c += 1024) s[0] += to_f32(x[c]);
    row_sum<1024, 1>(s, buf, half, 0, threadIdx.x);
    const float mean = s[0] * a.inv_cols;
    s[0] = 0.f;
#pragma unroll 8
    for (int c = threadIdx.x; c < a.cols; c += 1024) {
        const float d = to_f32(x[c]) - mean;
        s[0] = fmaf(d, d, s[0]);
    }
    row_sum<1024, 1>(s, buf, half, 0, threadIdx.x);
    const float rstd = 1.f / sqrtf(s[0] * a.inv_cols + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    for (int c0 = threadIdx.x; c0 < a.cols; c0 += 4 * 1024) {  // loads of four columns ahead of their stores
        float h[4], g[4], b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = min(c0 + k * 1024, a.cols - 1);
            h[k] = to_f32(x[c]);
            g[k] = ga ? to_f32(ga[c]) : 1.f;
            b[k] = be ? to_f32(be[c]) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c0 + k * 1024 < a.cols) y[c0 + k * 1024] = from_f32<T>(fmaf((h[k] - mean) * rstd, g[k], b[k]));
    }
}

// One partial row of dgamma and dbeta per block: the groups' sums added in group
// order through `gsum` ((GROUPS - 1) TPR EPT floats).
template <int VEC, int TPR, int EPT, int GROUPS>
__device__ __forceinline__ void write_partials(const LnArgs &a, float (&dg)[EPT], float (&db)[EPT],
                                               int group, int t, float *gsum) {
    float *part = a.part + (size_t)blockIdx.x * 2 * a.cols;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float(&acc)[EPT] = w ? db : dg;
        if constexpr (GROUPS > 1) {
            __syncthreads();
            if (group > 0)
#pragma unroll
                for (int e = 0; e < EPT; ++e) gsum[((group - 1) * EPT + e) * TPR + t] = acc[e];
            __syncthreads();
            if (group == 0)
                for (int g = 0; g < GROUPS - 1; ++g)
#pragma unroll
                    for (int e = 0; e < EPT; ++e) acc[e] += gsum[(g * EPT + e) * TPR + t];
        }
        if (group == 0)
#pragma unroll
            for (int i = 0; i < EPT / VEC; ++i) {
                const int c = (i * TPR + t) * VEC;
                if (c < a.cols)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) part[(size_t)w * a.cols + c + j] = acc[i * VEC + j];
            }
    }
}

// ---- backward: a group of TPR threads walks rows; threads own columns

// Blocks per SM, and registers for as many (20000x1001 bf16 49 us; where the compiler
// took more, and the fourth block waited, 69).  A residual takes more of them:
// 60000x257 with three blocks 55 us, with four, which spill, 106; 20000x1001 59, 106.
__host__ __device__ constexpr int bwd_per_sm(int tpr, bool res) {
    return tpr >= 512 ? 1 : tpr == 256 ? 2 : res ? 3 : 4;
}

template <typename T, typename P, int VEC, int TPR, int EPT, bool RES>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, bwd_per_sm(TPR, RES))
    ln_bwd_kernel(const LnArgs a) {
    constexpr int NV = EPT / VEC;
    constexpr int BLOCK = TPR < 128 ? 128 : TPR;
    constexpr int GROUPS = BLOCK / TPR;
    __shared__ float buf[BLOCK / 32 * 2 * 2];
    __shared__ float gsum[GROUPS > 1 ? (GROUPS - 1) * TPR * EPT : 1];
    const int group = threadIdx.x / TPR, t = threadIdx.x % TPR;
    int half = 0;
    float dg[EPT], db[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) dg[i] = db[i] = 0.f;
    ptx::griddep_launch_dependents();
    const P *gp = static_cast<const P *>(a.gamma);
    const T *xb = static_cast<const T *>(a.x), *dyb = static_cast<const T *>(a.dy);
    const T *rb = static_cast<const T *>(a.residual);
    T *dxb = static_cast<T *>(a.dx);
    const long long step = (long long)gridDim.x * GROUPS;
    long long row = (long long)blockIdx.x * GROUPS + group;
    Pack<T, VEC> px[NV], pd[NV];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](long long r) {
        if (r >= a.rows) return;
        const T *x = xb + r * a.ld_x, *dy = dyb + r * a.ld_dy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < a.cols) {
                px[i] = load_pack<T, VEC>(x + c);
                pd[i] = load_pack<T, VEC>(dy + c);
            }
        }
        mean = a.mean_in[r];
        rstd = a.rstd_in[r];
    };
    fetch(row);
    for (; row < a.rows; row += step) {
        float h[EPT], d[EPT];
        float s[2] = {0.f, 0.f};
        const float r = rstd;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < a.cols) {
                // gamma from L1 every row: registers are what limits the rows
                // in flight
                Pack<P, VEC> pg;
                if (gp) pg = load_pack<P, VEC>(gp + c);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int e = i * VEC + j;
                    h[e] = (to_f32(px[i].v[j]) - mean) * r;
                    const float dv = to_f32(pd[i].v[j]);
                    dg[e] = fmaf(dv, h[e], dg[e]);
                    db[e] += dv;
                    d[e] = gp ? dv * to_f32(pg.v[j]) : dv;
                    s[0] += d[e];
                    s[1] = fmaf(d[e], h[e], s[1]);
                }
            }
        }
        Pack<T, VEC> pr[NV];
        if constexpr (RES) {
            const T *rp = rb + row * a.ld_res;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * VEC;
                if (c < a.cols) pr[i] = load_pack<T, VEC>(rp + c);
            }
        }
        fetch(row + step);
        row_sum<TPR, 2>(s, buf, half, group, t);
        const float m1 = s[0] * a.inv_cols, m2 = s[1] * a.inv_cols;
        T *dx = dxb + row * a.ld_dx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < a.cols) {
                Pack<T, VEC> o;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int e = i * VEC + j;
                    float v = r * (d[e] - fmaf(h[e], m2, m1));
                    if constexpr (RES) v += to_f32(pr[i].v[j]);
                    o.v[j] = from_f32<T>(v);
                }
                *reinterpret_cast<Pack<T, VEC> *>(dx + c) = o;
            }
        }
    }
    write_partials<VEC, TPR, EPT, GROUPS>(a, dg, db, group, t, gsum);
}

// ---- many rows: the same two kernels fed by asynchronous copies

// Each thread copies the 16-byte vectors it will use itself, S - 1 rows ahead,
// into its own slots of shared memory: the bytes in flight cost no registers,
// and as no thread reads another's slots the ring needs no barrier.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kRing = 4;  // rows of a group in flight or in use (backward)
__host__ __device__ constexpr int ring_block(int tpr) { return tpr < 256 ? 256 : tpr; }

template <typename T, typename P, int TPR, int EPT, int RING>
__global__ void __launch_bounds__(ring_block(TPR)) ln_fwd_ring_kernel(const LnArgs a) {
    constexpr int VEC = 16 / sizeof(T), NV = EPT / VEC, BLOCK = ring_block(TPR);
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float buf[BLOCK / 32 * 2];
    const int group = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * (BLOCK / TPR);
    long long row = (long long)blockIdx.x * (BLOCK / TPR) + group;
    int half = 0;
    const T *xb = static_cast<const T *>(a.x);
    const P *ga = static_cast<const P *>(a.gamma), *be = static_cast<const P *>(a.beta);
    const uint32_t mine = ptx::smem_u32(ring) + threadIdx.x * 16;
    auto fetch = [&](long long r, int st) {
        if (r < a.rows) {
            const T *x = xb + r * a.ld_x;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * VEC;
                if (c < a.cols) copy16(mine + (st * NV + i) * (BLOCK * 16), x + c);
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) fetch(row + i * step, i);
    // two columns per instruction: the issue slots are what bounded one at a time
    // (60% of them at 4.5 TB/s of 65536 x 2048 bf16)
    const float2 one = make_float2(1.f, 1.f), zero = make_float2(0.f, 0.f);
    for (int st = 0; row < a.rows; row += step, st = (st + 1) % RING) {
        copies_wait<RING - 2>();
        float2 v[EPT / 2];
        float2 sum = zero;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * TPR + t) * VEC < a.cols) {
                const Pack<T, VEC> p = *reinterpret_cast<const Pack<T, VEC> *>(
                    ring + ((st * NV + i) * BLOCK + threadIdx.x) * 16);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    v[i * VEC / 2 + j] = pair_of(p, j);
                    sum = ptx::add2(sum, v[i * VEC / 2 + j]);
                }
            }
        fetch(row + (RING - 1) * step, (st + RING - 1) % RING);
        float s[1] = {sum.x + sum.y};
        row_sum<TPR, 1>(s, buf, half, group, t);
        const float mean = s[0] * a.inv_cols;
        const float2 nm = make_float2(-mean, -mean);
        sum = zero;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * TPR + t) * VEC < a.cols)
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    float2 &d = v[i * VEC / 2 + j];
                    d = ptx::add2(d, nm);
                    sum = ptx::fma2(d, d, sum);
                }
        s[0] = sum.x + sum.y;
        row_sum<TPR, 1>(s, buf, half, group, t);
        const float rstd = 1.f / sqrtf(s[0] * a.inv_cols + a.eps);
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        const float2 r2 = make_float2(rstd, rstd);
        T *y = static_cast<T *>(a.y) + row * a.ld_y;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < a.cols) {
                Pack<P, VEC> g, b;  // from L1 after the first row
                if (ga) g = load_pack<P, VEC>(ga + c);
                if (be) b = load_pack<P, VEC>(be + c);
                Pack<T, VEC> o;
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    const float2 h = ptx::mul2(v[i * VEC / 2 + j], r2);
                    set_pair(o, j, ptx::fma2(h, ga ? pair_of(g, j) : one, be ? pair_of(b, j) : zero));
                }
                *reinterpret_cast<Pack<T, VEC> *>(y + c) = o;
            }
        }
    }
}

// Blocks per SM that the ring backward is compiled and launched for.
__host__ __device__ constexpr int ring_bwd_per_sm(int tpr) { return tpr <= 256 ? 2 : 1; }

template <typename T, typename P, int TPR, int EPT, bool RES>
__global__ void __launch_bounds__(ring_block(TPR), ring_bwd_per_sm(TPR))
    ln_bwd_ring_kernel(const LnArgs a) {
    constexpr int VEC = 16 / sizeof(T), NV = EPT / VEC, BLOCK = ring_block(TPR);
    constexpr int GROUPS = BLOCK / TPR, NT = RES ? 3 : 2;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float buf[BLOCK / 32 * 2 * 2];
    const int group = threadIdx.x / TPR, t = threadIdx.x % TPR;
    int half = 0;
    float2 dg[EPT / 2], db[EPT / 2];
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) dg[i] = db[i] = make_float2(0.f, 0.f);
    ptx::griddep_launch_dependents();
    const P *gp = static_cast<const P *>(a.gamma);
    const T *xb = static_cast<const T *>(a.x), *dyb = static_cast<const T *>(a.dy);
    const T *rb = static_cast<const T *>(a.residual);
    T *dxb = static_cast<T *>(a.dx);
    const long long step = (long long)gridDim.x * GROUPS;
    long long row = (long long)blockIdx.x * GROUPS + group;
    const uint32_t mine = ptx::smem_u32(ring) + threadIdx.x * 16;
    float nmean = 0.f, nrstd = 0.f;
    auto fetch = [&](long long r, int st) {
        if (r < a.rows) {
            const T *x = xb + r * a.ld_x, *dy = dyb + r * a.ld_dy;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TPR + t) * VEC;
                const uint32_t to = mine + (st * NT * NV + i) * (BLOCK * 16);
                if (c < a.cols) {
                    copy16(to, x + c);
                    copy16(to + NV * BLOCK * 16, dy + c);
                    if constexpr (RES) copy16(to + 2 * NV * BLOCK * 16, rb + r * a.ld_res + c);
                }
            }
        }
        copies_commit();
    };
    auto stats = [&](long long r) {
        if (r < a.rows) nmean = a.mean_in[r], nrstd = a.rstd_in[r];
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(row + i * step, i);
    stats(row);
    for (int st = 0; row < a.rows; row += step, st = (st + 1) % kRing) {
        const float mean = nmean, r = nrstd;
        stats(row + step);
        copies_wait<kRing - 2>();
        auto slot = [&](int which, int i) {
            return *reinterpret_cast<const Pack<T, VEC> *>(
                ring + (((st * NT + which) * NV + i) * BLOCK + threadIdx.x) * 16);
        };
        float2 h[EPT / 2], g[EPT / 2];
        Pack<T, VEC> pr[RES ? NV : 1];
        float2 s0 = make_float2(0.f, 0.f), s1 = s0;
        const float2 nm = make_float2(-mean, -mean), r2 = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < a.cols) {
                const Pack<T, VEC> px = slot(0, i), pd = slot(1, i);
                if constexpr (RES) pr[i] = slot(2, i);
                Pack<P, VEC> pg;  // from L1 after the first row
                if (gp) pg = load_pack<P, VEC>(gp + c);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    const int e = i * VEC / 2 + j;
                    h[e] = ptx::mul2(ptx::add2(pair_of(px, j), nm), r2);
                    const float2 d = pair_of(pd, j);
                    dg[e] = ptx::fma2(d, h[e], dg[e]);
                    db[e] = ptx::add2(db[e], d);
                    g[e] = gp ? ptx::mul2(d, pair_of(pg, j)) : d;
                    s0 = ptx::add2(s0, g[e]);
                    s1 = ptx::fma2(g[e], h[e], s1);
                }
            }
        }
        fetch(row + (kRing - 1) * step, (st + kRing - 1) % kRing);
        float s[2] = {s0.x + s0.y, s1.x + s1.y};
        row_sum<TPR, 2>(s, buf, half, group, t);
        const float m1 = s[0] * a.inv_cols, m2 = s[1] * a.inv_cols;
        const float2 n1 = make_float2(-m1, -m1), n2 = make_float2(-m2, -m2);
        T *dx = dxb + row * a.ld_dx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + t) * VEC;
            if (c < a.cols) {
                Pack<T, VEC> o;
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    const int e = i * VEC / 2 + j;
                    const float2 u = ptx::add2(g[e], ptx::fma2(h[e], n2, n1));
                    if constexpr (RES) set_pair(o, j, ptx::fma2(u, r2, pair_of(pr[i], j)));
                    else set_pair(o, j, ptx::mul2(u, r2));
                }
                *reinterpret_cast<Pack<T, VEC> *>(dx + c) = o;
            }
        }
    }
    float sg[EPT], sb[EPT];
#pragma unroll
    for (int e = 0; e < EPT / 2; ++e) {
        sg[2 * e] = dg[e].x, sg[2 * e + 1] = dg[e].y;
        sb[2 * e] = db[e].x, sb[2 * e + 1] = db[e].y;
    }
    write_partials<VEC, TPR, EPT, GROUPS>(a, sg, sb, group, t, reinterpret_cast<float *>(ring));
}

// Rows too long for registers: mean g and mean(g h) of each row first, then dx
// and the column sums over blocks of (columns, rows), which re-read x and dy.
template <typename T, typename P>
__global__ void __launch_bounds__(512) ln_bwd_rowsums_kernel(const LnArgs a) {
    __shared__ float buf[64];
    const long long row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
    const T *dy = static_cast<const T *>(a.dy) + row * a.ld_dy;
    const P *ga = static_cast<const P *>(a.gamma);
    const float mean = a.mean_in[row], rstd = a.rstd_in[row];
    int half = 0;
    float s[2] = {0.f, 0.f};
#pragma unroll 8
    for (int c = threadIdx.x; c < a.cols; c += 512) {
        const float g = to_f32(dy[c]) * (ga ? to_f32(ga[c]) : 1.f);
        s[0] += g;
        s[1] = fmaf(g, (to_f32(x[c]) - mean) * rstd, s[1]);
    }
    row_sum<512, 2>(s, buf, half, 0, threadIdx.x);
    if (threadIdx.x == 0) a.rowc[row] = make_float2(s[0] * a.inv_cols, s[1] * a.inv_cols);
}

template <typename T, typename P>
__global__ void __launch_bounds__(256) ln_bwd_wide_kernel(const LnArgs a) {
    constexpr int E = kWideCols / 256;
    const int c0 = blockIdx.x * kWideCols + threadIdx.x;
    const T *xb = static_cast<const T *>(a.x), *dyb = static_cast<const T *>(a.dy);
    const T *rb = static_cast<const T *>(a.residual);
    const P *gp = static_cast<const P *>(a.gamma);
    float ga[E], dg[E], db[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = c0 + e * 256;
        dg[e] = db[e] = 0.f;
        ga[e] = gp && c < a.cols ? to_f32(gp[c]) : 1.f;
    }
    // a row's loads before the stores of the row before: none would move ahead of them by itself
    // (10000x9001 bf16, with the row sums: 573 -> 238 us)
    T px[E], pd[E], pr[E];
    float mean = 0.f, rstd = 0.f;
    float2 m = make_float2(0.f, 0.f);
    auto fetch = [&](long long row) {
        if (row >= a.rows) return;
        const T *x = xb + row * a.ld_x, *dy = dyb + row * a.ld_dy;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = c0 + e * 256;
            if (c < a.cols) {
                px[e] = x[c];
                pd[e] = dy[c];
                if (rb) pr[e] = rb[row * a.ld_res + c];
            }
        }
        mean = a.mean_in[row];
        rstd = a.rstd_in[row];
        m = a.rowc[row];
    };
    fetch(blockIdx.y);
    for (long long row = blockIdx.y; row < a.rows; row += gridDim.y) {
        T *dx = static_cast<T *>(a.dx) + row * a.ld_dx;
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (c0 + e * 256 < a.cols) {
                const float h = (to_f32(px[e]) - mean) * rstd, d = to_f32(pd[e]);
                dg[e] = fmaf(d, h, dg[e]);
                db[e] += d;
                v[e] = rstd * (d * ga[e] - fmaf(h, m.y, m.x));
                if (rb) v[e] += to_f32(pr[e]);
            }
        }
        fetch(row + gridDim.y);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (c0 + e * 256 < a.cols) dx[c0 + e * 256] = from_f32<T>(v[e]);
    }
    float *part = a.part + (size_t)blockIdx.y * 2 * a.cols;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = c0 + e * 256;
        if (c < a.cols) {
            part[c] = dg[e];
            part[(size_t)a.cols + c] = db[e];
        }
    }
}

// dgamma and dbeta from the blocks' partial rows, added in a fixed order: 32
// warps take every 32nd partial of 32 columns, then one adds the 32 sums.
__global__ void __launch_bounds__(1024)
    ln_colsum_kernel(const float *part, int nblk, int cols, int accumulate, float *dgamma,
                     float *dbeta) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, which = blockIdx.y;
    float *out = which ? dbeta : dgamma;
    ptx::griddep_wait();
    if (out == nullptr) return;
    float s = 0.f;
    if (c < cols) {
        const float *p = part + (size_t)which * cols + c;
        const size_t row = (size_t)2 * cols;
        int b = w;
        for (; b + 96 < nblk; b += 128)  // four loads in flight
            s += (p[b * row] + p[(b + 32) * row]) + (p[(b + 64) * row] + p[(b + 96) * row]);
        for (; b < nblk; b += 32) s += p[b * row];
    }
    sm[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 32; ++i) s += sm[i][lane];
        out[c] = accumulate ? out[c] + s : s;
    }
}

// ---- launch plans

struct LnPlan {
    int tpr;       // backward: threads per row, 0 = the wide path
    int ring_tpr;  // backward: the ring kernel's threads per row, 0 = not that kernel
    int nblk;      // backward: partial rows
    size_t off_rowc, part_bytes, total;
};

int bwd_tpr(int cols) {
    for (int t = 32; t <= kLnMaxTpr; t *= 2)
        if (cols <= t * kLnEpt) return t;
    return 0;
}

// Whether a call's rows move as 16-byte vectors and are enough for the ring: a
// row for every group of a block per SM.  (In us, ring and rows held in registers:
// bf16 forward 65536x2048 98, 128; 4864x2048 13.9, 14.8; 2432x512 3.4, 4.6;
// backward 32768x4096 142, 243; 608x4096 16.9, 18.8; 304x4096 13.1, 14.8; 2432x512
// 7.7, 11.0.  The one size found where it loses: forward 65536x512 31, 29.)
bool ring_rows(long long rows, int tpr) {
    const int groups = tpr < 256 ? 256 / tpr : 1;
    return rows >= (long long)groups * kNumSMs;
}

// The plan of a backward call whose rows move as 16-byte vectors or not.  Blocks:
// a row per group while that needs no more than a block per SM; past that at
// least 4 rows per group, so that the partial rows stay small beside the data
// they come from.  (fp32, 255 columns, us with at least 1, 4, 16 rows: 8192 rows
// 11.1, 10.3, 16.5; 1000 rows 7.6, 6.6, 7.0; the ring, bf16, a block per SM and two
// of fewer rows: 608x4096 16.9, 21.0; 1216x2048 12.2, 14.1; 304x4096 13.1 and with
// half of the blocks 14.4.)
LnPlan ln_bwd_plan(const cba_layernorm_desc_t &d, bool vec, bool res) {
    LnPlan p{};
    p.tpr = bwd_tpr(d.cols);
    if (vec) {
        const int e = d.type == CBA_F32 ? 8 : 16;
        for (int t = 32; t <= kLnMaxTpr && !p.ring_tpr; t *= 2)
            if (d.cols <= t * e) p.ring_tpr = t;
        if (p.ring_tpr && !ring_rows(d.rows, p.ring_tpr)) p.ring_tpr = 0;
    }
    const int tpr = p.ring_tpr ? p.ring_tpr : p.tpr, block = p.ring_tpr ? 256 : 128;
    const int groups = tpr && tpr < block ? block / tpr : 1;
    const int per_sm = p.ring_tpr ? ring_bwd_per_sm(tpr) : tpr == 0 ? 1 : bwd_per_sm(tpr, res);
    long long most = (long long)kNumSMs * per_sm;
    if (tpr == 0) most = std::max(1LL, most * 6 / ((d.cols + kWideCols - 1) / kWideCols));
    const long long one = std::min<long long>(kNumSMs, (d.rows + groups - 1) / groups);
    const long long four = (d.rows + 4LL * groups - 1) / (4LL * groups);
    p.nblk = (int)std::max(1LL, std::min(most, std::max(one, four)));
    if (d.rows == 0) p.nblk = 0;
    p.part_bytes = ((size_t)p.nblk * 2 * d.cols * sizeof(float) + 255) / 256 * 256;
    p.off_rowc = p.part_bytes;
    p.total = p.part_bytes;
    if (p.tpr == 0) p.total += ((size_t)d.rows * sizeof(float2) + 255) / 256 * 256;
    p.total = std::max<size_t>(p.total, 256);
    return p;
}

template <typename T, typename P, int TPR, int EPT>
cudaError_t fwd_ring(const LnArgs &a, cudaStream_t st) {
    // rows of 128 bytes per thread: two ahead fill the memory pipe
    constexpr int ring = EPT * (int)sizeof(T) >= 128 ? 3 : 4;
    constexpr int block = ring_block(TPR), rpb = block / TPR, smem = ring * block * EPT * (int)sizeof(T);
    auto kern = ln_fwd_ring_kernel<T, P, TPR, EPT, ring>;
    static std::atomic<int> kept{0};
    int per_sm = 0;
    cudaError_t e = allow_smem<ln_fwd_ring_kernel<T, P, TPR, EPT, ring>>(smem);
    if (e == cudaSuccess)
        e = kept_value(kept, &per_sm,
                       [&](int *n) { return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, block, smem); });
    if (e != cudaSuccess) return e;
    const long long blocks = std::min<long long>((a.rows + rpb - 1) / rpb, (long long)kNumSMs * per_sm);
    kern<<<(unsigned)blocks, block, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, typename P, int VEC>
cudaError_t fwd_vec(const LnArgs &a, cudaStream_t st) {
    if constexpr (VEC > 1) {
        // a row per warp as long as it fits: its two sums then need no barrier
        constexpr int E = 128 / sizeof(T);
        if (a.cols <= 8 * E && ring_rows(a.rows, 32)) return fwd_ring<T, P, 32, E / 4>(a, st);
        if (a.cols <= 16 * E && ring_rows(a.rows, 32)) return fwd_ring<T, P, 32, E / 2>(a, st);
        if (a.cols <= 32 * E && ring_rows(a.rows, 32)) return fwd_ring<T, P, 32, E>(a, st);
        if (a.cols <= 64 * E && ring_rows(a.rows, 64)) return fwd_ring<T, P, 64, E>(a, st);
        if (a.cols <= 128 * E && ring_rows(a.rows, 128)) return fwd_ring<T, P, 128, E>(a, st);
        if (a.cols <= 256 * E && ring_rows(a.rows, 256)) return fwd_ring<T, P, 256, E>(a, st);
    }
#define CBA_LN_FWD(TPR, EPT)                                                                    \
    do {                                                                                        \
        constexpr int block = TPR < 128 ? 128 : TPR, rpb = block / TPR;                         \
        ln_fwd_kernel<T, P, VEC, TPR, EPT>                                                      \
            <<<(unsigned)((a.rows + rpb - 1) / rpb), block, 0, st>>>(a);                        \
        return cudaGetLastError();                                                              \
    } while (0)
    if (a.cols <= 256) CBA_LN_FWD(32, 8);
    if (a.cols <= 512) CBA_LN_FWD(32, 16);
    if (a.cols <= 1024) CBA_LN_FWD(32, 32);
    if (a.cols <= 2048) CBA_LN_FWD(64, 32);
    if (a.cols <= 4096) CBA_LN_FWD(128, 32);
    if (a.cols <= 8192) CBA_LN_FWD(256, 32);
    if (a.cols <= 16384) CBA_LN_FWD(512, 32);
#undef CBA_LN_FWD
    ln_fwd_long_kernel<T, P><<<(unsigned)a.rows, 1024, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, typename P, int TPR, int EPT, bool RES>
cudaError_t bwd_ring(const LnArgs &a, const LnPlan &p, cudaStream_t st) {
    constexpr int block = ring_block(TPR), smem = kRing * (RES ? 3 : 2) * block * EPT * (int)sizeof(T);
    static_assert((block / TPR - 1) * TPR * EPT * 4 <= smem, "the groups' sums fit the ring");
    cudaError_t e = allow_smem<ln_bwd_ring_kernel<T, P, TPR, EPT, RES>>(smem);
    if (e != cudaSuccess) return e;
    ln_bwd_ring_kernel<T, P, TPR, EPT, RES><<<p.nblk, block, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, typename P, int VEC, bool RES>
cudaError_t bwd_vec(const LnArgs &a, const LnPlan &p, cudaStream_t st) {
    if constexpr (VEC > 1) {
        constexpr int E = sizeof(T) == 4 ? 8 : 16;
        if (p.ring_tpr) switch (p.ring_tpr) {
            case 32: return bwd_ring<T, P, 32, E, RES>(a, p, st);
            case 64: return bwd_ring<T, P, 64, E, RES>(a, p, st);
            case 128: return bwd_ring<T, P, 128, E, RES>(a, p, st);
            case 256: return bwd_ring<T, P, 256, E, RES>(a, p, st);
            default: return bwd_ring<T, P, 512, E, RES>(a, p, st);
            }
    }
    switch (p.tpr) {
    case 32:
        if (a.cols <= 256) ln_bwd_kernel<T, P, VEC, 32, 8, RES><<<p.nblk, 128, 0, st>>>(a);
        else ln_bwd_kernel<T, P, VEC, 32, 16, RES><<<p.nblk, 128, 0, st>>>(a);
        break;
    case 64: ln_bwd_kernel<T, P, VEC, 64, 16, RES><<<p.nblk, 128, 0, st>>>(a); break;
    case 128: ln_bwd_kernel<T, P, VEC, 128, 16, RES><<<p.nblk, 128, 0, st>>>(a); break;
    case 256: ln_bwd_kernel<T, P, VEC, 256, 16, RES><<<p.nblk, 256, 0, st>>>(a); break;
    case 512: ln_bwd_kernel<T, P, VEC, 512, 16, RES><<<p.nblk, 512, 0, st>>>(a); break;
    default: {
        ln_bwd_rowsums_kernel<T, P><<<(unsigned)a.rows, 512, 0, st>>>(a);
        const dim3 grid((unsigned)((a.cols + kWideCols - 1) / kWideCols), (unsigned)p.nblk);
        ln_bwd_wide_kernel<T, P><<<grid, 256, 0, st>>>(a);
    }
    }
    return cudaGetLastError();
}

// Calls f(T{}, P{}) with the descriptor's element and parameter types.
template <typename F>
cudaError_t with_types(const cba_layernorm_desc_t &d, F f) {
    const bool pf = d.param_type == CBA_F32;
    switch (d.type) {
    case CBA_F32: return f(float{}, float{});
    case CBA_F16: return pf ? f(__half{}, float{}) : f(__half{}, __half{});
    default: return pf ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
    }
}

int check_desc(const cba_layernorm_desc_t *d) {
    if (!d || d->rows < 0 || d->cols < 1) return CBA_ERR_ARG;
    if (!dtype_ok(d->type) || !dtype_ok(d->param_type)) return CBA_ERR_ARG;
    if (d->accumulate != 0 && d->accumulate != 1) return CBA_ERR_ARG;
    if (!(std::isfinite(d->eps) && d->eps >= 0.f)) return CBA_ERR_ARG;
    const long long lds[] = {d->ld_x, d->ld_y, d->ld_dy, d->ld_dx, d->ld_residual};
    for (long long l : lds) {
        if (l != 0 && l < d->cols) return CBA_ERR_ARG;
        if (l > (1LL << 31)) return CBA_ERR_UNSUPPORTED;
    }
    if (d->param_type != CBA_F32 && d->param_type != d->type) return CBA_ERR_UNSUPPORTED;
    if (d->rows >= (1LL << 31) || d->cols > (1 << 30)) return CBA_ERR_UNSUPPORTED;
    return CBA_OK;
}

// 16-byte accesses: whole vectors in every row, aligned bases and strides.
bool vector_ok(const cba_layernorm_desc_t &d, std::initializer_list<const void *> ptrs,
               std::initializer_list<long long> lds) {
    const int vec = 16 / (int)dtype_bytes(d.type);
    if (d.cols % vec) return false;
    for (const void *p : ptrs)
        if (!aligned_to(p, 16)) return false;
    for (long long l : lds)
        if (l % vec) return false;
    return true;
}

bool elements_aligned(size_t e, std::initializer_list<const void *> ptrs) {
    for (const void *p : ptrs)
        if (!aligned_to(p, e)) return false;
    return true;
}

}  // namespace

}  // namespace cba

using namespace cba;

extern "C" {

int cba_layernorm_forward(const cba_layernorm_desc_t *d, const void *x, const void *gamma,
                          const void *beta, void *y, float *mean, float *rstd, void *stream) {
    const int rc = check_desc(d);
    if (rc != CBA_OK) return rc;
    if (d->rows == 0) return CBA_OK;
    if (!x || !y) return CBA_ERR_ARG;
    if (!elements_aligned(dtype_bytes(d->type), {x, y}) ||
        !elements_aligned(dtype_bytes(d->param_type), {gamma, beta}) ||
        !elements_aligned(4, {mean, rstd}))
        return CBA_ERR_ALIGN;
    LnArgs a{};
    a.x = x; a.gamma = gamma; a.beta = beta; a.y = y; a.mean = mean; a.rstd = rstd;
    a.rows = d->rows; a.cols = d->cols; a.eps = d->eps; a.inv_cols = 1.f / (float)d->cols;
    a.ld_x = d->ld_x ? d->ld_x : d->cols;
    a.ld_y = d->ld_y ? d->ld_y : d->cols;
    cudaGetLastError();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = select_device_of(y);
    if (e == cudaSuccess) {
        const bool v = vector_ok(*d, {x, gamma, beta, y}, {a.ld_x, a.ld_y});
        e = with_types(*d, [&](auto t, auto p) {
            using T = decltype(t);
            using P = decltype(p);
            return v ? fwd_vec<T, P, 16 / sizeof(T)>(a, st) : fwd_vec<T, P, 1>(a, st);
        });
    }
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

size_t cba_layernorm_workspace_bytes(const cba_layernorm_desc_t *d) {
    if (check_desc(d) != CBA_OK) return 0;
    // whether rows move as vectors depends on the call's pointers: room for both (and with a
    // residual there are no more blocks)
    return std::max(ln_bwd_plan(*d, false, false).total, ln_bwd_plan(*d, true, false).total);
}

int cba_layernorm_backward(const cba_layernorm_desc_t *d, const void *x, const void *dy,
                           const void *gamma, const float *mean, const float *rstd,
                           const void *residual, void *dx, float *dgamma, float *dbeta,
                           void *workspace, size_t workspace_bytes, void *stream) {
    const int rc = check_desc(d);
    if (rc != CBA_OK) return rc;
    if (d->rows > 0 && (!x || !dy || !mean || !rstd || !dx)) return CBA_ERR_ARG;
    if (!elements_aligned(dtype_bytes(d->type), {x, dy, residual, dx}) ||
        !elements_aligned(dtype_bytes(d->param_type), {gamma}) ||
        !elements_aligned(4, {mean, rstd, dgamma, dbeta}))
        return CBA_ERR_ALIGN;
    if (!workspace || workspace_bytes < cba_layernorm_workspace_bytes(d)) return CBA_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return CBA_ERR_ALIGN;
    LnArgs a{};
    a.x = x; a.dy = dy; a.gamma = gamma; a.residual = residual; a.dx = dx;
    a.mean_in = mean; a.rstd_in = rstd;
    a.part = static_cast<float *>(workspace);
    a.rows = d->rows; a.cols = d->cols; a.inv_cols = 1.f / (float)d->cols;
    a.ld_x = d->ld_x ? d->ld_x : d->cols;
    a.ld_dy = d->ld_dy ? d->ld_dy : d->cols;
    a.ld_dx = d->ld_dx ? d->ld_dx : d->cols;
    a.ld_res = d->ld_residual ? d->ld_residual : d->cols;
    cudaGetLastError();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = select_device_of(workspace);
    const bool v = vector_ok(*d, {x, dy, gamma, residual, dx}, {a.ld_x, a.ld_dy, a.ld_dx, residual ? a.ld_res : 0});
    const LnPlan p = ln_bwd_plan(*d, v, residual != nullptr);
    a.rowc = ws_at<float2>(workspace, p.off_rowc);
    if (e == cudaSuccess && d->rows > 0) {
        e = with_types(*d, [&](auto t, auto pt) {
            using T = decltype(t);
            using P = decltype(pt);
            constexpr int V = 16 / sizeof(T);
            if (residual) return v ? bwd_vec<T, P, V, true>(a, p, st) : bwd_vec<T, P, 1, true>(a, p, st);
            return v ? bwd_vec<T, P, V, false>(a, p, st) : bwd_vec<T, P, 1, false>(a, p, st);
        });
    }
    if (e == cudaSuccess && (dgamma || dbeta))
        e = launch_pdl(ln_colsum_kernel, dim3((unsigned)((d->cols + 31) / 32), 2), dim3(1024), 0, st,
                       a.part, p.nblk, d->cols, d->accumulate, dgamma, dbeta);
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

}  // extern "C"
