// cba_qknorm.cu -- norms of queries and keys for each head with the rotation by
// position in the same pass, forward and backward.
//
//   r = 1 / sqrt(mean_c x^2 + eps),  n = x r,  h = n gamma,  y = R h
//   g = R^T dy,  dgamma = sum g n,  w = g gamma,  dx = r (w - n mean_c(w n))
//   R turns the pair (a, b) to (a cos - b sin, a sin + b cos); cos and sin from the
//   table's row of the token's position, elements past rot_dim stay
//
// Each element is read once and each result written once: the bound is memory.  A
// head's elements lie in the registers of 1 to 32 lanes, 8 (PAIRS_SPLIT: 8 of each
// half) to a lane, and its sums are shuffles.  A warp takes a token's heads in
// turn, kSteps x 32 / lanes of them, with all their loads ahead of the first use.
#include <algorithm>
#include <cmath>

#include "cba_internal.cuh"
#include "cba_ptx.cuh"
#include "cba_types.cuh"

namespace cba {

namespace {

constexpr int kQkMaxDim = 256;
constexpr int kWarps = 8;                     // of a block
constexpr int kSteps = 4, kBwdSteps = 2;      // heads of a lane in flight
constexpr int kBwdBlocks = 2 * kNumSMs;       // at most; one partial row of dgamma each

// Where the two elements of a pair lie.
enum Pairs {
    PAIRS_LOCAL,  // (2j, 2j + 1), or no rotation: in one lane's 8 elements
    PAIRS_SPLIT,  // (j, j + dim / 2) with dim / 2 a multiple of 8: a lane holds 8 of either half
    PAIRS_ANY     // (j, j + rot / 2): exchanged through shared memory
};

struct QkArgs {
    // queries and keys
    const void *x[2], *dy[2], *gamma[2];
    void *out[2];
    long long sx[2][3], sdy[2][3], so[2][3];  // batch, token, head
    int heads[2], parts[2];                   // parts: a warp's tasks per token
    const float2 *table;
    const int *pos;
    int tokens, len, dim, rot, positions, norm;
    float sign, eps, inv_dim;                 // sign: -1 turns back
    int lanes_log;                            // lanes of a head
    int q_blocks;                             // backward: blocks of the queries
    float *partial;
};

template <typename T>
using Vec = Pack<T, 8>;

template <typename T>
__device__ __forceinline__ Vec<T> load8(const void *p, long long at) {
    Vec<T> v;
    const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const T *>(p) + at);
#pragma unroll
    for (int i = 0; i < (int)sizeof(Vec<T>) / 16; ++i) reinterpret_cast<uint4 *>(&v)[i] = s[i];
    return v;
}
template <typename T>
__device__ __forceinline__ void store8(void *p, long long at, const Vec<T> &v) {
    uint4 *s = reinterpret_cast<uint4 *>(static_cast<T *>(p) + at);
#pragma unroll
    for (int i = 0; i < (int)sizeof(Vec<T>) / 16; ++i) s[i] = reinterpret_cast<const uint4 *>(&v)[i];
}

// A lane's place in its head and the angles of its elements at one position.
template <int PAIRS>
struct Lane {
    static constexpr int NV = PAIRS == PAIRS_SPLIT ? 2 : 1;  // vectors of 8 elements
    static constexpr int NE = 8 * NV;
    static constexpr int NC = PAIRS == PAIRS_LOCAL ? 4 : 8;  // angles
    int slot, l, at[NV];
    bool on;
    float cs[NC], sn[NC];

    __device__ __forceinline__ Lane(const QkArgs &a) {
        const int lane = threadIdx.x & 31;
        slot = lane >> a.lanes_log;
        l = lane & ((1 << a.lanes_log) - 1);
        at[0] = l * 8;
        if constexpr (NV == 2) at[1] = a.dim / 2 + l * 8;
        on = l * 8 < a.dim / NV;
    }
    // (an element past rot_dim turns by the angle 0)
    __device__ __forceinline__ void angles(const QkArgs &a, int token) {
        if (a.rot == 0) {
#pragma unroll
            for (int i = 0; i < NC; ++i) cs[i] = 1.f, sn[i] = 0.f;
            return;
        }
        const int p = min(max(a.pos ? a.pos[token] : token % a.len, 0), a.positions - 1);
        const float2 *row = a.table + (long long)p * (a.rot / 2);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            int j;
            bool in;
            if constexpr (PAIRS == PAIRS_LOCAL) {
                j = l * 4 + i, in = on && j < a.rot / 2;
            } else if constexpr (PAIRS == PAIRS_SPLIT) {
                j = l * 8 + i, in = on;
            } else {
                const int e = l * 8 + i;
                j = e < a.rot / 2 ? e : e - a.rot / 2, in = on && e < a.rot;
            }
            const float2 v = in ? __ldg(row + j) : make_float2(1.f, 0.f);
            cs[i] = v.x;
            sn[i] = a.sign * v.y;
        }
    }
    // The sum over the lanes of a head.
    __device__ __forceinline__ float head_sum(const QkArgs &a, float v) const {
        for (int o = (1 << a.lanes_log) >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    // Turns h in place; `inverse`: by the opposite angles.  buf: the warp's 256 floats.
    __device__ __forceinline__ void turn(const QkArgs &a, float (&h)[NE], float *buf) const {
        if constexpr (PAIRS == PAIRS_LOCAL) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = h[2 * i], y = h[2 * i + 1];
                h[2 * i] = x * cs[i] - y * sn[i];
                h[2 * i + 1] = x * sn[i] + y * cs[i];
            }
        } else if constexpr (PAIRS == PAIRS_SPLIT) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = h[i], y = h[8 + i];
                h[i] = x * cs[i] - y * sn[i];
                h[8 + i] = x * sn[i] + y * cs[i];
            }
        } else {
            float *mine = buf + (slot << a.lanes_log) * 8;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) mine[l * 8 + i] = h[i];
            __syncwarp();
            const int half = a.rot / 2;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = l * 8 + i;
                if (e < half) h[i] = h[i] * cs[i] - mine[e + half] * sn[i];
                else if (e < a.rot) h[i] = h[i] * cs[i] + mine[e - half] * sn[i];
            }
        }
    }
    // 1 / sqrt(mean x^2 + eps) of a head.  Squares that overflow are summed again at
    // 2^-66 times the elements: the mean is then so large that eps does not count.
    __device__ __forceinline__ float rnorm(const QkArgs &a, const float (&x)[NE]) const {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) s = fmaf(x[i], x[i], s);
        s = head_sum(a, s);
        float r = 1.f / sqrtf(fmaf(s, a.inv_dim, a.eps));
        if (__any_sync(0xffffffffu, !(s < INFINITY))) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const float y = x[i] * 0x1p-66f;
                t = fmaf(y, y, t);
            }
            t = head_sum(a, t);
            if (!(s < INFINITY)) r = 0x1p-66f / sqrtf(t * a.inv_dim);
        }
        return r;
    }
};

template <typename P, int NE, int NV>
__device__ __forceinline__ void load_gamma(const void *gamma, const int (&at)[NV], bool on, float (&g)[NE]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        Vec<P> p;
        if (gamma && on) p = load8<P>(gamma, at[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[v * 8 + i] = gamma && on ? to_f32(p.v[i]) : 1.f;
    }
}

template <typename T, int NE, int NV>
__device__ __forceinline__ void unpack(const Vec<T> (&v)[NV], bool on, float (&x)[NE]) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k * 8 + i] = on ? to_f32(v[k].v[i]) : 0.f;
}

template <typename T, typename P, int PAIRS>
__global__ void __launch_bounds__(kWarps * 32) qk_fwd_kernel(const QkArgs a) {
    using L = Lane<PAIRS>;
    constexpr int NV = L::NV, NE = L::NE;
    __shared__ float bufs[PAIRS == PAIRS_ANY ? kWarps * 256 : 1];
    const int warp = threadIdx.x >> 5, parts = a.parts[0] + a.parts[1];
    const unsigned task = blockIdx.x * kWarps + warp;
    const int token = (int)(task / parts);
    if (token >= a.tokens) return;
    int part = (int)(task - (unsigned)token * parts);
    const int w = part >= a.parts[0];
    if (w) part -= a.parts[0];
    L lane(a);
    const int per = 32 >> a.lanes_log;
    const long long b = token / a.len, t = token - b * a.len;
    const long long x0 = b * a.sx[w][0] + t * a.sx[w][1], o0 = b * a.so[w][0] + t * a.so[w][1];
    Vec<T> px[kSteps][NV];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const int h = (part * kSteps + u) * per + lane.slot;
        if (lane.on && h < a.heads[w])
#pragma unroll
            for (int v = 0; v < NV; ++v) px[u][v] = load8<T>(a.x[w], x0 + h * a.sx[w][2] + lane.at[v]);
    }
    lane.angles(a, token);
    float gamma[NE];
    load_gamma<P>(a.gamma[w], lane.at, lane.on, gamma);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        const int first = (part * kSteps + u) * per, h = first + lane.slot;
        if (first >= a.heads[w]) break;  // the whole warp
        const bool on = lane.on && h < a.heads[w];
        float x[NE];
        unpack<T>(px[u], on, x);
        if (a.norm) {
            const float r = lane.rnorm(a, x);
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = x[i] * r * gamma[i];
        }
        lane.turn(a, x, bufs + warp * (PAIRS == PAIRS_ANY ? 256 : 0));
        if (on) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                Vec<T> y;
#pragma unroll
                for (int i = 0; i < 8; ++i) y.v[i] = from_f32<T>(x[v * 8 + i]);
                store8<T>(a.out[w], o0 + h * a.so[w][2] + lane.at[v], y);
            }
        }
    }
}

// Blocks below q_blocks walk the queries' tasks, the others the keys'; a warp adds
// up its lanes' parts of dgamma, a block its warps', in a fixed order.
template <typename T, typename P, int PAIRS>
__global__ void __launch_bounds__(kWarps * 32, 2) qk_bwd_kernel(const QkArgs a) {
    using L = Lane<PAIRS>;
    constexpr int NV = L::NV, NE = L::NE;
    __shared__ float bufs[kWarps * 256];
    const int warp = threadIdx.x >> 5, lane_id = threadIdx.x & 31;
    ptx::griddep_launch_dependents();
    const int w = (int)blockIdx.x >= a.q_blocks;
    const unsigned blk = w ? blockIdx.x - a.q_blocks : blockIdx.x, blks = w ? gridDim.x - a.q_blocks : a.q_blocks;
    const unsigned tasks = (unsigned)a.tokens * a.parts[w];
    L lane(a);
    const int per = 32 >> a.lanes_log;
    float gamma[NE], dg[NE];
    load_gamma<P>(a.gamma[w], lane.at, lane.on, gamma);
#pragma unroll
    for (int i = 0; i < NE; ++i) dg[i] = 0.f;
    for (unsigned task = blk * kWarps + warp; task < tasks; task += blks * kWarps) {
        const int token = (int)(task / a.parts[w]), part = (int)(task - (unsigned)token * a.parts[w]);
        const long long b = token / a.len, t = token - b * a.len;
        const long long x0 = b * a.sx[w][0] + t * a.sx[w][1], o0 = b * a.so[w][0] + t * a.so[w][1],
                        d0 = b * a.sdy[w][0] + t * a.sdy[w][1];
        Vec<T> px[kBwdSteps][NV], pd[kBwdSteps][NV];
#pragma unroll
        for (int u = 0; u < kBwdSteps; ++u) {
            const int h = (part * kBwdSteps + u) * per + lane.slot;
            if (lane.on && h < a.heads[w])
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    px[u][v] = load8<T>(a.x[w], x0 + h * a.sx[w][2] + lane.at[v]);
                    pd[u][v] = load8<T>(a.dy[w], d0 + h * a.sdy[w][2] + lane.at[v]);
                }
        }
        lane.angles(a, token);
#pragma unroll
        for (int u = 0; u < kBwdSteps; ++u) {
            const int first = (part * kBwdSteps + u) * per, h = first + lane.slot;
            if (first >= a.heads[w]) break;
            const bool on = lane.on && h < a.heads[w];
            float x[NE], g[NE];
            unpack<T>(px[u], on, x);
            unpack<T>(pd[u], on, g);
            lane.turn(a, g, bufs + warp * 256);
            const float r = lane.rnorm(a, x);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                x[i] = on ? x[i] * r : 0.f;  // n (of a lane without a head r may be infinite)
                dg[i] = fmaf(g[i], x[i], dg[i]);
                g[i] *= gamma[i];
                s = fmaf(g[i], x[i], s);
            }
            s = lane.head_sum(a, s) * a.inv_dim;
            if (on) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    Vec<T> y;
#pragma unroll
                    for (int i = 0; i < 8; ++i) y.v[i] = from_f32<T>(r * (g[v * 8 + i] - x[v * 8 + i] * s));
                    store8<T>(a.out[w], o0 + h * a.so[w][2] + lane.at[v], y);
                }
            }
        }
    }
    // the heads of a warp side by side, then the block's warps
#pragma unroll
    for (int i = 0; i < NE; ++i)
        for (int o = 16; o >= 1 << a.lanes_log; o >>= 1) dg[i] += __shfl_xor_sync(0xffffffffu, dg[i], o);
    __syncwarp();
    if (lane_id < 1 << a.lanes_log && lane.on)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) bufs[warp * 256 + lane.at[v] + i] = dg[v * 8 + i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.dim; c += kWarps * 32) {
        float s = bufs[c];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) s += bufs[k * 256 + c];
        a.partial[(long long)blockIdx.x * a.dim + c] = s;
    }
}

// dgamma of 32 columns of one side: warps take every 32nd partial row, then one adds
// the 32 sums.
__global__ void __launch_bounds__(1024)
    qk_dgamma_kernel(const float *partial, int dim, int q_blocks, int blocks, float *dgq, float *dgk, int accumulate) {
    __shared__ float sums[32][33];
    ptx::griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const int from = blockIdx.y ? q_blocks : 0, to = blockIdx.y ? blocks : q_blocks;
    float *out = blockIdx.y ? dgk : dgq;
    if (!out) return;
    float s = 0.f;
    if (c < dim)
#pragma unroll 4
        for (int i = from + warp; i < to; i += 32) s += partial[(long long)i * dim + c];
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < dim) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += sums[i][lane];
        out[c] = accumulate ? out[c] + s : s;
    }
}

// ---- host side

int check_desc(const cba_qk_norm_rope_desc_t *d) {
    if (!d || d->batch < 1 || d->len < 0 || d->heads_q < 1 || d->heads_k < 0 || d->dim < 1) return CBA_ERR_ARG;
    if (!dtype_ok(d->type) || !dtype_ok(d->param_type)) return CBA_ERR_ARG;
    if ((d->norm != 0 && d->norm != 1) || (d->interleaved != 0 && d->interleaved != 1) ||
        (d->accumulate != 0 && d->accumulate != 1))
        return CBA_ERR_ARG;
    if (d->rot_dim < 0 || d->rot_dim > d->dim || d->rot_dim % 2 != 0 || (d->rot_dim > 0 && d->positions < 1))
        return CBA_ERR_ARG;
    if (!(std::isfinite(d->eps) && d->eps >= 0.f)) return CBA_ERR_ARG;
    if (d->param_type != CBA_F32 && d->param_type != d->type) return CBA_ERR_UNSUPPORTED;
    if (d->dim % 8 != 0 || d->dim > kQkMaxDim) return CBA_ERR_UNSUPPORTED;
    // tasks are counted in 32 bits: one per token and head at most
    if ((double)d->batch * d->len * ((double)d->heads_q + d->heads_k + 2) >= 2147483648.0) return CBA_ERR_UNSUPPORTED;
    const int vec = 16 / (int)dtype_bytes(d->type);
    const cba_attn_strides_t *ss[] = {&d->q, &d->k, &d->yq, &d->yk, &d->dyq, &d->dyk, &d->dq, &d->dk};
    for (int i = 0; i < 8; ++i) {
        const long long v[] = {ss[i]->batch, ss[i]->token, ss[i]->head};
        if (!v[0] && !v[1] && !v[2]) continue;  // contiguous
        const long long n[] = {d->batch, d->len, i % 2 ? d->heads_k : d->heads_q};
        for (int j = 0; j < 3; ++j) {
            if (v[j] < 0 || (n[j] > 1 && v[j] < d->dim)) return CBA_ERR_ARG;
            if (v[j] % vec != 0) return CBA_ERR_ALIGN;
            if (v[j] >= (1LL << 38)) return CBA_ERR_UNSUPPORTED;
        }
    }
    return CBA_OK;
}

void strides_of(const cba_qk_norm_rope_desc_t &d, const cba_attn_strides_t &s, int heads, long long *out) {
    const bool none = !s.batch && !s.token && !s.head;
    out[0] = none ? (long long)d.len * heads * d.dim : s.batch;
    out[1] = none ? (long long)heads * d.dim : s.token;
    out[2] = none ? d.dim : s.head;
}

Pairs pairs_of(const cba_qk_norm_rope_desc_t &d) {
    if (d.interleaved || d.rot_dim == 0) return PAIRS_LOCAL;
    return d.rot_dim == d.dim && d.dim % 16 == 0 ? PAIRS_SPLIT : PAIRS_ANY;
}

// What both directions share; `steps`: a warp's heads per lane.
QkArgs base_args(const cba_qk_norm_rope_desc_t &d, const float *table, const int *pos, int steps) {
    QkArgs a{};
    a.table = reinterpret_cast<const float2 *>(table);
    a.pos = pos;
    a.tokens = d.batch * d.len;
    a.len = d.len;
    a.dim = d.dim;
    a.rot = d.rot_dim;
    a.positions = d.positions;
    a.norm = d.norm;
    a.sign = 1.f;
    a.eps = d.eps;
    a.inv_dim = 1.f / (float)d.dim;
    const int lanes = pairs_of(d) == PAIRS_SPLIT ? d.dim / 16 : d.dim / 8;
    while ((1 << a.lanes_log) < lanes) ++a.lanes_log;
    const int per = (32 >> a.lanes_log) * steps;
    a.heads[0] = d.heads_q;
    a.heads[1] = d.heads_k;
    for (int w = 0; w < 2; ++w) a.parts[w] = (a.heads[w] + per - 1) / per;
    return a;
}

// Blocks of the backward pass, and the queries' among them: as many as have a task
// for each warp, shared by the heads.
void plan_blocks(const cba_qk_norm_rope_desc_t &d, int *blocks, int *q_blocks) {
    const QkArgs a = base_args(d, nullptr, nullptr, kBwdSteps);
    long long need[2];
    for (int w = 0; w < 2; ++w) need[w] = ((long long)a.tokens * a.parts[w] + kWarps - 1) / kWarps;
    if (need[0] + need[1] > kBwdBlocks) {
        const long long all = need[0] + need[1];
        need[1] = d.heads_k ? std::max(1LL, kBwdBlocks * need[1] / all) : 0;
        need[0] = kBwdBlocks - need[1];
    }
    *q_blocks = (int)need[0];
    *blocks = (int)(need[0] + need[1]);
}

template <typename F>
cudaError_t dispatch(const cba_qk_norm_rope_desc_t &d, F f) {
    auto pairs = [&](auto t, auto p) {
        switch (pairs_of(d)) {
            case PAIRS_LOCAL: return f(t, p, std::integral_constant<int, PAIRS_LOCAL>{});
            case PAIRS_SPLIT: return f(t, p, std::integral_constant<int, PAIRS_SPLIT>{});
            default: return f(t, p, std::integral_constant<int, PAIRS_ANY>{});
        }
    };
    auto param = [&](auto t) { return d.param_type == CBA_F32 ? pairs(t, 0.f) : pairs(t, t); };
    return d.type == CBA_F32 ? param(0.f) : d.type == CBA_F16 ? param(__half{}) : param(__nv_bfloat16{});
}

cudaError_t launch_fwd(const cba_qk_norm_rope_desc_t &d, const QkArgs &a, cudaStream_t st) {
    const long long tasks = (long long)a.tokens * (a.parts[0] + a.parts[1]);
    return dispatch(d, [&](auto t, auto p, auto pairs) {
        qk_fwd_kernel<decltype(t), decltype(p), pairs()><<<(unsigned)((tasks + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(a);
        return cudaGetLastError();
    });
}

// The pointers that either direction needs, NULL and alignment.
int check_shared(const cba_qk_norm_rope_desc_t &d, const void *const *need, int n, const void *gamma_q, const void *gamma_k,
                 const float *table, const int *pos) {
    if (d.len > 0) {
        for (int i = 0; i < n; ++i)
            if (!need[i] && (i % 2 == 0 || d.heads_k > 0)) return CBA_ERR_ARG;
        if (d.rot_dim > 0 && (!table || (!pos && d.len > d.positions))) return CBA_ERR_ARG;
    }
    if (!d.norm && (gamma_q || gamma_k)) return CBA_ERR_ARG;
    for (int i = 0; i < n; ++i)
        if (!aligned_to(need[i], 16)) return CBA_ERR_ALIGN;
    if (!aligned_to(gamma_q, 16) || !aligned_to(gamma_k, 16) || !aligned_to(table, 16) || !aligned_to(pos, 4))
        return CBA_ERR_ALIGN;
    return CBA_OK;
}

}  // namespace

}  // namespace cba

using namespace cba;

extern "C" {

int cba_qk_norm_rope_forward(const cba_qk_norm_rope_desc_t *d, const void *q, const void *k,
                             const void *gamma_q, const void *gamma_k, const float *table,
                             const int *pos, void *yq, void *yk, void *stream) {
    int rc = check_desc(d);
    if (rc != CBA_OK) return rc;
    const void *need[] = {q, k, yq, yk};
    rc = check_shared(*d, need, 4, gamma_q, gamma_k, table, pos);
    if (rc != CBA_OK) return rc;
    if (d->len == 0) return CBA_OK;
    QkArgs a = base_args(*d, table, pos, kSteps);
    a.x[0] = q; a.x[1] = k;
    a.gamma[0] = gamma_q; a.gamma[1] = gamma_k;
    a.out[0] = yq; a.out[1] = yk;
    strides_of(*d, d->q, d->heads_q, a.sx[0]);
    strides_of(*d, d->k, d->heads_k, a.sx[1]);
    strides_of(*d, d->yq, d->heads_q, a.so[0]);
    strides_of(*d, d->yk, d->heads_k, a.so[1]);
    cudaGetLastError();
    cudaError_t e = select_device_of(yq);
    if (e == cudaSuccess) e = launch_fwd(*d, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

size_t cba_qk_norm_rope_workspace_bytes(const cba_qk_norm_rope_desc_t *d) {
    if (check_desc(d) != CBA_OK) return 0;
    int blocks, q_blocks;
    plan_blocks(*d, &blocks, &q_blocks);
    return std::max((size_t)256, ((size_t)blocks * d->dim * sizeof(float) + 255) / 256 * 256);
}

int cba_qk_norm_rope_backward(const cba_qk_norm_rope_desc_t *d, const void *q, const void *k,
                              const void *gamma_q, const void *gamma_k, const float *table,
                              const int *pos, const void *dyq, const void *dyk, void *dq, void *dk,
                              float *dgamma_q, float *dgamma_k, void *workspace,
                              size_t workspace_bytes, void *stream) {
    int rc = check_desc(d);
    if (rc != CBA_OK) return rc;
    // without the norm the gradient does not depend on q and k
    const void *need[] = {dyq, dyk, dq, dk, d->norm ? q : dyq, d->norm ? k : dyk};
    rc = check_shared(*d, need, 6, gamma_q, gamma_k, table, pos);
    if (rc != CBA_OK) return rc;
    if (!d->norm && (dgamma_q || dgamma_k)) return CBA_ERR_ARG;
    if (!aligned_to(dgamma_q, 4) || !aligned_to(dgamma_k, 4)) return CBA_ERR_ALIGN;
    if (!workspace || workspace_bytes < cba_qk_norm_rope_workspace_bytes(d)) return CBA_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return CBA_ERR_ALIGN;
    QkArgs a = base_args(*d, table, pos, d->norm ? kBwdSteps : kSteps);
    a.sign = -1.f;
    a.x[0] = d->norm ? q : dyq; a.x[1] = d->norm ? k : dyk;
    a.dy[0] = dyq; a.dy[1] = dyk;
    a.gamma[0] = gamma_q; a.gamma[1] = gamma_k;
    a.out[0] = dq; a.out[1] = dk;
    strides_of(*d, d->norm ? d->q : d->dyq, d->heads_q, a.sx[0]);
    strides_of(*d, d->norm ? d->k : d->dyk, d->heads_k, a.sx[1]);
    strides_of(*d, d->dyq, d->heads_q, a.sdy[0]);
    strides_of(*d, d->dyk, d->heads_k, a.sdy[1]);
    strides_of(*d, d->dq, d->heads_q, a.so[0]);
    strides_of(*d, d->dk, d->heads_k, a.so[1]);
    cudaGetLastError();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = select_device_of(workspace);
    if (e == cudaSuccess && !d->norm) {
        if (d->len > 0) e = launch_fwd(*d, a, st);
        return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
    }
    int blocks;
    plan_blocks(*d, &blocks, &a.q_blocks);
    a.partial = static_cast<float *>(workspace);
    if (e == cudaSuccess && blocks > 0)
        e = dispatch(*d, [&](auto t, auto p, auto pairs) {
            qk_bwd_kernel<decltype(t), decltype(p), pairs()><<<(unsigned)blocks, kWarps * 32, 0, st>>>(a);
            return cudaGetLastError();
        });
    if (e == cudaSuccess && (dgamma_q || dgamma_k)) {
        const dim3 grid((unsigned)(d->dim + 31) / 32, 2);
        if (blocks > 0)
            e = launch_pdl(qk_dgamma_kernel, grid, dim3(1024), 0, st, (const float *)a.partial, d->dim, a.q_blocks, blocks,
                           dgamma_q, dgamma_k, d->accumulate);
        else
            qk_dgamma_kernel<<<grid, 1024, 0, st>>>(a.partial, d->dim, 0, 0, dgamma_q, dgamma_k, d->accumulate);
        if (e == cudaSuccess) e = cudaGetLastError();
    }
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

}  // extern "C"
