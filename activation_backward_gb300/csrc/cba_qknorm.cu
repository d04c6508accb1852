// cba_qknorm.cu -- norms of queries and keys for each head with the rotation by
// position in the same pass, forward and backward.
//
//   r = 1 / sqrt(mean_c x^2 + eps),  n = x r,  h = n gamma,  y = R h
//   g = R^T dy,  dgamma = sum g n,  w = g gamma,  dx = r (w - n mean_c(w n))
//   R turns the pair (a, b) to (a cos - b sin, a sin + b cos); cos and sin from the
//   table's row of the token's position, elements past rot_dim stay
//
// Each element is read once and each result written once: the bound is memory.  A
// head's elements lie in the registers of 1 to 32 lanes, 8 (or 8 of each
// half) to a lane, and its sums are shuffles.  A warp walks tokens and, within one, its
// heads, 32 / lanes of them a step; lanes copy their own elements asynchronously to
// shared memory a few steps ahead, and the warp its tokens' rows of the table.  Blocks
// are the queries' or the keys', in the proportion of their steps.
//
// Measured (us), 4 x 8192 tokens, 32/8 heads of 128, bf16: forward 134 (0.74 of the copy rate; issue
// slots 51% taken), backward 187, of which 6 for the sum of dgamma's rows (0.80; 57%).  2 x 169
// tokens, 8 heads of 64: 5.8 and 9.7, one and two launches (3.5 and 6.4 on the device).
#include <algorithm>
#include <cmath>

#include "cba_internal.cuh"
#include "cba_ptx.cuh"
#include "cba_types.cuh"

namespace cba {

namespace {

constexpr int kQkMaxDim = 256;
constexpr int kWarps = 8;                     // of a block
// Steps in flight; blocks per SM.  (Above: forward 4 steps 134 us, 6 136; backward 2 steps 185, 4
// 192; 3 blocks, whose registers spill, 195 and 340; without shared memory 190 and 294.)
__host__ __device__ constexpr int qk_ahead(bool bwd) { return bwd ? 2 : 4; }
constexpr int kQkPerSm = 2;

// Where the two elements of a pair lie.  A lane has 8 elements of a head, or, where dim is a multiple of
// 16, 8 of either half: a step's sums and addresses cost what they cost for 8.  (2 x 8192 tokens, 16/4
// heads of 128, half of each turned, forward and backward: 47.5 and 67 us, with 8 elements 60 and 77; pairs
// (2j, 2j + 1): 48 and 68, with 8 elements 55 and 73.  2 x 16384, heads of 40: shuffles do not reach,
// through shared memory 86 and 101.)
enum Pairs {
    PAIRS_LOCAL,   // (2j, 2j + 1), or no rotation: in one lane's 8 elements
    PAIRS_LOCAL2,  // the same of either half
    PAIRS_SPLIT,   // (j, j + dim / 2): in the two halves
    PAIRS_LANES,   // (j, j + rot / 2) with rot / 2 a multiple of 8: in two lanes, exchanged by shuffles
    PAIRS_LANES2,  // the same in the first half, with the second beside it
    PAIRS_ANY      // (j, j + rot / 2): exchanged through shared memory
};

__host__ __device__ constexpr bool is_local(int p) { return p == PAIRS_LOCAL || p == PAIRS_LOCAL2; }
__host__ __device__ constexpr bool is_lanes(int p) { return p == PAIRS_LANES || p == PAIRS_LANES2; }

struct QkArgs {
    // queries and keys
    const void *x[2], *dy[2], *gamma[2];
    void *out[2];
    long long sx[2][3], sdy[2][3], so[2][3];  // batch, token, head
    int heads[2], steps[2];                   // steps: of a token
    int parts[2];                             // warps that share a token's heads: 1, 2, 4 or 8
    const float2 *table;
    const int *pos;
    int tokens, len, dim, rot, positions, norm;
    float sign, eps, inv_dim;                 // sign: -1 turns back
    int lanes_log;                            // lanes of a head
    int q_blocks;                             // blocks of the queries
    int warp_bytes, row_bytes;                // shared memory of a warp, of a row of the table
    float *partial;                           // backward: a row of dgamma per block
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
// Elements 2 j and 2 j + 1 of a vector, a word at a time (halves put together one by one
// cost as many instructions again), and the other way.
template <typename T>
__device__ __forceinline__ float2 two_of(const Vec<T> &v, int j) {
    if constexpr (sizeof(T) == 4) return make_float2(v.v[2 * j], v.v[2 * j + 1]);
    const uint32_t u = reinterpret_cast<const uint32_t *>(&v)[j];
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ void set_two(Vec<T> &v, int j, float2 x) {
    if constexpr (sizeof(T) == 4) {
        v.v[2 * j] = x.x, v.v[2 * j + 1] = x.y;
    } else if constexpr (std::is_same<T, __half>::value) {
        reinterpret_cast<__half2 *>(&v)[j] = __float22half2_rn(x);
    } else {
        reinterpret_cast<__nv_bfloat162 *>(&v)[j] = __float22bfloat162_rn(x);
    }
}

// Asynchronous copies of this thread, global to shared.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T>
__device__ __forceinline__ void store8(void *p, long long at, const Vec<T> &v) {
    uint4 *s = reinterpret_cast<uint4 *>(static_cast<T *>(p) + at);
#pragma unroll
    for (int i = 0; i < (int)sizeof(Vec<T>) / 16; ++i) s[i] = reinterpret_cast<const uint4 *>(&v)[i];
}

// A lane's place in its head, and what turns its elements at one position.
template <int PAIRS>
struct Lane {
    static constexpr int NV = PAIRS == PAIRS_LOCAL || PAIRS == PAIRS_LANES || PAIRS == PAIRS_ANY ? 1 : 2;  // vectors of 8 elements
    static constexpr int NE = 8 * NV, N2 = NE / 2;
    static constexpr int NC = PAIRS == PAIRS_LOCAL ? 4 : 8;   // angles
    int slot, l, at[NV], lanes, other;  // other: PAIRS_LANES: the lane with the pairs' other elements
    int place[PAIRS == PAIRS_ANY ? 8 : 1];  // of the pairs' other elements in shared memory
    bool on;
    float cs[NC], sn[NC];

    __device__ __forceinline__ Lane(const QkArgs &a) {
        const int lane = threadIdx.x & 31;
        lanes = 1 << a.lanes_log;
        slot = lane >> a.lanes_log;
        l = lane & (lanes - 1);
        at[0] = l * 8;
        if constexpr (NV == 2) at[1] = a.dim / 2 + l * 8;
        on = l * 8 < a.dim / NV;
        const int apart = a.rot / 16;
        other = lane + (l < apart ? apart : l < 2 * apart ? -apart : 0);
        if constexpr (PAIRS == PAIRS_ANY)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = l * 8 + i, half = a.rot / 2;
                place[i] = e < a.rot ? spread(lane * 8 + i + (e < half ? half : -half)) : kZero;
            }
    }
    // PAIRS_ANY: where element i of a warp's 256 lies, so that lanes that read 8 elements apart use
    // different banks; behind them a -0 for elements past rot_dim.
    static constexpr int kZero = 256 + 7, kPlaces = 256 + 8;
    static __device__ __forceinline__ int spread(int i) { return i + (i >> 5); }
    // The angles of a token, from its row of the table.  (Elements past rot_dim: 1 and 0.)
    __device__ __forceinline__ void angles(const QkArgs &a, const float2 *row) {
        if constexpr (PAIRS == PAIRS_SPLIT) {  // (a lane past the head's elements holds zeros, whatever it reads)
            const float4 *r4 = reinterpret_cast<const float4 *>(row + (on ? l * 8 : 0));
            const float2 s2 = make_float2(a.sign, a.sign);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = r4[i];
                const float2 s = ptx::mul2(make_float2(v.y, v.w), s2);
                cs[2 * i] = v.x, cs[2 * i + 1] = v.z;
                sn[2 * i] = s.x, sn[2 * i + 1] = s.y;
            }
        } else if constexpr (is_lanes(PAIRS)) {
            const bool second = l >= a.rot / 16, in = l < a.rot / 8;
            const float4 *r4 = reinterpret_cast<const float4 *>(row + (in ? l * 8 - (second ? a.rot / 2 : 0) : 0));
            const float sign = second ? a.sign : -a.sign;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = r4[i];
                cs[2 * i] = in ? v.x : 1.f, cs[2 * i + 1] = in ? v.z : 1.f;
                sn[2 * i] = in ? sign * v.y : 0.f, sn[2 * i + 1] = in ? sign * v.w : 0.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int e = l * 8 + i;
                const bool second = !is_local(PAIRS) && e >= a.rot / 2;
                const int j = is_local(PAIRS) ? at[i / 4] / 2 + i % 4 : second ? e - a.rot / 2 : e;
                const bool in = on && j < a.rot / 2;
                const float2 v = in ? row[j] : make_float2(1.f, 0.f);
                cs[i] = v.x;
                sn[i] = in ? (is_local(PAIRS) || second ? a.sign : -a.sign) * v.y : 0.f;
            }
        }
    }
    // The sum over the lanes of a head.
    __device__ __forceinline__ float head_sum(float v) const {
        for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    // What a square below 2^-149 loses is 2^-50 of this mean.  Raised, elements are below 2^54, and the
    // smallest number's square is 2^-98.
    static constexpr float kSmallMean = 0x1p-100f, kRaise = 0x1p100f;
    // Turns h in place by the angles.  buf: the warp's kPlaces floats.
    __device__ __forceinline__ void turn(const QkArgs &a, float2 (&h)[N2], float *buf) const {
        if constexpr (is_local(PAIRS)) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const float2 x = h[i];
                // (past rot_dim an infinity times the angle's 0 would be NaN)
                if (at[i / 4] / 2 + i % 4 < a.rot / 2) h[i] = make_float2(x.x * cs[i] - x.y * sn[i], x.x * sn[i] + x.y * cs[i]);
            }
        } else if constexpr (PAIRS == PAIRS_SPLIT) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = h[i], y = h[4 + i];
                const float2 c = make_float2(cs[2 * i], cs[2 * i + 1]), s = make_float2(sn[2 * i], sn[2 * i + 1]);
                h[i] = ptx::fma2(x, c, ptx::mul2(y, make_float2(-s.x, -s.y)));
                h[4 + i] = ptx::fma2(x, s, ptx::mul2(y, c));
            }
        } else if constexpr (is_lanes(PAIRS)) {
            const bool in = l < a.rot / 8;  // (past rot_dim, where an infinity times 0 would be NaN, -0 is added)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 y = make_float2(__shfl_sync(0xffffffffu, h[i].x, other), __shfl_sync(0xffffffffu, h[i].y, other));
                if (!in) y = make_float2(-0.f, -0.f);
                const float2 c = make_float2(cs[2 * i], cs[2 * i + 1]), s = make_float2(sn[2 * i], sn[2 * i + 1]);
                h[i] = ptx::fma2(h[i], c, ptx::mul2(y, s));
            }
        } else {
            float *v = reinterpret_cast<float *>(h);
            const int mine = spread((threadIdx.x & 31) * 8);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) buf[mine + i] = v[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], cs[i], buf[place[i]] * sn[i]);
        }
    }
    // 1 / sqrt(mean x^2 + eps) of a head, r, as r / raise by which x, raised, becomes n.  Squares that
    // overflow are summed again at 2^-70 times the elements, where 256 of the largest have 2^124.
    // Where mean and eps together are below kSmallMean, squares may have lost bits or vanished: x
    // becomes kRaise x, whose squares are summed.  (A branch behind dx for an r past the largest
    // number, a mean below 2^-256, takes 2% of the backward call: 4 x 8192 tokens, 32/8 heads of 128 187 us,
    // 190.)
    __device__ __forceinline__ float rnorm(const QkArgs &a, float2 (&x)[N2], float &raise) const {
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < N2; ++i) q = ptx::fma2(x[i], x[i], q);
        const float s = fmaf(head_sum(q.x + q.y), a.inv_dim, a.eps);
        float r = rsqrtf(s);  // (2 ulp: below the sum's own error)
        const bool large = !(s < INFINITY), small = s < kSmallMean;
        raise = 1.f;
        if (__any_sync(0xffffffffu, large || small)) {
            const float f = large ? 0x1p-70f : small ? kRaise : 1.f;
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < N2; ++i) {
                const float2 y = make_float2(x[i].x * f, x[i].y * f);
                t = fmaf(y.x, y.x, fmaf(y.y, y.y, t));
                if (small) x[i] = y;
            }
            t = rsqrtf(fmaf(head_sum(t), a.inv_dim, a.eps * f * f));
            if (large) r = f * t;
            if (small) r = t, raise = kRaise;
        }
        return r;
    }
};

template <typename P, int N2, int NV>
__device__ __forceinline__ void load_gamma(const void *gamma, const int (&at)[NV], bool on, float2 (&g)[N2]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        Vec<P> p;
        if (gamma && on) p = load8<P>(gamma, at[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[v * 4 + i] = gamma && on ? two_of<P>(p, i) : make_float2(1.f, 1.f);
    }
}

template <typename T, int N2, int NV>
__device__ __forceinline__ void unpack(const Vec<T> (&v)[NV], float2 (&x)[N2]) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[k * 4 + i] = two_of<T>(v[k], i);
}
template <typename T, int N2, int NV>
__device__ __forceinline__ void pack_store(T *out, const int (&at)[NV], const float2 (&x)[N2]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        Vec<T> y;
#pragma unroll
        for (int i = 0; i < 4; ++i) set_two<T>(y, i, x[v * 4 + i]);
        store8<T>(out, at[v], y);
    }
}

// Blocks below q_blocks walk the queries' heads, the others the keys'.  Backward: a warp
// adds up its lanes' parts of dgamma, a block its warps', in a fixed order.
template <typename T, typename P, int PAIRS, bool BWD, bool SHARED>
__global__ void __launch_bounds__(kWarps * 32, kQkPerSm) qk_kernel(const QkArgs a) {
    using L = Lane<PAIRS>;
    constexpr int NV = L::NV, NE = L::NE, N2 = L::N2, AHEAD = qk_ahead(BWD), NT = BWD ? 2 : 1, Q = sizeof(T) / 2;
    constexpr uint32_t STEP = NT * NV * Q * 512;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane_id = threadIdx.x & 31;
    if (BWD) ptx::griddep_launch_dependents();
    const int w = (int)blockIdx.x >= a.q_blocks;
    const int blk = w ? (int)blockIdx.x - a.q_blocks : (int)blockIdx.x;
    // (SHARED: warps share a token's heads; in one kernel for both long calls take 2% longer)
    const int parts = SHARED ? a.parts[w] : 1, own = blk * kWarps + warp;
    // from one token of a warp to its next
    const int stride = (w ? (int)gridDim.x - a.q_blocks : a.q_blocks) * kWarps / parts;
    L lane(a);
    const int per = 32 >> a.lanes_log, share = (a.steps[w] + parts - 1) / parts * per, from = SHARED ? own % parts * share : 0;
    const int heads = SHARED ? min(a.heads[w], from + share) : a.heads[w];  // the end of the warp's
    uint8_t *ring = smem + warp * a.warp_bytes, *rows = ring + AHEAD * STEP;
    float *buf = reinterpret_cast<float *>(rows + (AHEAD + 1) * a.row_bytes);  // PAIRS_ANY
    const uint32_t to = ptx::smem_u32(ring) + lane_id * 16, to_rows = ptx::smem_u32(rows);

    // A token's sequence and index in it, moved on by `stride` tokens.  (Divisions cost as much as a step.)
    struct Place {
        int token, b, t;
    };
    const int sb = stride / a.len, sr = stride - sb * a.len;
    auto begin = [&]() {
        const int token = !SHARED ? own : from < heads ? own / parts : a.tokens, b = token / a.len;
        return Place{token, b, token - b * a.len};
    };
    auto move_on = [&](Place &p) {
        p.token += stride, p.b += sb, p.t += sr;
        if (p.t >= a.len) p.t -= a.len, ++p.b;
    };
    // the copies' place: token, head in it, stage of the ring and of the rows, the next token's position;
    // pointers to the lane's head move on by `per` heads
    const T *fx = nullptr, *fdy = nullptr;
    const long long xs = per * a.sx[w][2], ds = per * a.sdy[w][2], os = per * a.so[w][2];
    Place f = begin();
    int fh = from, fs = 0, fr = 0;
    auto position = [&](const Place &p) {
        if (p.token >= a.tokens || a.rot == 0) return 0;
        return min(max(a.pos ? __ldg(a.pos + p.token) : p.t, 0), a.positions - 1);
    };
    auto place = [&]() {
        fx = static_cast<const T *>(a.x[w]) + f.b * a.sx[w][0] + f.t * a.sx[w][1] + (from + lane.slot) * a.sx[w][2];
        if (BWD) fdy = static_cast<const T *>(a.dy[w]) + f.b * a.sdy[w][0] + f.t * a.sdy[w][1] + (from + lane.slot) * a.sdy[w][2];
    };
    place();
    auto after = [&](Place p) {
        move_on(p);
        return position(p);
    };
    int at_pos = position(f), next_pos = after(f);
    auto fetch = [&]() {
        if (f.token < a.tokens) {
            if (fh == from)
                for (int j = lane_id; j < a.rot / 2; j += 32)
                    copy_async<8>(to_rows + fr * a.row_bytes + j * 8, a.table + (long long)at_pos * (a.rot / 2) + j);
            if (lane.on && fh + lane.slot < heads) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const uint32_t at = to + fs * STEP + (v * Q + q) * 512;
                        copy_async<16>(at, fx + lane.at[v] + q * 4);
                        if (BWD) copy_async<16>(at + NV * Q * 512, fdy + lane.at[v] + q * 4);
                    }
            }
        }
        copies_commit();
        fs = fs + 1 == AHEAD ? 0 : fs + 1;
        fx += xs, fh += per;
        if (BWD) fdy += ds;
        if (fh >= heads) {
            fh = from;
            move_on(f);
            fr = fr == AHEAD ? 0 : fr + 1;
            at_pos = next_pos;
            next_pos = after(f);
            place();
        }
    };
    auto have = [&](int st, int which, bool on, float2 (&x)[N2]) {
        Vec<T> p[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                uint4 u = *reinterpret_cast<const uint4 *>(ring + st * STEP + (which * NV * Q + v * Q + q) * 512 + lane_id * 16);
                if (!on) u = make_uint4(0, 0, 0, 0);
                reinterpret_cast<uint4 *>(&p[v])[q] = u;
            }
        unpack<T>(p, x);
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch();
    if (PAIRS == PAIRS_ANY && lane_id == 0) buf[L::kZero] = -0.f;
    float2 gamma[N2], dg[BWD ? N2 : 1];
    load_gamma<P>(a.gamma[w], lane.at, lane.on, gamma);
    if constexpr (BWD)
#pragma unroll
        for (int i = 0; i < N2; ++i) dg[i] = make_float2(0.f, 0.f);
    int st = 0, row = 0;
    for (Place c = begin(); c.token < a.tokens; move_on(c)) {
        T *out = static_cast<T *>(a.out[w]) + c.b * a.so[w][0] + c.t * a.so[w][1] + (from + lane.slot) * a.so[w][2];
        // forward, PAIRS_SPLIT: (a, b) becomes r (ca a + cb b, da a + db b)
        float2 ca[4], cb[4], da[4], db[4];
        for (int h = from; h < heads; h += per, out += os) {
            copies_wait<AHEAD - 1>();
            if (h == from) {
                __syncwarp();  // the row was copied by all lanes
                lane.angles(a, reinterpret_cast<const float2 *>(rows + row * a.row_bytes));
                __syncwarp();  // read by all before it is copied over
                row = row == AHEAD ? 0 : row + 1;
                if constexpr (!BWD && PAIRS == PAIRS_SPLIT) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 c = make_float2(lane.cs[2 * j], lane.cs[2 * j + 1]), s = make_float2(lane.sn[2 * j], lane.sn[2 * j + 1]);
                        ca[j] = ptx::mul2(gamma[j], c);
                        cb[j] = ptx::mul2(gamma[4 + j], make_float2(-s.x, -s.y));
                        da[j] = ptx::mul2(gamma[j], s);
                        db[j] = ptx::mul2(gamma[4 + j], c);
                    }
                }
            }
            const bool on = lane.on && h + lane.slot < heads;
            float2 x[N2];
            have(st, 0, on, x);
            if constexpr (BWD) {
                float2 g[N2];
                have(st, 1, on, g);
                fetch();
                lane.turn(a, g, buf);
                float raise;
                const float r = lane.rnorm(a, x, raise);
                const float2 r2 = make_float2(r, r);
                float2 q = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < N2; ++e) {
                    if (on) x[e] = ptx::mul2(x[e], r2);  // n (of a lane without a head 0: r may be infinite)
                    dg[e] = ptx::fma2(g[e], x[e], dg[e]);
                    g[e] = ptx::mul2(g[e], gamma[e]);
                    q = ptx::fma2(g[e], x[e], q);
                }
                const float s = lane.head_sum(q.x + q.y) * -a.inv_dim, rx = r * raise;
#pragma unroll
                for (int e = 0; e < N2; ++e) x[e] = ptx::mul2(ptx::fma2(x[e], make_float2(s, s), g[e]), make_float2(rx, rx));
            } else {
                fetch();
                float raise;
                const float r = a.norm ? lane.rnorm(a, x, raise) : 1.f;
                const float2 r2 = make_float2(r, r);
                if constexpr (PAIRS == PAIRS_SPLIT) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 u = ptx::mul2(x[j], r2), v = ptx::mul2(x[4 + j], r2);
                        x[j] = ptx::fma2(u, ca[j], ptx::mul2(v, cb[j]));
                        x[4 + j] = ptx::fma2(u, da[j], ptx::mul2(v, db[j]));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < N2; ++j) x[j] = ptx::mul2(ptx::mul2(x[j], r2), gamma[j]);
                    lane.turn(a, x, buf);
                }
            }
            if (on) pack_store<T>(out, lane.at, x);
            st = st + 1 == AHEAD ? 0 : st + 1;
        }
    }
    if constexpr (BWD) {
    copies_wait<0>();
    __syncthreads();
    float *bufs = reinterpret_cast<float *>(smem);
    // the heads of a warp side by side, then the block's warps
    float sums[NE];
#pragma unroll
    for (int i = 0; i < N2; ++i) sums[2 * i] = dg[i].x, sums[2 * i + 1] = dg[i].y;
#pragma unroll
    for (int i = 0; i < NE; ++i)
        for (int o = 16; o >= lane.lanes; o >>= 1) sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], o);
    if (lane_id < lane.lanes && lane.on)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) bufs[warp * 256 + lane.at[v] + i] = sums[v * 8 + i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.dim; c += kWarps * 32) {
        float s = bufs[c];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) s += bufs[k * 256 + c];
        a.partial[(long long)blockIdx.x * a.dim + c] = s;
    }
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
    // tokens and heads are counted in 32 bits, beside a grid's stride of tokens and a warp's of heads
    if ((double)d->batch * d->len > 2147483648.0 - 65536.0) return CBA_ERR_UNSUPPORTED;
    if (d->heads_q > (1 << 30) || d->heads_k > (1 << 30)) return CBA_ERR_UNSUPPORTED;
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
    const bool halves = d.dim % 16 == 0;
    if (d.interleaved || d.rot_dim == 0) return halves ? PAIRS_LOCAL2 : PAIRS_LOCAL;
    if (d.rot_dim % 16 != 0) return PAIRS_ANY;
    if (d.rot_dim == d.dim) return PAIRS_SPLIT;
    return halves && d.rot_dim <= d.dim / 2 ? PAIRS_LANES2 : PAIRS_LANES;
}

// What both directions share.
QkArgs base_args(const cba_qk_norm_rope_desc_t &d, const float *table, const int *pos) {
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
    const Pairs pairs = pairs_of(d);
    const int lanes = pairs == PAIRS_LOCAL || pairs == PAIRS_LANES || pairs == PAIRS_ANY ? d.dim / 8 : d.dim / 16;
    while ((1 << a.lanes_log) < lanes) ++a.lanes_log;
    const int per = 32 >> a.lanes_log;
    a.heads[0] = d.heads_q;
    a.heads[1] = d.heads_k;
    // Few tokens share their heads among warps, up to a block for each SM.  (32/8 heads, forward and backward:
    // 8 x 1 tokens, heads of 128 3.3 and 5.8 us, a warp for a token's heads 5.8 and 9.7; 4 x 8, heads of 256
    // 3.9 and 6.5, 9.7 and 16.9.)
    for (int w = 0; w < 2; ++w) {
        a.steps[w] = (a.heads[w] + per - 1) / per;
        a.parts[w] = 1;
        while (a.parts[w] < kWarps && 2 * a.parts[w] <= a.steps[w] && 4LL * a.parts[w] * a.tokens <= kNumSMs * kWarps)
            a.parts[w] *= 2;
    }
    a.row_bytes = (d.rot_dim * 4 + 15) / 16 * 16;
    return a;
}

// Blocks, and the queries' among them: as many as have a token (or a part of its heads) for each warp, or that the
// SMs hold, shared by the steps.
void plan_blocks(const cba_qk_norm_rope_desc_t &d, const QkArgs &a, int *blocks, int *q_blocks) {
    const int most = kQkPerSm * kNumSMs;
    const long long each = ((long long)a.tokens + kWarps - 1) / kWarps;
    auto warps = [&](int w) { return ((long long)a.tokens * a.parts[w] + kWarps - 1) / kWarps; };
    long long need[2] = {warps(0), d.heads_k ? warps(1) : 0};
    if (need[0] + need[1] > most) {
        const long long all = (long long)a.steps[0] + a.steps[1];
        // (either side has a block at least, however few its heads beside the other's)
        need[1] = d.heads_k ? std::min({each, most - 1LL, std::max(1LL, (most * (long long)a.steps[1] + all / 2) / all)}) : 0;
        need[0] = std::min(each, most - need[1]);
    }
    *q_blocks = (int)need[0];
    *blocks = (int)(need[0] + need[1]);
}

template <typename F>
cudaError_t dispatch(const cba_qk_norm_rope_desc_t &d, F f) {
    auto pairs = [&](auto t, auto p) {
        switch (pairs_of(d)) {
            case PAIRS_LOCAL2: return f(t, p, std::integral_constant<int, PAIRS_LOCAL2>{});
            case PAIRS_LANES2: return f(t, p, std::integral_constant<int, PAIRS_LANES2>{});
            case PAIRS_LOCAL: return f(t, p, std::integral_constant<int, PAIRS_LOCAL>{});
            case PAIRS_SPLIT: return f(t, p, std::integral_constant<int, PAIRS_SPLIT>{});
            case PAIRS_LANES: return f(t, p, std::integral_constant<int, PAIRS_LANES>{});
            default: return f(t, p, std::integral_constant<int, PAIRS_ANY>{});
        }
    };
    auto param = [&](auto t) { return d.param_type == CBA_F32 ? pairs(t, 0.f) : pairs(t, t); };
    return d.type == CBA_F32 ? param(0.f) : d.type == CBA_F16 ? param(__half{}) : param(__nv_bfloat16{});
}

template <bool BWD>
cudaError_t launch(const cba_qk_norm_rope_desc_t &d, QkArgs a, int *blocks, cudaStream_t st) {
    plan_blocks(d, a, blocks, &a.q_blocks);
    return dispatch(d, [&](auto t, auto p, auto pairs) {
        using T = decltype(t);
        using P = decltype(p);
        constexpr int PAIRS = decltype(pairs)::value, AHEAD = qk_ahead(BWD);
        constexpr auto alone = qk_kernel<T, P, PAIRS, BWD, false>, shared = qk_kernel<T, P, PAIRS, BWD, true>;
        const bool share = a.parts[0] > 1 || a.parts[1] > 1;
        const int step = (BWD ? 2 : 1) * Lane<PAIRS>::NV * (int)sizeof(T) * 256;
        a.warp_bytes = AHEAD * step + (AHEAD + 1) * a.row_bytes + (PAIRS == PAIRS_ANY ? Lane<PAIRS>::kPlaces * 4 : 0);
        // (backward: the block's sums at the end)
        const int bytes = std::max(kWarps * a.warp_bytes, BWD ? kWarps * 1024 : 0);
        const int most = kWarps * (AHEAD * step + (AHEAD + 1) * kQkMaxDim * 4 + Lane<PAIRS>::kPlaces * 4);
        cudaError_t e = share ? allow_smem<shared>(most) : allow_smem<alone>(most);
        if (e != cudaSuccess) return e;
        (share ? shared : alone)<<<(unsigned)*blocks, kWarps * 32, bytes, st>>>(a);
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
    QkArgs a = base_args(*d, table, pos);
    a.x[0] = q; a.x[1] = k;
    a.gamma[0] = gamma_q; a.gamma[1] = gamma_k;
    a.out[0] = yq; a.out[1] = yk;
    strides_of(*d, d->q, d->heads_q, a.sx[0]);
    strides_of(*d, d->k, d->heads_k, a.sx[1]);
    strides_of(*d, d->yq, d->heads_q, a.so[0]);
    strides_of(*d, d->yk, d->heads_k, a.so[1]);
    cudaGetLastError();
    cudaError_t e = select_device_of(yq);
    int blocks;
    if (e == cudaSuccess) e = launch<false>(*d, a, &blocks, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

size_t cba_qk_norm_rope_workspace_bytes(const cba_qk_norm_rope_desc_t *d) {
    if (check_desc(d) != CBA_OK) return 0;
    int blocks, q_blocks;
    plan_blocks(*d, base_args(*d, nullptr, nullptr), &blocks, &q_blocks);
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
    QkArgs a = base_args(*d, table, pos);
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
    int blocks = 0;
    if (e == cudaSuccess && !d->norm) {
        if (d->len > 0) e = launch<false>(*d, a, &blocks, st);
        return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
    }
    a.partial = static_cast<float *>(workspace);
    if (e == cudaSuccess && d->len > 0) e = launch<true>(*d, a, &blocks, st);
    if (e == cudaSuccess && (dgamma_q || dgamma_k)) {
        const dim3 grid((unsigned)(d->dim + 31) / 32, 2);
        int q_blocks;
        plan_blocks(*d, a, &blocks, &q_blocks);
        if (d->len > 0)
            e = launch_pdl(qk_dgamma_kernel, grid, dim3(1024), 0, st, (const float *)a.partial, d->dim, q_blocks, blocks,
                           dgamma_q, dgamma_k, d->accumulate);
        else
            qk_dgamma_kernel<<<grid, 1024, 0, st>>>(a.partial, d->dim, 0, 0, dgamma_q, dgamma_k, d->accumulate);
        if (e == cudaSuccess) e = cudaGetLastError();
    }
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

}  // extern "C"
