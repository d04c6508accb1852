// cba_attention_fwd.cu -- attention's forward pass: o and the rows' log-sum-exp.
//
//   S = scale q k^T,  m = max_j S_ij over the allowed pairs
//   l = sum_j exp(S_ij - m),  o = sum_j exp(S_ij - m) v_j / l,  lse = m + log l
//
// One pass over the keys, with a running maximum and sum (Milakov and Gimelshein, "Online
// normalizer calculation for softmax", 2018).  A block takes two tiles of 128 query rows and walks
// their keys, 128 at a time: S of a tile by the tensor cores into TMEM, P = exp(S -
// m) by a warpgroup, a thread per row, back into TMEM in 16 bits, o += P v by the tensor
// cores.  While one tile's warpgroup computes P, the tensor cores have the other's
// products.  The running maximum m lags: it is raised, and o and l scaled down, only
// when a row's new one is past it by 2^8, so that most steps leave o alone.  (P is
// then 2^8 at most, in f16 2^15 with its power of two: P does not overflow, nor do f16's sums of P v;
// bf16's do where 2^8 sum |v| is past fp32's range.)
//
// P is rounded to the elements' type, since a product's two operands have one type; l sums it
// unrounded, in fp32.  The error of o against 64 bits, relative to its norm, is then 0.0020 to 0.0023 in bf16 and
// 0.00029 in f16, where an o of fp32 products rounded once has 0.0015 to 0.0017 and 0.00021.
// (P in two parts would double the product with v, half of the tensor cores' work.)
//
// The rows of a tile are the query heads that share a key/value head (or as many of
// them as fill 128 rows) by as many tokens as fit: a single token of eight such
// heads reads its keys once.
//
// Blocks come from the grid in order, heaviest first where the mask makes work fall (packed
// pairs that are numbered by the tokens: in that order); a block that is done takes over the next that has not started (cluster launch
// control), so that its loads and first products run under the last ones of the
// item before.  Where there are fewer pairs of tiles than SMs the keys are cut, each
// item leaves fp32 sums, and a second kernel joins them in the order of the keys.
//
// Measured (us; rates count the products of the pairs that the mask allows):
//   8192 tokens, 32/8 heads of 128, causal, bf16   346 after a pause, 368 in turn with other
//       calls: 1.59 and 1.49 PFLOP/s.  The chain S -> P -> o of the two tiles bounds it: 3300
//       cycles a step of the pair, of which the tensor cores have products for 2048
//   9 documents of 8192 tokens, 16/4 heads of 128  58: 536 items of 3208 steps, 21 steps or 36 us an SM;
//       to begin and end an item costs about 1.5 steps more, and the order by tokens leaves SMs idle at the end
//   32 x 676 tokens, 8 heads of 64, f16            64: the same chain with half the products; tensor
//       cores and exponentials' unit are each active for 29% of the cycles, issue slots taken for 41%
//   8 x 1 tokens over 8192 keys, 32/8 heads of 128 51 to 53: the keys and values at 5.2 TB/s, the
//       second kernel included
//   2 x 169 tokens, 8 heads of 64, bf16            10.2: one launch, two steps
// Tried: four warpgroups with half a row each (420 in the first case: they exchange maxima), both
// warpgroups on each tile (370), S two steps ahead in steps of 64 keys (430: products of 64 columns
// take more than half the time of 128), waits that spin in place of try_wait's own (367).
//
// Roles: warp 0 loads (TMA) and takes items, warp 1 (past dim 64 warps 1 and 2) issues
// the products, warps 4-7 and 8-11 are the two tiles' warpgroups.  Every wait is
// bounded (2 s); on a timeout the block sets the workspace's status bit, stops, waits
// (bounded) for its copies in flight, frees its TMEM and returns.
#include <cuda.h>

#include <algorithm>
#include <cmath>

#include "cba_attn.cuh"
#include "cba_internal.cuh"
#include "cba_ptx.cuh"
#include "cba_types.cuh"

namespace cba {

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kAfThreads = 384;
constexpr int kAfWarps = 8;                    // that compute P
// Registers per thread: 168 at launch, then moved to the two computing warpgroups, which
// hold a row of S.
constexpr int kAfCtlRegs = 72, kAfCompRegs = 216;
static_assert(128 * kAfCtlRegs + 256 * kAfCompRegs <= kAfThreads * 168);
constexpr float kLag = 8.f;                    // log2 by which m may lag behind
constexpr float kLargeLog = 1024.f;            // |m| in log2 from which S - m is formed first
constexpr float kHalfShift = 7.f;              // f16: P is held as 2^7 P

struct AfArgs {
    const int *cu_q, *cu_k;
    int batch, hq, hkv, group, dim, len_q, len_k;
    long long total_q, total_k;
    int causal;
    float cs;          // |scale| / ln 2
    int negative;      // scale < 0
    int hp;            // heads side by side in a tile
    int hparts;        // heads_q / hp
    int tt;            // tokens of a tile
    int pairs;         // of the longest sequence; with slots, all
    int slots;         // packed with loose bounds: pairs are numbered by the tokens
    int heads_at_once; // causal: heads (of all sequences) whose heaviest pairs come first together
    int chunk, chunks; // steps of an item at most; items per pair at most
    int units, items;
    int maps;          // there are queries and keys, and so tensor maps
    void *o;
    float *lse;
    long long so[3];
    unsigned *status;
    float *part;       // fp32 sums of cut items: [unit][chunk][tile][DP / 4][128 rows] float4
    float2 *ml;        // their m (in S's unit) and l: [unit][chunk][tile][128 rows]
};

// One item: the keys from step it0 on of a pair of tiles.
struct AfItem {
    long long q0, k0;    // first tokens of the sequence
    int b, h0, hk;       // head of the tiles' first row, key/value head
    int t0, lq, lk;      // first token of the pair, lengths
    int it0, n, cnt[2];  // steps from it0 on, of the pair and of each tile
    int unit, c, used;   // item c of `used`
    int live;
};
static_assert(sizeof(AfItem) <= 128);

// Sequence b's range of tokens; values of cu are clamped into the tensors, so that
// wrong ones give wrong results but no access out of bounds.
__device__ __forceinline__ void af_seq(const AfArgs &a, AfItem &w) {
    if (a.cu_q == nullptr) {
        w.q0 = w.k0 = 0;
        w.lq = a.len_q, w.lk = a.len_k;
        return;
    }
    const long long qa = min(max((long long)a.cu_q[w.b], 0LL), a.total_q);
    const long long qb = min(max((long long)a.cu_q[w.b + 1], qa), a.total_q);
    const long long ka = min(max((long long)a.cu_k[w.b], 0LL), a.total_k);
    const long long kb = min(max((long long)a.cu_k[w.b + 1], ka), a.total_k);
    w.q0 = qa, w.k0 = ka;
    w.lq = (int)min(qb - qa, (long long)a.len_q);
    w.lk = (int)min(kb - ka, (long long)a.len_k);
}

// Numbering by the tokens: pair t of sequence b has the slot cu[b] / (2 tt) + b + t.
// The next sequence's first slot lies past its last, so there are total / (2 tt) +
// batch at most, of which one per sequence may stand for no pair.
__device__ __forceinline__ int af_slot(const AfArgs &a, int b) {
    return (int)(min(max((long long)a.cu_q[b], 0LL), a.total_q) / (2 * a.tt)) + b;
}

// A whole warp's wait for barriers, each lane's its own: one vote where the phases are
// over.  (Lanes that leave a loop one by one, and a vote after it, cost a product's
// issuer 200 cycles and more; this 15.)
__device__ __forceinline__ bool warp_wait(AtWait w, volatile int *abort, unsigned *status) {
    const uint32_t bar = ptx::smem_u32(w.bar);
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, w.parity & 1u))) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, w.parity & 1u))) return true;
        if ((it & 63u) == 0) {
            const bool late = ptx::globaltimer_ns() - t0 > kAtLimitNs;
            if (__any_sync(0xffffffffu, late || *abort != 0)) {
                if (late) {
                    *abort = 1;
                    atomicOr(status, kStatusTimeout);
                }
                __syncwarp();
                return false;
            }
        }
    }
}

// Item `i` of the grid.  Called by any threads, each for itself.
__device__ __forceinline__ AfItem af_item(const AfArgs &a, int i) {
    AfItem w;
    w.c = i % a.chunks;
    const int u = w.unit = i / a.chunks;
    const int heads = a.slots ? a.hparts : a.hparts * a.batch;
    int head, pair;
    if (a.causal) {  // the pairs with the most keys first, a few heads at a time
        const int block = u / (a.heads_at_once * a.pairs), first = block * a.heads_at_once;
        const int n = min(a.heads_at_once, heads - first), r = u - first * a.pairs;
        head = first + r % n;
        pair = a.pairs - 1 - r / n;
    } else {
        pair = u % a.pairs;
        head = u / a.pairs;
    }
    if (a.slots) {
        int lo = 0, hi = a.batch;  // the last sequence whose slots begin at `pair` or before
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (af_slot(a, mid) <= pair) lo = mid;
            else hi = mid;
        }
        w.b = lo;
        pair -= af_slot(a, lo);
    } else {
        w.b = head / a.hparts;
        head -= w.b * a.hparts;
    }
    w.h0 = head * a.hp;
    w.hk = w.h0 / a.group;
    af_seq(a, w);
    // (a slot before the first sequence's, or past a sequence's last)
    const bool in = pair >= 0 && (long long)pair * 2 * a.tt < w.lq;
    w.t0 = in ? pair * 2 * a.tt : 0;
    int n[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int last = min(w.t0 + (x + 1) * a.tt, w.lq) - 1;  // the tile's last token
        int keys = in && w.t0 + x * a.tt < w.lq ? w.lk : 0;
        if (a.causal) keys = min(keys, max(last + w.lk - w.lq + 1, 0));
        n[x] = (keys + kT - 1) / kT;
    }
    const int all = max(n[0], n[1]);
    w.used = 1, w.it0 = 0, w.n = all;
    if (a.chunks > 1) {
        w.used = max(1, (all + a.chunk - 1) / a.chunk);
        const int each = (all + w.used - 1) / w.used;
        w.it0 = w.c * each;
        w.n = min(each, all - w.it0);
    }
    w.live = in && w.c < w.used;
    if (!w.live) w.n = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) w.cnt[x] = min(max(n[x] - w.it0, 0), w.n);
    return w;
}

template <int DP>
struct Af {
    static constexpr int ST = DP == 64 ? 8 : 4;   // tiles of the ring of keys and values
    // two warps issue the products in turns; up to dim 64, where a step's are few, one warp both tiles'
    static constexpr bool TURNS = DP == 128;
    static constexpr uint32_t TILE = DP / 64 * kBoxBytes;
    static constexpr uint32_t STAGE = kAfWarps * 2048;
    static constexpr uint32_t RING = 2 * TILE, OUT = RING + ST * TILE, BARS = OUT + STAGE;
    struct Bars {
        uint64_t q_full[2], q_empty[2];
        uint64_t kv_full[ST], kv_empty[ST];
        uint64_t s_full[2], p_ready[4], acc[2];  // (P in halves)
        uint64_t i_full[2], i_empty[2];
        uint64_t fix, clc, drain[2], turn[2];
        uint32_t tmem_base;
        int abort_flag;
    };
    // and the items, and the answer of the launch control
    static constexpr uint32_t ITEMS = (BARS + sizeof(Bars) + 15) / 16 * 16, CLC = ITEMS + 2 * 128, SMEM = CLC + 16;
};

template <int DP, bool BF16>
__global__ void __launch_bounds__(kAfThreads, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const AfArgs a) {
    using A = Af<DP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    constexpr uint32_t TILE = A::TILE;
    constexpr int ST = A::ST;
    const uint32_t sbase = ptx::smem_u32(smem), sQ = sbase, sKV = sbase + A::RING;
    auto &sb = *reinterpret_cast<typename A::Bars *>(smem + A::BARS);
    AfItem *slots = reinterpret_cast<AfItem *>(smem + A::ITEMS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && tid == 0) *a.status = 0;  // (a timeout takes two seconds more)
    if (sbase & 1023) {  // the swizzled tiles need it
        if (tid == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    if (tid == 0) {
        at_init_bars(sb.q_full, 4, 1);
        at_init_bars(sb.kv_full, ST, 1);
        at_init_bars(sb.kv_empty, ST, A::TURNS ? 2 : 1);
        at_init_bars(sb.s_full, 2, 1);
        at_init_bars(sb.p_ready, 4, kAfWarps / 2);
        at_init_bars(sb.acc, 2, 1);
        at_init_bars(sb.i_full, 2, 1);
        at_init_bars(sb.i_empty, 2, (A::TURNS ? 2 : 1) + kAfWarps);
        at_init_bars(&sb.fix, 6, 1);
        sb.abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0) {
        // the loads begin while TMEM is allocated
        if (lane == 0 && a.maps) {
            ptx::prefetch_map(&tq);
            ptx::prefetch_map(&tk);
            ptx::prefetch_map(&tv);
        }
        __syncwarp();
        ptx::named_bar_arrive(1, kAfThreads);
    } else {
        if (warp == 1) {
            ptx::tmem_alloc(ptx::smem_u32(&sb.tmem_base), 512);
            ptx::tmem_relinquish();
        }
        ptx::tc_fence_before();
        ptx::named_bar_sync(1, kAfThreads);
        ptx::tc_fence_after();
    }
    ptx::griddep_launch_dependents();
    const uint32_t tmem = warp == 0 ? 0 : *const_cast<volatile uint32_t *>(&sb.tmem_base);
    // S of the two tiles (P over its first half), then o of the two
    const uint32_t tS = tmem, tO = tmem + 256;
    volatile int *ab = &sb.abort_flag;
    const bool packed = a.cu_q != nullptr;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return ok = ok && warp_wait(AtWait{bar, parity}, ab, a.status);
    };
    // the k-th item handed out, NULL past the last (or on a timeout)
    auto take = [&](int k) -> const AfItem * {
        return wait(&sb.i_full[k & 1], (uint32_t)(k / 2)) && slots[k & 1].live ? slots + (k & 1) : nullptr;
    };
    auto done = [&](int k) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.i_empty[k & 1]));
    };

    // Products: a whole warp walks its loop and one elected lane issues.  Loops and conditions go by
    // votes, and which tile it is by a constant: descriptors and counters known to be uniform take
    // half the time to issue a product.
    // (a negative scale negates q in the product, so that S's largest is the exponent's)
    const uint32_t id_s = ptx::idesc_f16(128, 128, BF16, false) | (a.negative ? ptx::kNegateA : 0u);
    const int steps = (a.dim + 15) / 16;
    const uint32_t id_o = ptx::idesc_f16(128, steps * 16, BF16, true);
    auto some = [&](bool p) { return __any_sync(0xffffffffu, p) != 0; };
    // (of an elected lane) S of tile x with the keys in stage st; o += a half of P times the values
    auto issue_s = [&](int x, int st) {
        const ptx::Desc dq = ptx::desc_of(sQ + x * TILE, 16, 1024, 2), dk = ptx::desc_of(sKV + st * TILE, 16, 1024, 2);
        auto step = [&](int ks) {
            const uint32_t off = ((ks >> 2) * kBoxBytes + (ks & 3) * 32) >> 4;
            ptx::mma_f16(tS + x * kT, dq, off, dk, off, id_s, ks > 0);
        };
        if (steps == DP / 16) {  // a condition in each step doubles its issue time
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) step(ks);
        } else {
            for (int ks = 0; ks < steps; ++ks) step(ks);
        }
    };
    auto issue_o = [&](int x, int st, int half, bool first) {
        const ptx::Desc dv = ptx::desc_of(sKV + st * TILE + half * (64 * 128), kBoxBytes, 1024, 2);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            ptx::mma_f16_ts(tO + x * DP, tS + x * kT + half * 32 + ks * 8, dv, ks * (2048 >> 4), id_o, !first || ks > 0);
    };
    // the end: every product issued has finished before TMEM is released
    auto finish = [&](int x) {
        if (ptx::elect_one()) {
            if (!ok) *const_cast<volatile int *>(&sb.abort_flag) = 1;
            ptx::mma_commit(ptx::smem_u32(&sb.drain[x]));
        }
        __syncwarp();
        int no = 0;
        ptx::mbar_wait_bounded(ptx::smem_u32(&sb.drain[x]), 0, &no, a.status, kAtLimitNs);
        __syncwarp();
    };

    if (warp < 4) {
        ptx::regs_dec<kAfCtlRegs>();
        if (warp == 0) {
            uint32_t fphase = 0;
            const uint32_t bfix = ptx::smem_u32(&sb.fix), bclc = ptx::smem_u32(&sb.clc), answer = sbase + A::CLC;
            int kv = 0, nq[2] = {0, 0}, asked = 0, k = 0;
            auto hand_out = [&](const AfItem &w) {
                if (k >= 2 && !wait(&sb.i_empty[k & 1], (uint32_t)(k / 2 - 1))) return;
                if (lane == 0) {
                    slots[k & 1] = w;
                    ptx::mbar_arrive(ptx::smem_u32(&sb.i_full[k & 1]));
                }
                __syncwarp();
                ++k;
            };
            auto load_kv = [&](const CUtensorMap *tm, const AfItem &w, int key, bool fix) {
                const int st = kv % ST;
                if (kv >= ST && !wait(&sb.kv_empty[st], (uint32_t)(kv / ST - 1))) return;
                ++kv;
                ok = load_tile<DP>(sKV + st * TILE, tm, w.k0 + key, w.hk, packed ? 0 : w.b, fix ? w.lk - key : kT, packed,
                                   ptx::smem_u32(&sb.kv_full[st]), bfix, fphase, ab, a.status);
            };
            for (int i = (int)blockIdx.x; ok && i >= 0;) {
                const AfItem w = af_item(a, i);
                if (w.live) {
                    hand_out(w);
                    for (int x = 0; ok && x < 2; ++x) {
                        if (w.cnt[x] == 0) continue;
                        if (nq[x] > 0 && !wait(&sb.q_empty[x], (uint32_t)(nq[x] - 1))) break;
                        ++nq[x];
                        if (lane == 0) {
                            const uint32_t bar = ptx::smem_u32(&sb.q_full[x]);
                            ptx::mbar_arrive_expect_tx(bar, DP / 64 * a.hp * a.tt * 128);
#pragma unroll
                            for (int j = 0; j < DP / 64; ++j)
                                ptx::tma_load_4d(sQ + x * TILE + j * kBoxBytes, &tq, j * 64, w.h0, (int)(w.q0 + w.t0 + x * a.tt),
                                                 packed ? 0 : w.b, bar);
                        }
                        __syncwarp();
                        // the second tile is not needed before the first's keys
                        if (x == 0) load_kv(&tk, w, w.it0 * kT, false);
                    }
                    if (w.cnt[0] == 0 && w.n > 0) load_kv(&tk, w, w.it0 * kT, false);
                    for (int it = 0; ok && it < w.n; ++it) {
                        const int key = (w.it0 + it) * kT;
                        if (it > 0) load_kv(&tk, w, key, false);
                        // (rows past the sequence: of k masked, of v multiplied by P = 0)
                        if (ok) load_kv(&tv, w, key, true);
                    }
                }
                if (!ok) break;
                // the next item, once this one's loads have begun: earlier, and the items
                // would be dealt out before it is known who is done first
                if (lane == 0) {
                    ptx::fence_proxy_async_smem();
                    ptx::mbar_arrive_expect_tx(bclc, 16);
                    ptx::try_cancel_block(answer, bclc);
                }
                __syncwarp();
                if (!wait(&sb.clc, (uint32_t)asked++)) break;
                i = ptx::cancelled_block(answer);
                __syncwarp();
            }
            if (ok) {
                AfItem end{};
                hand_out(end);
            }
            if (!ok) {
                drain_ring(sb.q_full, 1, nq[0], a.status);
                drain_ring(sb.q_full + 1, 1, nq[1], a.status);
                drain_ring(sb.kv_full, ST, kv, a.status);
                drain_ring(&sb.clc, 1, asked, a.status);
            }
        } else if (!A::TURNS && warp == 1) {
            // The products of both tiles, in the order of their steps.  (32 x 676 tokens, 8 heads of 64: 64 us, in
            // turns 70.)
            Ring rk, rv;             // the ring's stage of the next keys, of the next values
            rv.step(ST);
            int gq[2] = {0, 0}, gp[2] = {0, 0};  // queries, P so far
            auto two = [&](Ring &r) { r.step(ST), r.step(ST); };
            auto full = [&](Ring r) { return AtWait{&sb.kv_full[r.s], r.ph}; };
            auto both = [&](AtWait u, AtWait v) { return ok = ok && warp_wait(lane & 1 ? v : u, ab, a.status); };
            // S of tile x with the keys at rk; `free`: their last use; `last`: the queries' too
            auto mma_s = [&](int x, bool free, bool last) {
                if (ptx::elect_one()) {
                    issue_s(x, rk.s);
                    ptx::mma_commit(ptx::smem_u32(&sb.s_full[x]));
                    if (free) ptx::mma_commit(ptx::smem_u32(&sb.kv_empty[rk.s]));
                    if (last) ptx::mma_commit(ptx::smem_u32(&sb.q_empty[x]));
                }
                __syncwarp();
            };
            auto mma_o = [&](int x, int half, bool first, bool free, bool last) {
                if (ptx::elect_one()) {
                    issue_o(x, rv.s, half, first);
                    if (free) ptx::mma_commit(ptx::smem_u32(&sb.kv_empty[rv.s]));
                    if (last) ptx::mma_commit(ptx::smem_u32(&sb.acc[x]));
                }
                __syncwarp();
            };
            const AfItem *w;
            for (int k = 0; (w = take(k)) != nullptr; ++k) {
                const int n = w->n, cnt[2] = {w->cnt[0], w->cnt[1]};
                done(k);
                // a step's last user of its keys and values is the second tile, if it has the step
                auto frees = [&](int x, int it) { return x == 1 || some(it >= cnt[1]); };
                if (!some(n > 0)) continue;
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (some(cnt[x] > 0)) {
                        if (!both({&sb.q_full[x], (uint32_t)gq[x]++}, full(rk))) break;
                        ptx::tc_fence_after();
                        mma_s(x, frees(x, 0), some(cnt[x] == 1));
                    }
                two(rk);
                for (int it = 0; ok && some(it < n); ++it) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (!some(it < cnt[x])) continue;
                        const bool more = some(it + 1 < cnt[x]);
                        // P's first half, the values, and the keys of the next S
                        if (!both({&sb.p_ready[2 * x], (uint32_t)gp[x]}, lane & 2 && more ? full(rk) : full(rv))) break;
                        ptx::tc_fence_after();
                        mma_o(x, 0, it == 0, false, false);
                        const AtWait second{&sb.p_ready[2 * x + 1], (uint32_t)gp[x]++};
                        if (!both(second, second)) break;
                        ptx::tc_fence_after();
                        mma_o(x, 1, false, frees(x, it), !more);
                        // S overwrites P: this warp's products run in the order of issue
                        if (more) mma_s(x, frees(x, it + 1), some(it + 2 == cnt[x]));
                    }
                    two(rv);
                    if (some(it + 1 < n)) two(rk);
                }
                if (!ok) break;
            }
            finish(0);
        } else if (A::TURNS && warp > 0 && warp < 3) {
            // The products of tile x, by a warp for each.  They take turns, of a step's products: products
            // that alternate between accumulators run at half the rate, and the waits of one hide
            // behind the other's turn.  (8192 tokens, 32/8 heads of 128: 353 us, with one warp for both
            // tiles 370.)
            auto products = [&](auto tile) {
            constexpr int x = decltype(tile)::value;
            Ring r;                  // the next tile of keys or values
            int gq = 0, gp = 0, turns = 0;  // queries, P, turns so far
            auto both = [&](AtWait u, AtWait v) { return ok = ok && warp_wait(lane & 1 ? v : u, ab, a.status); };
            auto full = [&]() { return AtWait{&sb.kv_full[r.s], r.ph}; };
            bool shared = false;  // both tiles have steps in this item
            auto my_turn = [&]() {
                if (!shared) return ok;
                const int j = turns++ - (1 - x);  // the other's pass that this one waits for
                return j < 0 || wait(&sb.turn[x], (uint32_t)j);
            };
            const uint32_t pass = ptx::smem_u32(&sb.turn[1 - x]);
            auto pass_on = [&]() {
                if (shared && lane == 0) ptx::mbar_arrive(pass);
                __syncwarp();
            };
            // S, the end of a turn
            auto mma_s = [&](bool last) {
                if (ptx::elect_one()) {
                    issue_s(x, r.s);
                    // (any earlier, and the other's products come between: S is late)
                    if (shared) ptx::mbar_arrive(pass);
                    ptx::mma_commit(ptx::smem_u32(&sb.s_full[x]));
                    ptx::mma_commit(ptx::smem_u32(&sb.kv_empty[r.s]));
                    if (last) ptx::mma_commit(ptx::smem_u32(&sb.q_empty[x]));
                }
                __syncwarp();
                r.step(ST);
            };
            auto mma_o = [&](int half, bool first) {
                if (ptx::elect_one()) {
                    issue_o(x, r.s, half, first);
                }
                __syncwarp();
            };
            const AfItem *w;
            for (int k = 0; (w = take(k)) != nullptr; ++k) {
                const int n = w->n, cnt = w->cnt[x], others = w->cnt[1 - x];
                done(k);
                if (!some(n > 0)) continue;
                const bool any = some(cnt > 0);
                shared = any && some(others > 0);
                if (any && !both({&sb.q_full[x], (uint32_t)gq++}, full())) break;
                if (!my_turn()) break;
                ptx::tc_fence_after();
                if (any) mma_s(some(cnt == 1));
                else pass_on();
                for (int it = 0; ok && some(it < cnt); ++it) {
                    // S overwrites P: this warp's products run in the order of issue
                    const bool more = some(it + 1 < cnt);
                    Ring next = r;
                    next.step(ST);
                    const AtWait p0{&sb.p_ready[2 * x], (uint32_t)gp}, p1{&sb.p_ready[2 * x + 1], (uint32_t)gp};
                    ++gp;
                    if (!both(p0, lane & 2 && more ? AtWait{&sb.kv_full[next.s], next.ph} : full())) break;
                    if (!my_turn()) break;
                    ptx::tc_fence_after();
                    mma_o(0, it == 0);
                    if (!both(p1, p1)) break;
                    ptx::tc_fence_after();
                    mma_o(1, false);
                    if (ptx::elect_one()) {
                        ptx::mma_commit(ptx::smem_u32(&sb.kv_empty[r.s]));
                        if (!more) ptx::mma_commit(ptx::smem_u32(&sb.acc[x]));
                    }
                    __syncwarp();
                    r.step(ST);
                    if (more) mma_s(some(it + 2 == cnt));
                    else pass_on();
                }
                // the other tile's steps alone: turns, keys and values that this one lets pass
                for (int it = cnt; ok && some(it < n); ++it) {
                    if (!my_turn()) break;
                    pass_on();
                    for (int j = 0; j < 2; ++j) {
                        if (!both(full(), full())) break;
                        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.kv_empty[r.s]));
                        __syncwarp();
                        r.step(ST);
                    }
                }
                if (!ok) break;
            }
            finish(x);
            };
            if (warp == 1) products(std::integral_constant<int, 0>{});
            else products(std::integral_constant<int, 1>{});
        }
    } else {
        ptx::regs_inc<kAfCompRegs>();
        const int x = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tS + x * kT + lanes, to = tO + x * DP + lanes;
        constexpr float shift = BF16 ? 0.f : kHalfShift;
        const float cs = a.cs;
        const float2 cs2 = make_float2(cs, cs);
        // this thread's row: token and head in its tile
        const int tok = r / a.hp, hd = r - tok * a.hp;
        uint8_t *stage = smem + A::OUT + (warp - 4) * 2048;
        int gs = 0, ga = 0;
        const AfItem *wp;
        for (int k = 0; (wp = take(k)) != nullptr; ++k) {
            const volatile AfItem &w = *wp;  // read where it is used: the registers hold a row of S
            const int cnt = w.cnt[x];
            // counted from the item's first step: the row sees the keys before `sees`; steps
            // that end by `all` need no mask
            int sees, all;
            {
                const int it0 = w.it0 * kT, first = w.t0 + x * a.tt, diag = w.lk - w.lq + 1 - it0;
                sees = all = w.lk - it0;
                if (a.causal) sees = min(sees, first + tok + diag), all = min(all, first + diag);
            }
            const int t = w.t0 + x * a.tt + tok;
            const bool row = tok < a.tt && t < w.lq;
            float m = -INFINITY;  // in S's unit
            float2 l0 = make_float2(0.f, 0.f), l1 = l0;
            for (int it = 0; it < cnt; ++it) {
                if (!wait(&sb.s_full[x], (uint32_t)gs)) break;
                ++gs;
                ptx::tc_fence_after();
                if (__builtin_expect(it * kT + kT > all, 0)) {  // -infinity over the masked columns of S
                    const int lim = sees - it * kT;
#pragma unroll 1
                    for (int c = max(all - it * kT, 0) & ~15; c < kT; c += 16) {
                        float v[16];
                        uint32_t u[16];
                        ptx::tmem_ld16(ts + c, v);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            asm volatile("" : "+f"(v[e]));
                            u[e] = __float_as_uint(c + e >= lim ? -INFINITY : v[e]);
                        }
                        ptx::tmem_st16(ts + c, u);
                    }
                    ptx::tmem_st_wait();
                }
                float s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) ptx::tmem_ld32(ts + c * 32, s[c]);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < kT; ++c) asm volatile("" : "+f"(s[c >> 5][c & 31]));  // used behind the wait
                float now = -INFINITY;
                {
                    float top[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        constexpr int Q = kT / 4;
                        auto at = [&](int e) { return s[(c * Q + e) >> 5][(c * Q + e) & 31]; };
                        top[c] = fmaxf(at(0), at(Q - 1));
#pragma unroll
                        for (int e = 1; e < Q - 1; e += 2) top[c] = ptx::max3(top[c], at(e), at(e + 1));
                    }
                    now = fmaxf(ptx::max3(top[0], top[1], top[2]), top[3]);
                }
                auto hand_over = [&](int h) {
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sb.p_ready[2 * x + h]));
                };
                // no row: whatever lies there (the next sequence's queries) raises nothing and has no vote
                if (!row) now = -INFINITY;
                // One vote for what is rare.  (-inf - -inf and inf - inf are NaN, which raises nothing.)
                const bool grown = (now - m) * cs > kLag, large = fabsf(fmaxf(m, now)) * cs > kLargeLog && now > -INFINITY;
                if (__builtin_expect(__any_sync(0xffffffffu, grown || large), 0)) {
                    if (__any_sync(0xffffffffu, grown)) {
                        const float up = fmaxf(m, now);
                        const float f = up == -INFINITY ? 1.f : ptx::ex2((m - up) * cs);
                        m = up;
                        l0 = ptx::mul2(l0, make_float2(f, f));
                        l1 = ptx::mul2(l1, make_float2(f, f));
                        // (the product before S has finished with o; the first one overwrites it)
#pragma unroll 1
                        for (int c = it > 0 ? 0 : DP; c < DP; c += 16) {
                            float v[16];
                            uint32_t u[16];
                            ptx::tmem_ld16(to + c, v);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                asm volatile("" : "+f"(v[e]));
                                u[e] = __float_as_uint(v[e] * f);
                            }
                            ptx::tmem_st16(to + c, u);
                        }
                    }
                    // S cs - m cs in one rounding is off by 2^-24 of m cs: where that is large, S - m comes first
                    if (__any_sync(0xffffffffu, fabsf(m) * cs > kLargeLog && m > -INFINITY)) {
                        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 1
                        for (int c = 0; c < kT; c += 16) {
                            float v[16];
                            uint32_t p[8];
                            ptx::tmem_ld16(ts + c, v);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                asm volatile("" : "+f"(v[2 * e]), "+f"(v[2 * e + 1]));
                                const float2 u = make_float2(ptx::ex2(fmaf(v[2 * e] - ref, cs, shift)),
                                                             ptx::ex2(fmaf(v[2 * e + 1] - ref, cs, shift)));
                                l0 = ptx::add2(l0, u);
                                p[e] = pack2<BF16>(u.x, u.y);
                            }
                            ptx::tmem_st8(ts + c / 2, p);  // (over columns that have been read)
                        }
                        hand_over(0), hand_over(1);
                        continue;
                    }
                }
                const float nm = shift - (m == -INFINITY ? 0.f : m) * cs;
                const float2 nm2 = make_float2(nm, nm);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 v = ptx::fma2(make_float2(s[c][2 * e], s[c][2 * e + 1]), cs2, nm2);
                        v = make_float2(ptx::ex2(v.x), ptx::ex2(v.y));
                        if (e & 1) l1 = ptx::add2(l1, v);
                        else l0 = ptx::add2(l0, v);
                        p[e] = pack2<BF16>(v.x, v.y);
                    }
                    if (c == 2) hand_over(0);  // the first half's stores have had the time of 32 columns
                    ptx::tmem_st16(ts + c * 16, p);
                }
                hand_over(1);
            }
            if (!ok || (cnt > 0 && !wait(&sb.acc[x], (uint32_t)ga))) break;
            if (cnt > 0) ++ga;
            ptx::tc_fence_after();
            const float l = (l0.x + l0.y) + (l1.x + l1.y);
            const bool none = l == 0.f;  // no key, or all of them at -infinity
            if (w.used > 1) {
                const long long slot = ((long long)w.unit * a.chunks + w.c) * 2 + x;
                a.ml[slot * kT + r] = make_float2(m, l);
                if (cnt > 0) {
                    float4 *at = reinterpret_cast<float4 *>(a.part) + slot * (DP / 4) * kT + r;
#pragma unroll 1
                    for (int c = 0; c < DP; c += 32) {
                        float v[32];
                        ptx::tmem_ld32(to + c, v);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) asm volatile("" : "+f"(v[e]));
                        if (row)
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                __stcg(at + (c + e) / 4 * kT, make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
                        __syncwarp();
                    }
                }
                ptx::tc_fence_before();
                done(k);
                continue;
            }
            if (row && a.lse)
                a.lse[packed ? (long long)(w.h0 + hd) * a.total_q + w.q0 + t
                             : ((long long)w.b * a.hq + w.h0 + hd) * a.len_q + t] =
                    none ? -INFINITY : fmaf(m, cs, __log2f(l) - shift) * kLn2;
            // 32 columns at a time through 2 KB of the warp's own (row = lane, its 16-byte chunk j
            // at j ^ ((row >> 1) & 3)); then four lanes store a row's 64 bytes
            const float inv = none ? 0.f : 1.f / l;
            uint16_t *out = static_cast<uint16_t *>(a.o) + w.b * a.so[0];
            long long at[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rr = quarter * 32 + i * 8 + (lane >> 2), tk2 = rr / a.hp, tt = w.t0 + x * a.tt + tk2;
                at[i] = tk2 < a.tt && tt < w.lq ? (w.q0 + tt) * a.so[1] + (w.h0 + rr - tk2 * a.hp) * a.so[2] : -1;
            }
#pragma unroll 1
            for (int c = 0; c < DP; c += 32) {
                float v[32];
                if (cnt > 0) {
                    ptx::tmem_ld32(to + c, v);
                    ptx::tmem_ld_wait();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    asm volatile("" : "+f"(v[e]));
                    v[e] = none ? 0.f : v[e] * inv;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 u;
                    u.x = pack2<BF16>(v[8 * j], v[8 * j + 1]);
                    u.y = pack2<BF16>(v[8 * j + 2], v[8 * j + 3]);
                    u.z = pack2<BF16>(v[8 * j + 4], v[8 * j + 5]);
                    u.w = pack2<BF16>(v[8 * j + 6], v[8 * j + 7]);
                    *reinterpret_cast<uint4 *>(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = u;
                }
                __syncwarp();
                const int j = lane & 3;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rr = i * 8 + (lane >> 2);
                    if (at[i] >= 0 && c + j * 8 < a.dim)
                        *reinterpret_cast<uint4 *>(out + at[i] + c + j * 8) =
                            *reinterpret_cast<const uint4 *>(stage + rr * 64 + ((j ^ ((rr >> 1) & 3)) << 4));
                }
                __syncwarp();
            }
            ptx::tc_fence_before();
            done(k);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Joins the items of a tile that was cut: weights exp(m_i - max m), in the items' order.
// Blocks (., y) per tile, a thread per row and 8 columns.
template <bool BF16>
__global__ void __launch_bounds__(256) attn_fwd_join_kernel(const AfArgs a, int dp) {
    const int unit = blockIdx.x >> 1, x = blockIdx.x & 1;
    AfItem w = af_item(a, unit * a.chunks);
    ptx::griddep_wait();
    if (!w.live || w.used == 1) return;
    constexpr float shift = BF16 ? 0.f : kHalfShift;
    const int first = w.t0 + x * a.tt, rows = max(0, min(a.tt, w.lq - first)) * a.hp, cols = a.dim / 8;
    for (int i = blockIdx.y * 256 + threadIdx.x; i < rows * cols; i += gridDim.y * 256) {
        const int r = i % rows, c = i / rows;
        float m = -INFINITY;
        const long long slot0 = (long long)unit * a.chunks * 2 + x;
        // (four items at a time, the last one again for those that are not there: loads in flight together)
        auto at = [&](int j) { return slot0 + 2 * min(j, w.used - 1); };
        for (int j0 = 0; j0 < w.used; j0 += 4)
#pragma unroll
            for (int u = 0; u < 4; ++u) m = fmaxf(m, __ldcg(a.ml + at(j0 + u) * kT + r).x);
        float l = 0.f, v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
        for (int j0 = 0; j0 < w.used; j0 += 4) {
            float2 ml[4];
            float4 y[4], z[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 *from = reinterpret_cast<const float4 *>(a.part) + (at(j0 + u) * (dp / 4) + 2 * c) * kT + r;
                ml[u] = __ldcg(a.ml + at(j0 + u) * kT + r);
                y[u] = __ldcg(from), z[u] = __ldcg(from + kT);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                // (without keys l is 0, and the sums may not have been written)
                if (j0 + u >= w.used || ml[u].y == 0.f) continue;
                const float f = ptx::ex2((ml[u].x - m) * a.cs);
                l = fmaf(f, ml[u].y, l);
                v[0] = fmaf(f, y[u].x, v[0]), v[1] = fmaf(f, y[u].y, v[1]), v[2] = fmaf(f, y[u].z, v[2]);
                v[3] = fmaf(f, y[u].w, v[3]), v[4] = fmaf(f, z[u].x, v[4]), v[5] = fmaf(f, z[u].y, v[5]);
                v[6] = fmaf(f, z[u].z, v[6]), v[7] = fmaf(f, z[u].w, v[7]);
            }
        }
        const bool none = l == 0.f;
        const float inv = none ? 0.f : 1.f / l;
        const int tok = r / a.hp, h = w.h0 + r - tok * a.hp;
        const long long t = first + tok;
        uint4 u;
        u.x = pack2<BF16>(v[0] * inv, v[1] * inv);
        u.y = pack2<BF16>(v[2] * inv, v[3] * inv);
        u.z = pack2<BF16>(v[4] * inv, v[5] * inv);
        u.w = pack2<BF16>(v[6] * inv, v[7] * inv);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o) + w.b * a.so[0] + (w.q0 + t) * a.so[1] + h * a.so[2] + c * 8) = u;
        if (c == 0 && a.lse)
            a.lse[a.cu_q ? (long long)h * a.total_q + w.q0 + t : ((long long)w.b * a.hq + h) * a.len_q + t] =
                none ? -INFINITY : fmaf(m, a.cs, __log2f(l) - shift) * kLn2;
    }
}

// ---- host side

int check_desc(const cba_attention_desc_t *d) {
    if (!d || d->batch < 1 || d->heads_q < 1 || d->heads_kv < 1 || d->dim < 1 || d->len_q < 0 || d->len_k < 0 ||
        d->heads_q % d->heads_kv != 0)
        return CBA_ERR_ARG;
    if (!dtype_ok(d->type) || (d->causal != 0 && d->causal != 1) || (d->packed != 0 && d->packed != 1) ||
        !std::isfinite(d->scale))
        return CBA_ERR_ARG;
    if (d->packed && (d->total_q < 0 || d->total_k < 0)) return CBA_ERR_ARG;
    if (d->type == CBA_F32 || d->dim > 128 || d->dim % 8 != 0) return CBA_ERR_UNSUPPORTED;
    const long long lim = 1LL << 30;
    if (d->len_q > lim || d->len_k > lim || (d->packed && (d->total_q > lim || d->total_k > lim)))
        return CBA_ERR_UNSUPPORTED;
    const cba_attn_strides_t *ss[] = {&d->q, &d->o, &d->k, &d->v};
    for (int i = 0; i < 4; ++i) {
        const long long v[] = {ss[i]->batch, ss[i]->token, ss[i]->head};
        if (!v[0] && !v[1] && !v[2]) continue;  // contiguous
        const bool kside = i >= 2;
        const long long n[] = {d->packed ? 1 : d->batch,
                               d->packed ? (kside ? d->total_k : d->total_q) : (kside ? d->len_k : d->len_q),
                               kside ? d->heads_kv : d->heads_q};
        for (int j = 0; j < 3; ++j) {
            if (v[j] < 0 || (n[j] > 1 && v[j] < d->dim)) return CBA_ERR_ARG;
            if (v[j] % 8 != 0) return CBA_ERR_ALIGN;
            if (v[j] >= (1LL << 38)) return CBA_ERR_UNSUPPORTED;
        }
    }
    return CBA_OK;
}

// Packed: pairs are counted by the tokens where counting up to the bounds would look at
// more than this many times as many.  (64 documents of 700 to 1024 tokens, 32 heads of 128,
// causal: with bounds of all tokens 650 us by the tokens and 3170 up to the bounds; with tight
// ones 650 and 600, since then a head's longest pairs come first.)
constexpr long long kLoose = 2;

struct AfPlan {
    int dp, hp, hparts, tt, pairs, slots, heads_at_once, chunk, chunks, units;
    size_t off_ml, off_part, total;
};

// The heads side by side in a tile: the most of a group that leave no more than 8 of its
// 128 rows empty.  (32/8 heads of 128, single tokens over 8 x 8192 keys: 56 us, with one head
// a tile 163; 2 x 4096 tokens, 28/4 heads, causal, where the keys are read often anyway: 191, 198.)
int heads_in_tile(int group) {
    for (int d = std::min(group, kT); d > 1; --d)
        if (group % d == 0 && kT / d * d >= kT - 8) return d;
    return 1;
}

// Steps of an item at most, for `units` pairs of `n` steps, `all` of them together, that are
// equally long (even) or of any lengths up to that.  In steps of 1.7 us: a begun item is taken to
// cost 1.5, its fp32 sums 1.7 times `part` (1: 256 rows of 128 elements) to be written and 0.0155 times
// `part` to be read by all SMs, the second kernel 3; items of any lengths keep the SMs even but for half an
// item, uncut ones, of which the heaviest come first, but for nothing.  (32/8 heads of 128: single tokens over
// 8 x 8192 keys 51 us, not cut 86, over 65536 keys 52 and 634; causal, 2 x 1634 tokens, 2/1 heads 17
// and 25; 1 x 4096, 16/4 heads, not cut 54, cut by 8 94.)
int plan_chunk(double units, int n, double all, bool even, double part) {
    int best = n;
    double least = 0;
    for (int k = 1; k <= std::min(64, (n + 2) / 3); ++k) {
        const int c = (n + k - 1) / k;
        const double items = even || k == 1 ? units * k : std::min(units * k, all / c + 0.5 * units);
        const double rounds = std::ceil(items / kNumSMs);
        double t = even ? rounds * c : std::max(all / kNumSMs + (k > 1 ? 0.5 * c : 0), (double)c);
        t += 1.5 * rounds;
        if (k > 1) t += 1.7 * part * rounds + 3 + 0.1 * k + 0.0155 * part * items;
        if (k == 1 || t < least) best = c, least = t;
    }
    return best;
}

int check_attn(const cba_attention_desc_t *d, AfPlan *p) {
    const int rc = check_desc(d);
    if (rc != CBA_OK) return rc;
    p->dp = d->dim <= 64 ? 64 : 128;
    p->hp = heads_in_tile(d->heads_q / d->heads_kv);
    p->hparts = d->heads_q / p->hp;
    p->tt = kT / p->hp;
    const long long len_q = d->packed ? std::min((long long)d->len_q, d->total_q) : d->len_q;
    const long long len_k = d->packed ? std::min((long long)d->len_k, d->total_k) : d->len_k;
    const long long two = 2 * p->tt;
    long long pairs = (len_q + two - 1) / two;
    p->slots = 0;
    if (d->packed) {
        const long long by_tokens = d->total_q / two + d->batch;
        if (pairs * d->batch > kLoose * by_tokens) p->slots = 1, pairs = by_tokens;
    }
    const double all_units = (double)pairs * (p->slots ? 1 : d->batch) * p->hparts;
    if (all_units >= (double)(1LL << 30)) return CBA_ERR_UNSUPPORTED;
    const long long units = (long long)all_units;
    p->pairs = (int)pairs;
    p->units = (int)units;
    // Keys and values of the heads that are worked on together stay in the L2.  (Causal: 8 x 8192 tokens,
    // 32/8 heads of 128: 2770 us, all heads together 2920; 64 documents of 700 to 1024 tokens, 32 heads: 600,
    // all 677, with 4 together, whose light ends leave SMs idle, 750.)
    const double bytes = 4.0 * std::max(1LL, len_k) * d->dim;
    p->heads_at_once = (int)std::min((double)p->hparts * (p->slots ? 1 : d->batch), std::max(16.0, 48e6 / bytes));
    p->chunk = std::max(1, (int)((len_k + kT - 1) / kT));
    p->chunks = 1;
    if (units > 0 && units < 2 * kNumSMs && p->chunk > 4) {
        const int n = p->chunk;
        const bool even = !d->packed && (!d->causal || len_q <= two);
        // the share of the pairs that a causal mask leaves
        const double seen = !d->causal || even ? 1 : len_q <= len_k ? 1 - 0.5 * len_q / len_k : 0.5 * len_k / len_q;
        const double part = (double)std::min(len_q, two) / two * p->dp / 128;
        p->chunk = plan_chunk((double)units, n, seen * units * n, even, part);
        p->chunks = (n + p->chunk - 1) / p->chunk;
    }
    const size_t tiles = p->chunks > 1 ? (size_t)p->units * p->chunks * 2 : 0;
    p->off_ml = 256;
    p->off_part = p->off_ml + tiles * kT * sizeof(float2);
    p->total = p->off_part + tiles * kT * p->dp * sizeof(float);
    return CBA_OK;
}

// The map of k or v: (dim, token, head, batch), boxes of a step's keys x 64; of q: (dim, head,
// token, batch), boxes of a tile's tokens x heads x 64.
bool af_map(CUtensorMap *m, const void *base, const cba_attention_desc_t &d, int heads, long long tokens, const long long *st,
            const AfPlan &p, bool is_q) {
    uint64_t dims[4] = {(uint64_t)d.dim, (uint64_t)tokens, (uint64_t)heads, (uint64_t)(d.packed ? 1 : d.batch)};
    uint64_t strides[3] = {(uint64_t)st[1] * 2, (uint64_t)st[2] * 2, (uint64_t)st[0] * 2};
    uint32_t box[4] = {64, (uint32_t)kT, 1, 1};
    if (is_q) {
        std::swap(dims[1], dims[2]);
        std::swap(strides[0], strides[1]);
        box[1] = (uint32_t)p.hp;
        box[2] = (uint32_t)p.tt;
    }
    for (int i = 0; i < 3; ++i)  // an axis of one index has no stride of its own
        if (dims[i + 1] == 1) strides[i] = 16;
    return tma_encode_16(m, base, d.type == CBA_BF16, 4, dims, strides, box);
}

template <int DP, bool BF16>
cudaError_t af_launch(const AfPlan &p, const AfArgs &a, const CUtensorMap *tm, cudaStream_t st) {
    // without queries there is nothing but the status to be written
    if (a.items == 0) return cudaMemsetAsync(a.status, 0, sizeof(unsigned), st);
    cudaError_t e = allow_smem<attn_fwd_kernel<DP, BF16>>((int)Af<DP>::SMEM);
    if (e != cudaSuccess) return e;
    attn_fwd_kernel<DP, BF16><<<(unsigned)a.items, kAfThreads, Af<DP>::SMEM, st>>>(tm[0], tm[1], tm[2], a);
    e = cudaGetLastError();
    if (e == cudaSuccess && p.chunks > 1)
        e = launch_pdl(attn_fwd_join_kernel<BF16>, dim3((unsigned)p.units * 2, (unsigned)(a.dim + 15) / 16), dim3(256), 0, st,
                       a, DP);
    return e;
}

}  // namespace

}  // namespace cba

using namespace cba;

extern "C" {

size_t cba_attention_forward_workspace_bytes(const cba_attention_desc_t *d) {
    AfPlan p;
    return check_attn(d, &p) == CBA_OK ? p.total : 0;
}

int cba_attention_forward(const cba_attention_desc_t *d, const void *q, const void *k, const void *v,
                          const int *cu_q, const int *cu_k, void *o, float *lse, void *workspace,
                          size_t workspace_bytes, void *stream) {
    AfPlan p;
    const int rc = check_attn(d, &p);
    if (rc != CBA_OK) return rc;
    const long long tq = d->packed ? d->total_q : d->len_q, tk = d->packed ? d->total_k : d->len_k;
    if (tq > 0 && (!q || !o)) return CBA_ERR_ARG;
    if (tk > 0 && (!k || !v)) return CBA_ERR_ARG;
    if (d->packed ? (!cu_q || !cu_k) : (cu_q || cu_k)) return CBA_ERR_ARG;
    const void *ptrs[] = {q, k, v, o};
    for (const void *x : ptrs)
        if (!aligned_to(x, 16)) return CBA_ERR_ALIGN;
    if (!aligned_to(lse, 4) || !aligned_to(cu_q, 4) || !aligned_to(cu_k, 4)) return CBA_ERR_ALIGN;
    if (!workspace || workspace_bytes < p.total) return CBA_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return CBA_ERR_ALIGN;

    AfArgs a{};
    a.cu_q = cu_q; a.cu_k = cu_k;
    a.batch = d->batch; a.hq = d->heads_q; a.hkv = d->heads_kv; a.group = d->heads_q / d->heads_kv;
    a.dim = d->dim; a.len_q = d->len_q; a.len_k = d->len_k;
    a.total_q = d->total_q; a.total_k = d->total_k;
    a.causal = d->causal;
    // S is negated for a negative scale, so that its largest is the exponent's; a scale of 0 becomes one whose
    // products with fp32 logits of size vanish, and with the masked -infinity do not become NaN
    a.cs = d->scale == 0.f ? 1e-37f : std::min(std::fabs(d->scale) * kLog2e, 3e38f);
    a.negative = d->scale < 0.f;
    a.hp = p.hp; a.hparts = p.hparts; a.tt = p.tt; a.pairs = p.pairs; a.slots = p.slots;
    a.heads_at_once = p.heads_at_once; a.chunk = p.chunk; a.chunks = p.chunks;
    a.units = p.units; a.items = p.units * p.chunks;
    a.o = o; a.lse = lse;
    a.status = static_cast<unsigned *>(workspace);
    a.ml = ws_at<float2>(workspace, p.off_ml);
    a.part = ws_at<float>(workspace, p.off_part);
    long long sq[3], sk[3], sv[3];
    fill_strides(*d, d->q, d->heads_q, tq, sq);
    fill_strides(*d, d->k, d->heads_kv, tk, sk);
    fill_strides(*d, d->v, d->heads_kv, tk, sv);
    fill_strides(*d, d->o, d->heads_q, tq, a.so);
    // without queries (or keys) the kernel loads nothing of them
    CUtensorMap tm[3] = {};
    a.maps = tq > 0 && tk > 0;
    if (a.maps &&
        (!af_map(&tm[0], q, *d, d->heads_q, tq, sq, p, true) || !af_map(&tm[1], k, *d, d->heads_kv, tk, sk, p, false) ||
         !af_map(&tm[2], v, *d, d->heads_kv, tk, sv, p, false)))
        return CBA_ERR_UNSUPPORTED;
    cudaGetLastError();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = select_device_of(workspace);
    if (e == cudaSuccess) {
        const bool bf = d->type == CBA_BF16;
        if (p.dp == 64) e = bf ? af_launch<64, true>(p, a, tm, st) : af_launch<64, false>(p, a, tm, st);
        else e = bf ? af_launch<128, true>(p, a, tm, st) : af_launch<128, false>(p, a, tm, st);
    }
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

}  // extern "C"
