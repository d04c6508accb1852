// cba_attention_fwd.cu -- attention's forward pass: o and the rows' log-sum-exp.
//
//   S = scale q k^T,  m = max_j S_ij over the allowed pairs
//   l = sum_j exp(S_ij - m),  o = sum_j exp(S_ij - m) v_j / l,  lse = m + log l
//
// One pass over the keys with a running maximum and sum: when the maximum grows,
// the sums so far are scaled down.  A warp per query row, the row's elements over
// its lanes.
#include <algorithm>
#include <cmath>

#include "cba_internal.cuh"
#include "cba_ptx.cuh"
#include "cba_types.cuh"

namespace cba {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AfArgs {
    const int *cu_q, *cu_k;
    int batch, hq, hkv, group, dim, len_q, len_k;
    long long total_q, total_k;
    int causal;
    float scale;
    const void *q, *k, *v;
    void *o;
    float *lse;
    long long sq[3], sk[3], sv[3], so[3];
    unsigned *status;
};

template <typename T>
__global__ void __launch_bounds__(128) attn_fwd_rows_kernel(const AfArgs a) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    const int lane = threadIdx.x & 31;
    const long long tokens = a.cu_q ? a.total_q : (long long)a.batch * a.len_q;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= tokens * a.hq) return;
    const int h = (int)(row / tokens);
    const long long t = row - (long long)h * tokens;
    // the row's sequence and index in it
    int b, i, lq, lk;
    long long q0 = 0, k0 = 0;
    if (a.cu_q) {
        int lo = 0, hi = a.batch;  // the last sequence that starts at t or before
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.cu_q[mid] <= t) lo = mid;
            else hi = mid;
        }
        b = 0;
        q0 = min(max((long long)a.cu_q[lo], 0LL), a.total_q);
        const long long q1 = min(max((long long)a.cu_q[lo + 1], q0), a.total_q);
        k0 = min(max((long long)a.cu_k[lo], 0LL), a.total_k);
        const long long k1 = min(max((long long)a.cu_k[lo + 1], k0), a.total_k);
        if (t < q0 || t >= q1 || t - q0 >= a.len_q) return;
        lq = (int)min(q1 - q0, (long long)a.len_q);
        lk = (int)min(k1 - k0, (long long)a.len_k);
        i = (int)(t - q0);
    } else {
        b = (int)(t / a.len_q);
        i = (int)(t - (long long)b * a.len_q);
        lq = a.len_q, lk = a.len_k;
    }
    const int hk = h / a.group;
    const T *q = static_cast<const T *>(a.q) + b * a.sq[0] + (q0 + i) * a.sq[1] + h * a.sq[2];
    const T *k = static_cast<const T *>(a.k) + b * a.sk[0] + k0 * a.sk[1] + hk * a.sk[2];
    const T *v = static_cast<const T *>(a.v) + b * a.sv[0] + k0 * a.sv[1] + hk * a.sv[2];
    float qs[4], acc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        qs[e] = lane * 4 + e < a.dim ? to_f32(q[lane * 4 + e]) : 0.f;
        acc[e] = 0.f;
    }
    const int n = a.causal ? min(lk, i + lk - lq + 1) : lk;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
        float s = 0.f, vs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = lane * 4 + e < a.dim;
            s = fmaf(qs[e], in ? to_f32(k[j * a.sk[1] + lane * 4 + e]) : 0.f, s);
            vs[e] = in ? to_f32(v[j * a.sv[1] + lane * 4 + e]) : 0.f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= a.scale;
        const float top = fmaxf(m, s), ref = top == -INFINITY ? 0.f : top;
        const float was = expf(m - ref), p = expf(s - ref);
        l = l * was + p;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = acc[e] * was + p * vs[e];
        m = top;
    }
    T *o = static_cast<T *>(a.o) + b * a.so[0] + (q0 + i) * a.so[1] + h * a.so[2];
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (lane * 4 + e < a.dim) o[lane * 4 + e] = from_f32<T>(l == 0.f ? 0.f : acc[e] * inv);
    if (lane == 0 && a.lse)
        a.lse[a.cu_q ? (long long)h * a.total_q + t : ((long long)b * a.hq + h) * a.len_q + i] =
            l == 0.f ? -INFINITY : m + logf(l);
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
    const double rows = d->packed ? (double)d->total_q : (double)d->batch * d->len_q;
    if (rows * d->heads_q >= 4294967296.0) return CBA_ERR_UNSUPPORTED;
    return CBA_OK;
}

// The strides that the kernels use; packed sequences have none from one to the next.
void fill_strides(const cba_attention_desc_t &d, const cba_attn_strides_t &s, int heads, long long len, long long *out) {
    const bool none = !s.batch && !s.token && !s.head;
    out[0] = d.packed ? 0 : none ? len * heads * d.dim : s.batch;
    out[1] = none ? (long long)heads * d.dim : s.token;
    out[2] = none ? d.dim : s.head;
}

}  // namespace

}  // namespace cba

using namespace cba;

extern "C" {

size_t cba_attention_forward_workspace_bytes(const cba_attention_desc_t *d) {
    return check_desc(d) == CBA_OK ? 256 : 0;
}

int cba_attention_forward(const cba_attention_desc_t *d, const void *q, const void *k, const void *v,
                          const int *cu_q, const int *cu_k, void *o, float *lse, void *workspace,
                          size_t workspace_bytes, void *stream) {
    const int rc = check_desc(d);
    if (rc != CBA_OK) return rc;
    const long long tq = d->packed ? d->total_q : d->len_q, tk = d->packed ? d->total_k : d->len_k;
    if (tq > 0 && (!q || !o)) return CBA_ERR_ARG;
    if (tk > 0 && (!k || !v)) return CBA_ERR_ARG;
    if (d->packed ? (!cu_q || !cu_k) : (cu_q || cu_k)) return CBA_ERR_ARG;
    const void *ptrs[] = {q, k, v, o};
    for (const void *x : ptrs)
        if (!aligned_to(x, 16)) return CBA_ERR_ALIGN;
    if (!aligned_to(lse, 4) || !aligned_to(cu_q, 4) || !aligned_to(cu_k, 4)) return CBA_ERR_ALIGN;
    if (!workspace || workspace_bytes < cba_attention_forward_workspace_bytes(d)) return CBA_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return CBA_ERR_ALIGN;
    AfArgs a{};
    a.cu_q = cu_q; a.cu_k = cu_k;
    a.batch = d->batch; a.hq = d->heads_q; a.hkv = d->heads_kv; a.group = d->heads_q / d->heads_kv;
    a.dim = d->dim; a.len_q = d->len_q; a.len_k = d->len_k;
    a.total_q = d->total_q; a.total_k = d->total_k;
    a.causal = d->causal; a.scale = d->scale;
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    a.status = static_cast<unsigned *>(workspace);
    fill_strides(*d, d->q, d->heads_q, tq, a.sq);
    fill_strides(*d, d->k, d->heads_kv, tk, a.sk);
    fill_strides(*d, d->v, d->heads_kv, tk, a.sv);
    fill_strides(*d, d->o, d->heads_q, tq, a.so);
    cudaGetLastError();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = select_device_of(workspace);
    if (e == cudaSuccess) {
        const long long rows = (d->packed ? tq : tq * d->batch) * d->heads_q;
        const unsigned grid = (unsigned)std::max(1LL, (rows + 3) / 4);
        if (d->type == CBA_BF16) attn_fwd_rows_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
        else attn_fwd_rows_kernel<__half><<<grid, 128, 0, st>>>(a);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? CBA_OK : report_cuda_error(e);
}

}  // extern "C"
