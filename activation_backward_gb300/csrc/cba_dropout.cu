// cba_dropout.cu -- dropout whose mask is a function of a seed, a counter and the
// element's index, with the shortcut added in the same pass.
//
//   y_i = (word_i >= p 2^32 ? x_i / (1 - p) : 0) + residual_i
//   word_i: word i mod 4 of Philox4x32-10 at the counter offset + i / 4
//
// Philox4x32-10 is the generator of Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3" (2011): ten rounds of two 32 x 32 bit products whose
// halves are mixed with the key.  The mask is never stored: the gradient's call
// computes the words again.
//
// Memory bounds large calls, with the words' products close behind.  Measured: 65536 x 2048 bf16
// with a residual 133 us (0.89 of the copy rate; issue slots 66% taken), 43264 x 255 fp32 as one run
// 14.9 us (0.87; 18.4 from a cold start), 338 x 512 fp32 5.1.  Rows with gaps that are no whole vectors:
// 20000 x 1001 fp32, gaps of 3, 57 us, with a residual 64 (0.41, 0.56).
#include <algorithm>
#include <cmath>

#include "cba_internal.cuh"
#include "cba_ptx.cuh"
#include "cba_types.cuh"

namespace cba {

namespace {

struct DrArgs {
    const void *x, *res;
    void *y;
    const unsigned long long *step;  // added to the counter's offset; may be NULL
    unsigned long long offset;
    unsigned key0, key1;
    unsigned bound;                  // words below it are dropped
    int all;                         // 1: p = 1, every element is dropped
    float scale;
    long long n, cols;               // elements, elements of a row
    long long ld_x, ld_res, ld_y;
};

__device__ __forceinline__ uint4 philox(unsigned long long counter, unsigned k0, unsigned k1) {
    unsigned x0 = (unsigned)counter, x1 = (unsigned)(counter >> 32), x2 = 0, x3 = 0;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const unsigned long long a = (unsigned long long)x0 * 0xD2511F53u, b = (unsigned long long)x2 * 0xCD9E8D57u;
        x0 = (unsigned)(b >> 32) ^ x1 ^ k0;
        x1 = (unsigned)b;
        x2 = (unsigned)(a >> 32) ^ x3 ^ k1;
        x3 = (unsigned)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

__device__ __forceinline__ unsigned long long first_counter(const DrArgs &a) {
    return a.offset + (a.step ? *a.step : 0ull);
}

__device__ __forceinline__ float drop(const DrArgs &a, float x, unsigned word) {
    return word >= a.bound && !a.all ? x * a.scale : 0.f;
}

// i / d and the remainder; in 32 bits where they do (a 64-bit division takes five times as long).
__device__ __forceinline__ void divide(long long i, long long d, bool small, long long &q, long long &r) {
    if (small) {
        const unsigned n = (unsigned)i / (unsigned)d;
        q = n, r = (unsigned)i - n * (unsigned)d;
    } else {
        q = i / d, r = i - q * d;
    }
}

constexpr int kVectors = 4;

// Vectors of 16 bytes: rows without gaps (FLAT: the tensors are one run of n elements),
// or rows of whole vectors.  (65536 x 2048 bf16 with a residual: 4 vectors of a thread in
// flight 133 us, 2 138, 1 165.)
template <typename T, bool RES, bool FLAT>
__global__ void __launch_bounds__(256) dropout_vec_kernel(const DrArgs a) {
    constexpr int V = 16 / sizeof(T), U = kVectors;
    const long long vecs = a.n / V;
    const long long v0 = (long long)blockIdx.x * (256 * U) + threadIdx.x;
    Pack<T, V> x[U], r[U];
    long long oy[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long v = v0 + u * 256;
        if (v >= vecs) continue;
        long long ox, orr;
        if (FLAT) {
            ox = orr = oy[u] = v * V;
        } else {
            long long row, c;
            divide(v, a.cols / V, a.n < (1LL << 32), row, c);
            c *= V;
            ox = row * a.ld_x + c, orr = row * a.ld_res + c, oy[u] = row * a.ld_y + c;
        }
        x[u] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.x) + ox);
        if (RES) r[u] = *reinterpret_cast<const Pack<T, V> *>(static_cast<const T *>(a.res) + orr);
    }
    const unsigned long long first = first_counter(a);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long v = v0 + u * 256;
        if (v >= vecs) continue;
        Pack<T, V> y;
#pragma unroll
        for (int g = 0; g < V / 4; ++g) {
            const uint4 w = philox(first + (unsigned long long)(v * (V / 4) + g), a.key0, a.key1);
            const unsigned ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = g * 4 + j;
                float f = drop(a, to_f32(x[u].v[e]), ws[j]);
                if (RES) f += to_f32(r[u].v[e]);
                y.v[e] = from_f32<T>(f);
            }
        }
        *reinterpret_cast<Pack<T, V> *>(static_cast<T *>(a.y) + oy[u]) = y;
    }
    if (FLAT && blockIdx.x == 0 && threadIdx.x < a.n - vecs * V) {  // behind the last whole vector
        const long long i = vecs * V + threadIdx.x;
        const uint4 w = philox(first + (unsigned long long)(i / 4), a.key0, a.key1);
        const unsigned ws[4] = {w.x, w.y, w.z, w.w};
        float f = drop(a, to_f32(static_cast<const T *>(a.x)[i]), ws[i & 3]);
        if (RES) f += to_f32(static_cast<const T *>(a.res)[i]);
        static_cast<T *>(a.y)[i] = from_f32<T>(f);
    }
}

// Any rows: a warp takes 128 elements, each lane the words of four in a row and, by
// shuffles, the elements 32 apart that lie side by side with the other lanes'.
template <typename T, bool RES>
__global__ void __launch_bounds__(256) dropout_any_kernel(const DrArgs a) {
    const int lane = threadIdx.x & 31;
    const long long i0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 128;
    if (i0 >= a.n) return;
    float x[4], r[4];
    long long oy[4];
    long long row, c;
    divide(i0 + lane, a.cols, a.n < (1LL << 32), row, c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const long long i = i0 + j * 32 + lane;
        if (j > 0) {
            c += 32;
            if (a.cols >= 32) {
                if (c >= a.cols) c -= a.cols, ++row;
            } else {
                const unsigned n = (unsigned)c / (unsigned)a.cols;
                row += n, c -= n * a.cols;
            }
        }
        oy[j] = -1;
        if (i >= a.n) continue;
        x[j] = to_f32(static_cast<const T *>(a.x)[row * a.ld_x + c]);
        if (RES) r[j] = to_f32(static_cast<const T *>(a.res)[row * a.ld_res + c]);
        oy[j] = row * a.ld_y + c;
    }
    const uint4 w = philox(first_counter(a) + (unsigned long long)(i0 / 4 + lane), a.key0, a.key1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int from = j * 8 + (lane >> 2);
        const unsigned w0 = __shfl_sync(0xffffffffu, w.x, from), w1 = __shfl_sync(0xffffffffu, w.y, from),
                       w2 = __shfl_sync(0xffffffffu, w.z, from), w3 = __shfl_sync(0xffffffffu, w.w, from);
        const unsigned word = lane & 2 ? (lane & 1 ? w3 : w2) : (lane & 1 ? w1 : w0);
        if (oy[j] < 0) continue;
        float f = drop(a, x[j], word);
        if (RES) f += r[j];
        static_cast<T *>(a.y)[oy[j]] = from_f32<T>(f);
    }
}

template <typename T, bool RES>
cudaError_t dropout_launch(const DrArgs &a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    auto vec = [&](const void *p, long long ld) { return aligned_to(p, 16) && ld % V == 0; };
    const bool flat = a.ld_x == a.cols && a.ld_y == a.cols && (!RES || a.ld_res == a.cols);
    const bool bases = aligned_to(a.x, 16) && aligned_to(a.y, 16) && (!RES || aligned_to(a.res, 16));
    const bool rows = a.cols % V == 0 && vec(a.x, a.ld_x) && vec(a.y, a.ld_y) && (!RES || vec(a.res, a.ld_res));
    const long long blocks = (a.n + 256 * kVectors * V - 1) / (256 * kVectors * V);
    if (flat && bases) dropout_vec_kernel<T, RES, true><<<(unsigned)blocks, 256, 0, st>>>(a);
    else if (rows) dropout_vec_kernel<T, RES, false><<<(unsigned)blocks, 256, 0, st>>>(a);
    else dropout_any_kernel<T, RES><<<(unsigned)((a.n + 1023) / 1024), 256, 0, st>>>(a);
    return cudaGetLastError();
}

int check_desc(const cba_dropout_desc_t *d) {
    if (!d || d->rows < 0 || d->cols < 1 || !dtype_ok(d->type)) return CBA_ERR_ARG;
    if (!(d->p >= 0.f && d->p <= 1.f)) return CBA_ERR_ARG;
    const long long lds[] = {d->ld_x, d->ld_residual, d->ld_y};
    for (const long long l : lds) {
        if (l != 0 && l < d->cols) return CBA_ERR_ARG;
        if (l > (1LL << 38)) return CBA_ERR_UNSUPPORTED;
    }
    // (a grid of one block per 1024 elements)
    if (d->rows > (1LL << 40) / d->cols) return CBA_ERR_UNSUPPORTED;
    return CBA_OK;
}

}  // namespace

}  // namespace cba

using namespace cba;

extern "C" {

int cba_dropout(const cba_dropout_desc_t *d, const void *x, const void *residual,
                const unsigned long long *step, void *y, void *stream) {
    const int rc = check_desc(d);
    if (rc != CBA_OK) return rc;
    if (d->rows == 0) return CBA_OK;
    if (!x || !y) return CBA_ERR_ARG;
    const size_t e = dtype_bytes(d->type);
    if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(residual, e) || !aligned_to(step, 8)) return CBA_ERR_ALIGN;
    DrArgs a{};
    a.x = x; a.res = residual; a.y = y; a.step = step;
    a.offset = d->offset;
    a.key0 = (unsigned)d->seed;
    a.key1 = (unsigned)(d->seed >> 32);
    const double bound = std::nearbyint((double)d->p * 4294967296.0);
    a.all = bound > 4294967295.0;
    a.bound = a.all ? 0xffffffffu : (unsigned)bound;
    a.scale = d->p < 1.f ? (float)(1.0 / (1.0 - (double)d->p)) : 0.f;
    a.n = d->rows * d->cols;
    a.cols = d->cols;
    a.ld_x = d->ld_x ? d->ld_x : d->cols;
    a.ld_res = d->ld_residual ? d->ld_residual : d->cols;
    a.ld_y = d->ld_y ? d->ld_y : d->cols;
    cudaGetLastError();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t err = select_device_of(y);
    if (err == cudaSuccess) {
        auto run = [&](auto t) {
            using T = decltype(t);
            return residual ? dropout_launch<T, true>(a, st) : dropout_launch<T, false>(a, st);
        };
        err = d->type == CBA_F32 ? run(0.f) : d->type == CBA_F16 ? run(__half{}) : run(__nv_bfloat16{});
    }
    return err == cudaSuccess ? CBA_OK : report_cuda_error(err);
}

}  // extern "C"
