// Row operators in front of an 8-bit product, for gfx950: root-mean-square
// norm with the residual's addition (forward, with an 8-bit output, and
// backward), rows to 8 bits with a scale each, and back.
//
// Forward, row t of [T, d], all in fp32, each output rounded once:
//   h = x + residual,  rstd = 1 / sqrt(mean_j h_j^2 + eps),  y = h rstd w
//   scale = max_j |y_j| fl(1/127),  q_j = rint(y_j / scale)
// The codes are those of the fp32 y, with the division rounded as IEEE has it:
// an outlier channel makes a code's step a large part of a row's rms, and a
// code that falls the other way at a tie is seen.  (One reduction would do, as
// rstd cancels in y / scale; it saved under 2% at 4096 x 8192, the row's bytes
// being what counts.)  Rows to 8 bits are the same with rstd = 1 and w the column scale.
//
// Backward, from dy into y and dh into h (rstd kept by the forward pass):
//   u = w dy,  dx = rstd (u - h rstd^2 mean_j(u_j h_j)) + dh,  dw_j = sum_t dy h rstd
// dx is the gradient of both x and the residual.  dw is summed per workgroup
// over its rows, then over workgroups in a fixed order: no atomics, bitwise
// reproducible.
//
// All of them are bound by HBM.  A workgroup owns a row (the backward pass: a
// sequence of rows) and holds it in registers between the reduction and the
// stores, P accesses of 16 bytes per thread; rows too long for that are read
// again from cache.  Measured at 4096 x 8192 in bf16 (a copy of 1 GiB: 5.1
// TB/s): norm with h and y 49.5 us, 5.4 TB/s; with h and codes 43.3 us, 5.4;
// rows to 8 bits 18.8 us, 5.4; back 16.8 us, 6.0; backward pass 48.9 us, 5.5,
// and 57.4 with dw.  A token of 4096: 3.0, 3.7, 2.7, 2.3 and 3.0 us.  Rows too
// long for the registers, norm with h and y: 31.5 us at 512 x 33000 in bf16, 4.3
// TB/s of the bytes that count (30720 in registers: 6.3).
#include "dora_device.h"
#include "dora_launch.h"

namespace dora {
namespace {

constexpr int kMaxWaves = 16;
constexpr uint32_t kInfBits = 0x7f800000u;
// Rows whose largest value is below 2^-119 quantise to zeros with scale 0: the
// scale would be subnormal there.  The error is below 2^-119.
constexpr uint32_t kTinyBits = (uint32_t)(127 - 119) << 23;

// Rows go in packs of 16 bytes.  Aligned rows (AL: pointers and row pitch
// multiples of 16 bytes) hold whole packs; in others a pack is read and
// written at its element's alignment, which the memory pipe splits (element
// by element it took 2.5 times as long at 2048 x 5121), and the last one may
// be partial: elements past the row's end read 0 and are not written.
template <typename E, bool AL>
__device__ __forceinline__ Pack<E> load_row(const E* p, int64_t left) {
    constexpr int N = Pack<E>::N;
    Pack<E> k;
    if (AL) {
        k = load_pack(p);
    } else if (left >= N) {
        __builtin_memcpy(&k.u, p, 16);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) k.e[e] = e < left ? p[e] : Cvt<E>::from_f(0.0f);
    }
    return k;
}

template <typename E, bool AL, int N>
__device__ __forceinline__ void store_row(E* p, const float (&v)[N], int64_t left) {
    static_assert(N == Pack<E>::N, "a pack");
    Pack<E> k;
#pragma unroll
    for (int e = 0; e < N; ++e) k.e[e] = Cvt<E>::from_f(v[e]);
    if (AL) {
        store_pack_stream(p, k);
    } else if (left >= N) {
        __builtin_memcpy(p, &k.u, 16);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < left) p[e] = k.e[e];
    }
}

template <typename E>
__device__ __forceinline__ float at(const Pack<E>& k, int e) {
    return Cvt<E>::to_f(k.e[e]);
}

// N weights (of the row's type) or column scales (fp32) as fp32.
template <typename W, bool AL, int N>
__device__ __forceinline__ void load_w(const W* w, int64_t left, float (&v)[N]) {
    constexpr int M = Pack<W>::N;
#pragma unroll
    for (int h = 0; h < N; h += M) {
        const Pack<W> k = load_row<W, AL>(w + h, left - h);
#pragma unroll
        for (int e = 0; e < M; ++e) v[h + e] = at(k, e);
    }
}

// What the codes of a row divide by: scale and its reciprocal, both 0 where
// the codes are 0 (scale 0 or NaN).
struct Divisor {
    float scale, recip;
};

__device__ __forceinline__ Divisor divisor(float scale) {
    return scale > 0.0f ? Divisor{scale, 1.0f / scale} : Divisor{0.0f, 0.0f};
}

// N codes: rint(p / scale) packed into bytes.  |p / scale| <= 127 up to a
// rounding or two, which rint takes back to 127.  The quotient is Markstein's:
// p times the reciprocal, corrected by its remainder, which is p / scale
// correctly rounded (a division for each element took 22.6 us at 4096 x 8192
// where this takes 18).  Below a largest |p| of 2^-94 the remainder may
// underflow, and a code next to a tie be the other one.
template <bool AL, int N>
__device__ __forceinline__ void store_codes(int8_t* q, const float (&p)[N], const Divisor& by, int64_t left) {
    int c[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float v = by.recip == 0.0f ? 0.0f : p[e];   // not a NaN's or an infinity's product with 0
        const float quot = v * by.recip;
        c[e] = (int)rintf(fmaf(fmaf(-quot, by.scale, v), by.recip, quot));
    }
    uint32_t u[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
        u[i] = (c[4 * i] & 255) | (c[4 * i + 1] & 255) << 8 | (c[4 * i + 2] & 255) << 16 | (uint32_t)c[4 * i + 3] << 24;
    if (AL) {
        __builtin_memcpy(__builtin_assume_aligned(q, N), u, N);
    } else if (left >= N) {
        __builtin_memcpy(q, u, N);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < left) q[e] = (int8_t)c[e];
    }
}

// The sum or the maximum over the workgroup, returned to every thread.  Sums
// are added in a fixed order.  red holds kMaxWaves entries and is free to be
// written again after the next barrier.
template <typename V, typename Op>
__device__ __forceinline__ V block_reduce(V v, V* red, Op op) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = op(v, __shfl_xor(v, o));
    const int nw = blockDim.x >> 6;
    if (nw == 1) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < nw; ++i) v = op(v, red[i]);
    return v;
}

__device__ __forceinline__ float block_sum(float v, float* red) {
    return block_reduce(v, red, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
    return block_reduce(v, red, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// |v|'s bits, whose order as integers is the values', NaN above infinity.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// A row's scale from the bits of its largest |value|: times fl(1/127), which is
// the quotient by 127 but for its last bit in 4.5% of values.  The codes are
// exact for the scale as it is stored; a division would change those of weights
// that are kept (torch's amax / 127 on the GPU is this product too).  A row that
// holds a NaN or an infinity has scale NaN (and codes 0), so all that comes of it
// is NaN.
__device__ __forceinline__ float code_scale(uint32_t top) {
    return top >= kInfBits ? __uint_as_float(0x7fc00000u) : top < kTinyBits ? 0.0f : __uint_as_float(top) * (1.0f / 127.0f);
}

__device__ __forceinline__ float row_rstd(float sum, int64_t d, float eps) { return rsqrtf(sum * (1.0f / (float)d) + eps); }

struct RowArgs {
    const void* x;
    const void* res;
    const void* w;
    int64_t row0, rows, d;   // workgroup b owns row row0 + b
    float eps;
    void* h;
    void* y;
    int8_t* q;
    float* scale;
    float* rstd;
};

// One row per workgroup, the row in registers.  NORM: the norm (w of type E,
// outputs h, y, q, rstd as asked); otherwise rows to 8 bits (w an optional
// fp32 column scale).
template <typename E, typename W, bool AL, int P, bool NORM>
__global__ __launch_bounds__(P > 4 ? 512 : 1024) void row_regs(RowArgs a) {
    constexpr int N = Pack<E>::N;
    __shared__ float rs[kMaxWaves];
    __shared__ uint32_t rt[kMaxWaves];
    const int64_t row = a.row0 + blockIdx.x, off = row * a.d;
    const E* x = static_cast<const E*>(a.x) + off;
    const W* w = static_cast<const W*>(a.w);
    const int d = (int)a.d, n = (d + N - 1) / N, nt = blockDim.x;
    float v[P][N];
    {
        Pack<E> xv[P], rv[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
            if (k < n) {
                xv[i] = load_row<E, AL>(x + k * N, d - k * N);
                if (NORM && a.res) rv[i] = load_row<E, AL>(static_cast<const E*>(a.res) + off + k * N, d - k * N);
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                v[i][e] = k < n ? at(xv[i], e) : 0.0f;
                if (NORM && a.res) v[i][e] += k < n ? at(rv[i], e) : 0.0f;
            }
        }
    }
    float rstd = 1.0f;
    if (NORM) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
#pragma unroll
            for (int e = 0; e < N; ++e) sum = fmaf(v[i][e], v[i][e], sum);
            if (a.h && k < n) store_row<E, AL>(static_cast<E*>(a.h) + off + k * N, v[i], d - k * N);
        }
        rstd = row_rstd(block_sum(sum, rs), a.d, a.eps);
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {   // v becomes y
        const int k = threadIdx.x + i * nt;
        if (k >= n) continue;
        float wv[N];
#pragma unroll
        for (int e = 0; e < N; ++e) wv[e] = 1.0f;
        if (w) load_w<W, AL>(w + k * N, d - k * N, wv);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            v[i][e] = (v[i][e] * rstd) * wv[e];
            const uint32_t m = magnitude(v[i][e]);
            top = m > top ? m : top;
        }
        if (NORM && a.y) store_row<E, AL>(static_cast<E*>(a.y) + off + k * N, v[i], d - k * N);
    }
    if (!a.q) return;
    const float scale = code_scale(block_max(top, rt));
    if (threadIdx.x == 0) a.scale[row] = scale;
    const Divisor by = divisor(scale);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int k = threadIdx.x + i * nt;
        if (k < n) store_codes<AL>(a.q + off + k * N, v[i], by, d - k * N);
    }
}

// The same for rows of any length, read once for each of their passes.
template <typename E, typename W, bool AL, bool NORM>
__global__ __launch_bounds__(1024) void row_long(RowArgs a) {
    constexpr int N = Pack<E>::N;
    __shared__ float rs[kMaxWaves];
    __shared__ uint32_t rt[kMaxWaves];
    const int64_t row = a.row0 + blockIdx.x, off = row * a.d, n = (a.d + N - 1) / N;
    const E* x = static_cast<const E*>(a.x) + off;
    const E* r = NORM && a.res ? static_cast<const E*>(a.res) + off : nullptr;
    const W* w = static_cast<const W*>(a.w);
    auto sum_at = [&](int64_t k, float (&v)[N]) __attribute__((always_inline)) {
        Pack<E> t = load_row<E, AL>(x + k * N, a.d - k * N);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = at(t, e);
        if (r) {
            t = load_row<E, AL>(r + k * N, a.d - k * N);
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] += at(t, e);
        }
    };
    auto scaled = [&](int64_t k, float (&v)[N], float rstd) __attribute__((always_inline)) {
        float wv[N];
#pragma unroll
        for (int e = 0; e < N; ++e) wv[e] = 1.0f;
        if (w) load_w<W, AL>(w + k * N, a.d - k * N, wv);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = (v[e] * rstd) * wv[e];
    };
    float rstd = 1.0f;
    if (NORM) {
        float sum = 0.0f;
        for (int64_t k = threadIdx.x; k < n; k += blockDim.x) {
            float v[N];
            sum_at(k, v);
#pragma unroll
            for (int e = 0; e < N; ++e) sum = fmaf(v[e], v[e], sum);
        }
        rstd = row_rstd(block_sum(sum, rs), a.d, a.eps);
        if (threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
    }
    float scale = 0.0f;
    if (a.q) {
        uint32_t top = 0;
        for (int64_t k = threadIdx.x; k < n; k += blockDim.x) {
            float v[N];
            sum_at(k, v);
            scaled(k, v, rstd);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const uint32_t m = magnitude(v[e]);
                top = m > top ? m : top;
            }
        }
        scale = code_scale(block_max(top, rt));
        if (threadIdx.x == 0) a.scale[row] = scale;
    }
    const Divisor by = divisor(scale);
    // each element is read by the thread that writes it, so h may be x or the
    // residual itself
    for (int64_t k = threadIdx.x; k < n; k += blockDim.x) {
        float v[N];
        sum_at(k, v);
        const int64_t left = a.d - k * N;
        if (NORM && a.h) store_row<E, AL>(static_cast<E*>(a.h) + off + k * N, v, left);
        scaled(k, v, rstd);
        if (NORM && a.y) store_row<E, AL>(static_cast<E*>(a.y) + off + k * N, v, left);
        if (a.q) store_codes<AL>(a.q + off + k * N, v, by, left);
    }
}

// ------------------------------------------------------------- backward

struct BwdArgs {
    const void* dy;
    const void* h;
    const void* w;
    const float* rstd;
    const void* dh;
    int64_t row0, rows, d;
    void* dx;
    float* part;   // dw partials [workgroups][d], or nullptr
};

// Rows blockIdx.x, blockIdx.x + gridDim.x, ... of one workgroup, each in
// registers between its reduction and its store.  Six accesses a thread (eight
// of fp32), for the longest rows, leave no registers for w and dh: they are
// loaded where they are used (with them in registers that spill, 4 accesses held
// to 128 took 60 us instead of 18 at 2048 x 5120).  Eight of fp32 at 1024 threads
// still spill 23 registers, 48 where rows are not aligned: 77 us at 512 x 28672,
// 3.0 TB/s, against 2.6 TB/s of the rows too long for them (512 x 40000, 124 us);
// six of bf16 do not: 35 us at 512 x 30720, 3.6 TB/s, against 1.8 (512 x 33000, 73
// us).
template <typename E, bool AL, int P>
__global__ __launch_bounds__(P == 4 ? 512 : P == 6 ? 640 : 1024) void rms_bwd_regs(BwdArgs a) {
    constexpr int N = Pack<E>::N;
    constexpr bool WIDE = P > 4;
    __shared__ float rs[2][kMaxWaves];
    const int d = (int)a.d, n = (d + N - 1) / N, nt = blockDim.x;
    const E* w = static_cast<const E*>(a.w);
    Pack<E> wv[WIDE ? 1 : P];
    float dw[P][N];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int k = threadIdx.x + i * nt;
#pragma unroll
        for (int e = 0; e < N; ++e) dw[i][e] = 0.0f;
        if (!WIDE && k < n) wv[i] = load_row<E, AL>(w + k * N, d - k * N);
    }
    int par = 0;   // the reduction's buffer: the other one than the last row's, which slow waves may still read
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, par ^= 1) {
        const int64_t off = row * a.d;
        const E* dh = a.dh ? static_cast<const E*>(a.dh) + off : nullptr;
        Pack<E> dyv[P], hv[P], gv[WIDE ? 1 : P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
            if (k < n) {
                dyv[i] = load_row<E, AL>(static_cast<const E*>(a.dy) + off + k * N, d - k * N);
                hv[i] = load_row<E, AL>(static_cast<const E*>(a.h) + off + k * N, d - k * N);
                if (!WIDE && dh) gv[i] = load_row<E, AL>(dh + k * N, d - k * N);
            }
        }
        const float r = a.rstd[row];
        float c = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
            if (k >= n) continue;
            if (WIDE) wv[0] = load_row<E, AL>(w + k * N, d - k * N);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float dv = at(dyv[i], e), hh = at(hv[i], e);
                c = fmaf(dv * at(wv[WIDE ? 0 : i], e), hh, c);
                dw[i][e] = fmaf(dv, hh * r, dw[i][e]);
            }
        }
        const float f = block_sum(c, rs[par]) / (float)a.d * r * r;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            // the row is kept as it was loaded: without this the compiler
            // holds the fp32 values of the first use, twice the registers
            asm volatile("" : "+v"(dyv[i].u), "+v"(hv[i].u));
            const int k = threadIdx.x + i * nt;
            if (k >= n) continue;
            if (WIDE) {
                wv[0] = load_row<E, AL>(w + k * N, d - k * N);
                if (dh) gv[0] = load_row<E, AL>(dh + k * N, d - k * N);
            }
            float o[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float u = at(dyv[i], e) * at(wv[WIDE ? 0 : i], e);
                o[e] = r * (u - at(hv[i], e) * f) + (dh ? at(gv[WIDE ? 0 : i], e) : 0.0f);
            }
            store_row<E, AL>(static_cast<E*>(a.dx) + off + k * N, o, d - k * N);
        }
    }
    if (a.part) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
            if (k >= n) continue;
            float* dst = a.part + (int64_t)blockIdx.x * a.d + k * N;
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (AL || k * N + e < d) dst[e] = dw[i][e];
        }
    }
}

// Rows of any length: dx with the row read twice, and dw's partials by
// columns.
template <typename E>
__global__ __launch_bounds__(1024) void rms_bwd_long(BwdArgs a) {
    __shared__ float rs[kMaxWaves];
    const int64_t row = a.row0 + blockIdx.x, off = row * a.d;
    const E* dy = static_cast<const E*>(a.dy) + off;
    const E* h = static_cast<const E*>(a.h) + off;
    const E* dh = a.dh ? static_cast<const E*>(a.dh) + off : nullptr;
    const E* w = static_cast<const E*>(a.w);
    const float r = a.rstd[row];
    float c = 0.0f;
    for (int64_t k = threadIdx.x; k < a.d; k += blockDim.x)
        c = fmaf(Cvt<E>::to_f(dy[k]) * Cvt<E>::to_f(w[k]), Cvt<E>::to_f(h[k]), c);
    const float f = block_sum(c, rs) / (float)a.d * r * r;
    for (int64_t k = threadIdx.x; k < a.d; k += blockDim.x) {
        const float u = Cvt<E>::to_f(dy[k]) * Cvt<E>::to_f(w[k]);
        const float o = r * (u - Cvt<E>::to_f(h[k]) * f) + (dh ? Cvt<E>::to_f(dh[k]) : 0.0f);
        static_cast<E*>(a.dx)[off + k] = Cvt<E>::from_f(o);
    }
}

template <typename E>
__global__ __launch_bounds__(256) void rms_dw_cols(BwdArgs a) {
    const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (col >= a.d) return;
    float s = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const int64_t i = row * a.d + col;
        s = fmaf(Cvt<E>::to_f(static_cast<const E*>(a.dy)[i]), Cvt<E>::to_f(static_cast<const E*>(a.h)[i]) * a.rstd[row], s);
    }
    a.part[(int64_t)blockIdx.y * a.d + col] = s;
}

// dw_j = sum of the partials of column j: lane w of a column adds partials w,
// w + kDwLanes, ... in order, a batch of loads at a time, then the lanes' sums
// are added in order.  N columns a thread (16 bytes where d is a multiple of
// 4).  One load at a time took 20 us at 512 x 5120, more than the pass before
// it.
constexpr int kDwCols = 32, kDwBatch = 16;

template <int N>
__global__ __launch_bounds__(256) void dw_finalize(const float* __restrict__ part, int nparts, int64_t d,
                                                   float* __restrict__ dw) {
    constexpr int kThreads = kDwCols / N, kDwLanes = 256 / kThreads;
    __shared__ float red[kDwLanes][kDwCols];
    const int c = threadIdx.x % kThreads * N, w = threadIdx.x / kThreads;
    for (int64_t j0 = (int64_t)blockIdx.x * kDwCols; j0 < d; j0 += (int64_t)gridDim.x * kDwCols) {
        const int64_t j = j0 + c;
        float s[N];
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = 0.0f;
        if (j < d) {
            for (int p0 = w; p0 < nparts; p0 += kDwLanes * kDwBatch) {
                float v[kDwBatch][N];
#pragma unroll
                for (int i = 0; i < kDwBatch; ++i) {
                    const int p = p0 + i * kDwLanes;
#pragma unroll
                    for (int e = 0; e < N; ++e) v[i][e] = 0.0f;
                    if (p >= nparts) continue;
                    if constexpr (N == 1)
                        v[i][0] = part[(int64_t)p * d + j];
                    else
                        load_w<float, true>(part + (int64_t)p * d + j, N, v[i]);
                }
#pragma unroll
                for (int i = 0; i < kDwBatch; ++i)
#pragma unroll
                    for (int e = 0; e < N; ++e) s[e] += v[i][e];
            }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) red[w][c + e] = s[e];
        __syncthreads();
        const int64_t o = j0 + threadIdx.x;
        if (threadIdx.x < kDwCols && o < d) {
            float v = red[0][threadIdx.x];
#pragma unroll
            for (int q = 1; q < kDwLanes; ++q) v += red[q][threadIdx.x];
            dw[o] = v;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------- dequantise

template <typename E, bool AL>
__global__ __launch_bounds__(256) void dequantize(const int8_t* __restrict__ q, const float* __restrict__ scale,
                                                  int64_t rows, int64_t d, E* __restrict__ out) {
    constexpr int N = Pack<E>::N;
    const int64_t n = (d + N - 1) / N;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const float s = scale[row];
        for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256) {
            const int8_t* src = q + row * d + k * N;
            const int64_t left = d - k * N;
            int8_t c[N] = {};
            if (AL) {
                __builtin_memcpy(c, __builtin_assume_aligned(src, N), N);
            } else if (left >= N) {
                __builtin_memcpy(c, src, N);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (e < left) c[e] = src[e];
            }
            float v[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                v[e] = (float)c[e] * s;
                // the product as it is in fp32: in fp16 the compiler otherwise
                // joins it with its conversion where rows are not aligned, and
                // not where they are, and the two round differently
                asm volatile("" : "+v"(v[e]));
            }
            store_row<E, AL>(out + row * d + k * N, v, left);
        }
    }
}

// ------------------------------------------------------------- launches

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Accesses per thread P and threads for a row of n accesses: few rows take
// the widest workgroup (latency), many rows about 256 threads each.  0 where
// the row does not fit the registers.
constexpr int64_t kManyRows = 512;

struct RowShape {
    int p, nt;
};

// Up to 4 accesses a thread a workgroup may have 1024 threads, with 8 of them
// 512 (pmax: the most that a kernel is built for).
RowShape row_shape(int64_t n, int64_t rows, int pmax) {
    const int64_t most = rows >= kManyRows ? 256 : 1024;
    int p = 1;
    while (p < pmax && n > most * p) p *= 2;
    const int64_t nt = ((n + p - 1) / p + 63) / 64 * 64;
    if (nt > (p > 4 ? 512 : 1024)) return {0, 1024};
    return {p, (int)nt};
}

// Rows per launch: a grid's threads are counted in 32 bits.
constexpr int64_t kRowsPerLaunch = (int64_t)1 << 21;

template <typename E, typename W, bool AL, bool NORM>
hipError_t launch_rows(RowArgs a, hipStream_t st) {
    const RowShape s = row_shape((a.d + Pack<E>::N - 1) / Pack<E>::N, a.rows, 8);
    for (a.row0 = 0; a.row0 < a.rows; a.row0 += kRowsPerLaunch) {
        const int64_t left = a.rows - a.row0;
        const unsigned g = (unsigned)(left < kRowsPerLaunch ? left : kRowsPerLaunch);
        switch (s.p) {
            case 1: row_regs<E, W, AL, 1, NORM><<<g, s.nt, 0, st>>>(a); break;
            case 2: row_regs<E, W, AL, 2, NORM><<<g, s.nt, 0, st>>>(a); break;
            case 4: row_regs<E, W, AL, 4, NORM><<<g, s.nt, 0, st>>>(a); break;
            case 8: row_regs<E, W, AL, 8, NORM><<<g, s.nt, 0, st>>>(a); break;
            default: row_long<E, W, AL, NORM><<<g, s.nt, 0, st>>>(a); break;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename E>
hipError_t norm_typed(const RowArgs& a, hipStream_t st) {
    constexpr int N = Pack<E>::N;
    const bool vec = a.d % N == 0 && aligned_to(a.x, 16) && aligned_to(a.res, 16) && aligned_to(a.w, 16) &&
                     aligned_to(a.h, 16) && aligned_to(a.y, 16) && aligned_to(a.q, N);
    return vec ? launch_rows<E, E, true, true>(a, st) : launch_rows<E, E, false, true>(a, st);
}

template <typename E>
hipError_t quantize_typed(const RowArgs& a, hipStream_t st) {
    constexpr int N = Pack<E>::N;
    const bool vec = a.d % N == 0 && aligned_to(a.x, 16) && aligned_to(a.w, 16) && aligned_to(a.q, N);
    return vec ? launch_rows<E, float, true, false>(a, st) : launch_rows<E, float, false, false>(a, st);
}

// Workgroups of the backward pass, each with its own row of dw partials: one
// for each row up to a CU each, then four rows each, so that the partials stay
// a fraction of what is read.
constexpr int64_t kBwdParts = 512, kBwdRows = 4;

int bwd_parts(int64_t rows) {
    if (rows <= 256) return (int)rows;
    const int64_t p = (rows + kBwdRows - 1) / kBwdRows;
    return (int)(p < 256 ? 256 : p < kBwdParts ? p : kBwdParts);
}

template <typename E, bool AL>
bool launch_bwd_regs(const BwdArgs& a, int parts, hipStream_t st) {
    const int64_t n = (a.d + Pack<E>::N - 1) / Pack<E>::N;
    constexpr int LONG = sizeof(E) == 4 ? 8 : 6;   // accesses a thread of the longest rows
    if (n > LONG * (LONG == 8 ? 1024 : 640)) return false;
    const RowShape s = n <= 4 * 512 ? row_shape(n, a.rows, 4) : RowShape{LONG, (int)(((n + LONG - 1) / LONG + 63) / 64 * 64)};
    switch (s.p) {
        case 1: rms_bwd_regs<E, AL, 1><<<parts, s.nt, 0, st>>>(a); break;
        case 2: rms_bwd_regs<E, AL, 2><<<parts, s.nt, 0, st>>>(a); break;
        case 4: rms_bwd_regs<E, AL, 4><<<parts, s.nt, 0, st>>>(a); break;
        default: rms_bwd_regs<E, AL, LONG><<<parts, s.nt, 0, st>>>(a); break;
    }
    return true;
}

template <typename E>
hipError_t bwd_typed(BwdArgs a, float* dw, hipStream_t st) {
    constexpr int N = Pack<E>::N;
    const int parts = bwd_parts(a.rows);
    if (a.rows > 0) {
        const bool vec = a.d % N == 0 && aligned_to(a.dy, 16) && aligned_to(a.h, 16) && aligned_to(a.w, 16) &&
                         aligned_to(a.dh, 16) && aligned_to(a.dx, 16);
        if (!(vec ? launch_bwd_regs<E, true>(a, parts, st) : launch_bwd_regs<E, false>(a, parts, st))) {
            // the columns first: dx may be written over dy or dh
            if (a.part) {
                rms_dw_cols<E><<<dim3((unsigned)((a.d + 255) / 256), (unsigned)parts), 256, 0, st>>>(a);
                const hipError_t e = hipGetLastError();
                if (e != hipSuccess) return e;
            }
            for (a.row0 = 0; a.row0 < a.rows; a.row0 += kRowsPerLaunch) {
                const int64_t left = a.rows - a.row0;
                rms_bwd_long<E><<<(unsigned)(left < kRowsPerLaunch ? left : kRowsPerLaunch), 1024, 0, st>>>(a);
                const hipError_t e = hipGetLastError();
                if (e != hipSuccess) return e;
            }
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dw) {
        const int64_t g = (a.d + kDwCols - 1) / kDwCols;
        const unsigned grid = (unsigned)(g < 65536 ? g : 65536);
        const int n = a.rows > 0 ? parts : 0;
        if (a.d % 4 == 0)   // the workspace is 256-byte aligned
            dw_finalize<4><<<grid, 256, 0, st>>>(a.part, n, a.d, dw);
        else
            dw_finalize<1><<<grid, 256, 0, st>>>(a.part, n, a.d, dw);
    }
    return hipGetLastError();
}

template <typename E>
hipError_t dequantize_typed(const int8_t* q, const float* scale, int64_t rows, int64_t d, void* out, hipStream_t st) {
    constexpr int N = Pack<E>::N;
    const bool vec = d % N == 0 && aligned_to(q, N) && aligned_to(out, 16);
    int64_t gx = ((d + N - 1) / N + 255) / 256;
    if (gx > 64) gx = 64;
    const dim3 grid((unsigned)gx, (unsigned)(rows < 65535 ? rows : 65535));
    if (vec)
        dequantize<E, true><<<grid, 256, 0, st>>>(q, scale, rows, d, static_cast<E*>(out));
    else
        dequantize<E, false><<<grid, 256, 0, st>>>(q, scale, rows, d, static_cast<E*>(out));
    return hipGetLastError();
}

}  // namespace

size_t rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t d) {
    return align_up((size_t)bwd_parts(rows) * (size_t)d * sizeof(float), 256);
}

hipError_t launch_rmsnorm(const void* x, const void* res, const void* w, float eps, int64_t rows, int64_t d, int dtype,
                          void* h, void* y, int8_t* q, float* scale, float* rstd, hipStream_t stream) {
    if (rows == 0) return hipSuccess;
    const RowArgs a{x, res, w, 0, rows, d, eps, h, y, q, scale, rstd};
    switch (dtype) {
        case kF32: return norm_typed<float>(a, stream);
        case kBF16: return norm_typed<bf16_t>(a, stream);
        default: return norm_typed<f16_t>(a, stream);
    }
}

hipError_t launch_rmsnorm_bwd(const void* dy, const void* h, const void* w, const float* rstd, const void* dh,
                              int64_t rows, int64_t d, int dtype, void* dx, float* dw, void* workspace,
                              hipStream_t stream) {
    const BwdArgs a{dy, h, w, rstd, dh, 0, rows, d, dx, dw ? static_cast<float*>(workspace) : nullptr};
    switch (dtype) {
        case kF32: return bwd_typed<float>(a, dw, stream);
        case kBF16: return bwd_typed<bf16_t>(a, dw, stream);
        default: return bwd_typed<f16_t>(a, dw, stream);
    }
}

hipError_t launch_quantize_rows(const void* x, const float* col_scale, int64_t rows, int64_t d, int dtype, int8_t* q,
                                float* scale, hipStream_t stream) {
    if (rows == 0) return hipSuccess;
    const RowArgs a{x, nullptr, col_scale, 0, rows, d, 0.0f, nullptr, nullptr, q, scale, nullptr};
    switch (dtype) {
        case kF32: return quantize_typed<float>(a, stream);
        case kBF16: return quantize_typed<bf16_t>(a, stream);
        default: return quantize_typed<f16_t>(a, stream);
    }
}

hipError_t launch_dequantize_rows(const int8_t* q, const float* scale, int64_t rows, int64_t d, int dtype, void* out,
                                  hipStream_t stream) {
    if (rows == 0) return hipSuccess;
    switch (dtype) {
        case kF32: return dequantize_typed<float>(q, scale, rows, d, out, stream);
        case kBF16: return dequantize_typed<bf16_t>(q, scale, rows, d, out, stream);
        default: return dequantize_typed<f16_t>(q, scale, rows, d, out, stream);
    }
}

}  // namespace dora
