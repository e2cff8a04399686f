// Row operators in front of an 8-bit product, for gfx950: root-mean-square
// norm with the residual's addition (forward, with an 8-bit output, and
// backward), rows to 8 bits with a scale each, and back.
//
// Forward, row t of [T, d], all in fp32, each output rounded once:
//   h = x + residual,  rstd = 1 / sqrt(mean_j h_j^2 + eps),  y = h rstd w
//   scale = max_j |y_j| / 127,  q_j = rint(y_j / scale)
// rstd cancels in q: with p = h w and a = max_j |p_j|, q_j = rint(p_j 127 / a)
// and scale = a rstd / 127, so the codes need one maximum over products that
// are at hand in the same pass as the sum of squares, and the row is read
// once.  Rows to 8 bits are the same with rstd = 1 and w the column scale.
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
// twice, the second time from cache.
#include "dora_device.h"
#include "dora_launch.h"

namespace dora {
namespace {

constexpr int kMaxWaves = 16;
constexpr uint32_t kInfBits = 0x7f800000u;
// Rows whose largest value is below 2^-119 quantise to zeros with scale 0:
// 127 / a would leave the fp32 range there.  The error is below 2^-119.
constexpr uint32_t kTinyBits = (uint32_t)(127 - 119) << 23;

// N consecutive elements in one access (16 bytes, or one element where rows
// or pointers are not 16-byte aligned), kept as loaded.
template <typename E, int N> struct Elems {
    Pack<E> k;
    __device__ __forceinline__ void load(const E* p) { k = load_pack(p); }
    __device__ __forceinline__ float operator[](int e) const { return Cvt<E>::to_f(k.e[e]); }
};
template <typename E> struct Elems<E, 1> {
    E k;
    __device__ __forceinline__ void load(const E* p) { k = *p; }
    __device__ __forceinline__ float operator[](int) const { return Cvt<E>::to_f(k); }
};

template <typename E, int N>
__device__ __forceinline__ void store_n(E* p, const float (&v)[N]) {
    if constexpr (N == 1) {
        *p = Cvt<E>::from_f(v[0]);
    } else {
        Pack<E> k;
#pragma unroll
        for (int e = 0; e < N; ++e) k.e[e] = Cvt<E>::from_f(v[e]);
        store_pack_stream(p, k);
    }
}

// N column scales / weights as fp32.
template <typename W, int N>
__device__ __forceinline__ void load_w(const W* w, int64_t col, float (&v)[N]) {
    constexpr int M = N * sizeof(W) > 16 ? 4 : N;   // fp32 scales beside 16-bit elements take two accesses
#pragma unroll
    for (int h = 0; h < N; h += M) {
        Elems<W, M> t;
        t.load(w + col + h);
#pragma unroll
        for (int e = 0; e < M; ++e) v[h + e] = t[e];
    }
}

// N codes: rint(p inv) packed into bytes.  |p inv| <= 127 up to one rounding,
// which rint takes back to 127.
template <int N>
__device__ __forceinline__ void store_codes(int8_t* q, const float (&p)[N], float inv) {
    int c[N];
#pragma unroll
    for (int e = 0; e < N; ++e) c[e] = (int)rintf(p[e] * inv);
    if constexpr (N == 1) {
        q[0] = (int8_t)c[0];
    } else {
        uint32_t u[N / 4];
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            u[i] = (c[4 * i] & 255) | (c[4 * i + 1] & 255) << 8 | (c[4 * i + 2] & 255) << 16 | (uint32_t)c[4 * i + 3] << 24;
        if constexpr (N == 4) {
            *reinterpret_cast<uint32_t*>(q) = u[0];
        } else {
            *reinterpret_cast<uint2*>(q) = make_uint2(u[0], u[1]);
        }
    }
}

// (sum, maximum) over the workgroup, returned to every thread.  Sums are
// added in a fixed order.  red holds kMaxWaves entries of each and is free to
// be written again after the next barrier.
__device__ __forceinline__ void block_reduce(float& sum, uint32_t& top, float* rs, uint32_t* rt) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        sum += __shfl_xor(sum, o);
        const uint32_t t = __shfl_xor(top, o);
        top = t > top ? t : top;
    }
    const int nw = blockDim.x >> 6;
    if (nw == 1) return;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
        rs[w] = sum;
        rt[w] = top;
    }
    __syncthreads();
    sum = rs[0];
    top = rt[0];
    for (int i = 1; i < nw; ++i) {
        sum += rs[i];
        top = rt[i] > top ? rt[i] : top;
    }
}

// What a row's codes need: the factor of p, and the row's scale.  A row that
// holds a NaN or an infinity has scale NaN and codes 0, so all that comes of
// it is NaN.
__device__ __forceinline__ void code_scale(uint32_t top, float rstd, float& inv, float& scale) {
    const float a = __uint_as_float(top);
    const bool tiny = top < kTinyBits, bad = top >= kInfBits;
    inv = tiny || bad ? 0.0f : 127.0f / a;
    scale = bad ? __uint_as_float(0x7fc00000u) : tiny ? 0.0f : a * rstd / 127.0f;
}

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

// Codes of a row with a NaN or infinity: 0 whatever p is (NaN * 0 is NaN, and
// a NaN's conversion to an integer is not to be relied on).
template <int N>
__device__ __forceinline__ void zero_unless(bool keep, float (&p)[N]) {
    if (keep) return;
#pragma unroll
    for (int e = 0; e < N; ++e) p[e] = 0.0f;
}

// One row per workgroup, the row in registers.  NORM: the norm (w of type E,
// outputs h, y, q, rstd as asked); otherwise rows to 8 bits (w an optional
// fp32 column scale).
template <typename E, typename W, int N, int P, bool NORM>
__global__ __launch_bounds__(P > 2 ? 512 : 1024) void row_regs(RowArgs a) {
    __shared__ float rs[kMaxWaves];
    __shared__ uint32_t rt[kMaxWaves];
    const int64_t row = a.row0 + blockIdx.x, off = row * a.d;
    const E* x = static_cast<const E*>(a.x) + off;
    const W* w = static_cast<const W*>(a.w);
    const int n = (int)(a.d / N), nt = blockDim.x;
    float v[P][N], p[P][N];
    {
        Elems<E, N> xv[P], rv[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
            if (k < n) {
                xv[i].load(x + (int64_t)k * N);
                if (NORM && a.res) rv[i].load(static_cast<const E*>(a.res) + off + (int64_t)k * N);
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                v[i][e] = k < n ? xv[i][e] : 0.0f;
                if (NORM && a.res) v[i][e] += k < n ? rv[i][e] : 0.0f;
            }
        }
    }
    float sum = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int k = threadIdx.x + i * nt;
        float wv[N];
#pragma unroll
        for (int e = 0; e < N; ++e) wv[e] = 1.0f;
        if (k < n && w) load_w<W, N>(w, (int64_t)k * N, wv);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (NORM) sum = fmaf(v[i][e], v[i][e], sum);
            p[i][e] = k < n ? v[i][e] * wv[e] : 0.0f;
            const uint32_t m = __float_as_uint(p[i][e]) & 0x7fffffffu;
            top = m > top ? m : top;
        }
        if (NORM && a.h && k < n) store_n<E, N>(static_cast<E*>(a.h) + off + (int64_t)k * N, v[i]);
    }
    block_reduce(sum, top, rs, rt);
    const float rstd = NORM ? 1.0f / sqrtf(sum / (float)a.d + a.eps) : 1.0f;
    float inv, scale;
    code_scale(top, rstd, inv, scale);
    if (threadIdx.x == 0) {
        if (NORM && a.rstd) a.rstd[row] = rstd;
        if (a.q) a.scale[row] = scale;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int k = threadIdx.x + i * nt;
        if (k >= n) continue;
        if (NORM && a.y) {
            float yv[N];
#pragma unroll
            for (int e = 0; e < N; ++e) yv[e] = p[i][e] * rstd;
            store_n<E, N>(static_cast<E*>(a.y) + off + (int64_t)k * N, yv);
        }
        if (a.q) {
            zero_unless<N>(inv != 0.0f, p[i]);
            store_codes<N>(a.q + off + (int64_t)k * N, p[i], inv);
        }
    }
}

// The same for rows of any length, read twice.
template <typename E, typename W, int N, bool NORM>
__global__ __launch_bounds__(1024) void row_long(RowArgs a) {
    __shared__ float rs[kMaxWaves];
    __shared__ uint32_t rt[kMaxWaves];
    const int64_t row = a.row0 + blockIdx.x, off = row * a.d, n = a.d / N;
    const E* x = static_cast<const E*>(a.x) + off;
    const E* r = NORM && a.res ? static_cast<const E*>(a.res) + off : nullptr;
    const W* w = static_cast<const W*>(a.w);
    auto at = [&](int64_t k, float (&v)[N], float (&p)[N]) __attribute__((always_inline)) {
        Elems<E, N> t;
        t.load(x + k * N);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = t[e];
        if (r) {
            t.load(r + k * N);
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] += t[e];
        }
#pragma unroll
        for (int e = 0; e < N; ++e) p[e] = 1.0f;
        if (w) load_w<W, N>(w, k * N, p);
#pragma unroll
        for (int e = 0; e < N; ++e) p[e] *= v[e];
    };
    float sum = 0.0f;
    uint32_t top = 0;
    for (int64_t k = threadIdx.x; k < n; k += blockDim.x) {
        float v[N], p[N];
        at(k, v, p);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (NORM) sum = fmaf(v[e], v[e], sum);
            const uint32_t m = __float_as_uint(p[e]) & 0x7fffffffu;
            top = m > top ? m : top;
        }
    }
    block_reduce(sum, top, rs, rt);
    const float rstd = NORM ? 1.0f / sqrtf(sum / (float)a.d + a.eps) : 1.0f;
    float inv, scale;
    code_scale(top, rstd, inv, scale);
    if (threadIdx.x == 0) {
        if (NORM && a.rstd) a.rstd[row] = rstd;
        if (a.q) a.scale[row] = scale;
    }
    // each element is read by the thread that writes it, so h may be x or the
    // residual itself
    for (int64_t k = threadIdx.x; k < n; k += blockDim.x) {
        float v[N], p[N];
        at(k, v, p);
        if (NORM && a.h) store_n<E, N>(static_cast<E*>(a.h) + off + k * N, v);
        if (NORM && a.y) {
            float yv[N];
#pragma unroll
            for (int e = 0; e < N; ++e) yv[e] = p[e] * rstd;
            store_n<E, N>(static_cast<E*>(a.y) + off + k * N, yv);
        }
        if (a.q) {
            zero_unless<N>(inv != 0.0f, p);
            store_codes<N>(a.q + off + k * N, p, inv);
        }
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
// registers between its reduction and its store.
template <typename E, int N, int P>
__global__ __launch_bounds__(P > 2 ? 512 : 1024) void rms_bwd_regs(BwdArgs a) {
    __shared__ float rs[2][kMaxWaves];
    __shared__ uint32_t rt[2][kMaxWaves];
    const int n = (int)(a.d / N), nt = blockDim.x;
    Elems<E, N> wv[P];
    float dw[P][N];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int k = threadIdx.x + i * nt;
#pragma unroll
        for (int e = 0; e < N; ++e) dw[i][e] = 0.0f;
        if (k < n) wv[i].load(static_cast<const E*>(a.w) + (int64_t)k * N);
    }
    int par = 0;   // the reduction's buffer: the other one than the last row's, which slow waves may still read
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, par ^= 1) {
        const int64_t off = row * a.d;
        Elems<E, N> dyv[P], hv[P], gv[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
            if (k < n) {
                dyv[i].load(static_cast<const E*>(a.dy) + off + (int64_t)k * N);
                hv[i].load(static_cast<const E*>(a.h) + off + (int64_t)k * N);
                if (a.dh) gv[i].load(static_cast<const E*>(a.dh) + off + (int64_t)k * N);
            }
        }
        const float r = a.rstd[row];
        float c = 0.0f;
        uint32_t none = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (threadIdx.x + i * nt >= n) continue;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float dv = dyv[i][e], hh = hv[i][e];
                c = fmaf(dv * wv[i][e], hh, c);
                dw[i][e] = fmaf(dv, hh * r, dw[i][e]);
            }
        }
        block_reduce(c, none, rs[par], rt[par]);
        const float f = c / (float)a.d * r * r;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
            if (k >= n) continue;
            float o[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float u = dyv[i][e] * wv[i][e];
                o[e] = r * (u - hv[i][e] * f) + (a.dh ? gv[i][e] : 0.0f);
            }
            store_n<E, N>(static_cast<E*>(a.dx) + off + (int64_t)k * N, o);
        }
    }
    if (a.part) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int k = threadIdx.x + i * nt;
            if (k >= n) continue;
            float* dst = a.part + (int64_t)blockIdx.x * a.d + (int64_t)k * N;
#pragma unroll
            for (int e = 0; e < N; ++e) dst[e] = dw[i][e];
        }
    }
}

// Rows of any length: dx with the row read twice, and dw's partials by
// columns.
template <typename E>
__global__ __launch_bounds__(1024) void rms_bwd_long(BwdArgs a) {
    __shared__ float rs[kMaxWaves];
    __shared__ uint32_t rt[kMaxWaves];
    const int64_t row = a.row0 + blockIdx.x, off = row * a.d;
    const E* dy = static_cast<const E*>(a.dy) + off;
    const E* h = static_cast<const E*>(a.h) + off;
    const E* dh = a.dh ? static_cast<const E*>(a.dh) + off : nullptr;
    const E* w = static_cast<const E*>(a.w);
    const float r = a.rstd[row];
    float c = 0.0f;
    uint32_t none = 0;
    for (int64_t k = threadIdx.x; k < a.d; k += blockDim.x)
        c = fmaf(Cvt<E>::to_f(dy[k]) * Cvt<E>::to_f(w[k]), Cvt<E>::to_f(h[k]), c);
    block_reduce(c, none, rs, rt);
    const float f = c / (float)a.d * r * r;
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
// w + 8, ... in order, then the eight sums in order.
constexpr int kDwCols = 32, kDwLanes = 8;

__global__ __launch_bounds__(256) void dw_finalize(const float* __restrict__ part, int nparts, int64_t d,
                                                   float* __restrict__ dw) {
    __shared__ float red[kDwLanes][kDwCols];
    const int c = threadIdx.x % kDwCols, w = threadIdx.x / kDwCols;
    for (int64_t j0 = (int64_t)blockIdx.x * kDwCols; j0 < d; j0 += (int64_t)gridDim.x * kDwCols) {
        const int64_t j = j0 + c;
        float s = 0.0f;
        if (j < d)
            for (int p = w; p < nparts; p += kDwLanes) s += part[(int64_t)p * d + j];
        red[w][c] = s;
        __syncthreads();
        if (w == 0 && j < d) {
            float v = red[0][c];
#pragma unroll
            for (int q = 1; q < kDwLanes; ++q) v += red[q][c];
            dw[j] = v;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------- dequantise

template <typename E, int N>
__global__ __launch_bounds__(256) void dequantize(const int8_t* __restrict__ q, const float* __restrict__ scale,
                                                  int64_t rows, int64_t d, E* __restrict__ out) {
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const float s = scale[row];
        for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < d / N; k += (int64_t)gridDim.x * 256) {
            float v[N];
            const int8_t* src = q + row * d + k * N;
            int8_t c[N];
            __builtin_memcpy(c, N == 1 ? src : static_cast<const int8_t*>(__builtin_assume_aligned(src, N)), N);
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = (float)c[e] * s;
            store_n<E, N>(out + row * d + k * N, v);
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

RowShape row_shape(int64_t n, int64_t rows) {
    const int64_t most = rows >= kManyRows ? 256 : 1024;
    int p = 1;
    while (p < 8 && n > most * p) p *= 2;
    const int64_t nt = ((n + p - 1) / p + 63) / 64 * 64;
    if (nt > (p > 2 ? 512 : 1024)) {
        if (n > 8 * 512) return {0, 1024};
        return {8, (int)(((n + 7) / 8 + 63) / 64 * 64)};
    }
    return {p, (int)nt};
}

// Rows per launch: a grid's threads are counted in 32 bits.
constexpr int64_t kRowsPerLaunch = (int64_t)1 << 21;

template <typename E, typename W, int N, bool NORM>
hipError_t launch_rows(RowArgs a, hipStream_t st) {
    const RowShape s = row_shape(a.d / N, a.rows);
    for (a.row0 = 0; a.row0 < a.rows; a.row0 += kRowsPerLaunch) {
        const int64_t left = a.rows - a.row0;
        const unsigned g = (unsigned)(left < kRowsPerLaunch ? left : kRowsPerLaunch);
        switch (s.p) {
            case 1: row_regs<E, W, N, 1, NORM><<<g, s.nt, 0, st>>>(a); break;
            case 2: row_regs<E, W, N, 2, NORM><<<g, s.nt, 0, st>>>(a); break;
            case 4: row_regs<E, W, N, 4, NORM><<<g, s.nt, 0, st>>>(a); break;
            case 8: row_regs<E, W, N, 8, NORM><<<g, s.nt, 0, st>>>(a); break;
            default: row_long<E, W, N, NORM><<<g, s.nt, 0, st>>>(a); break;
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
    return vec ? launch_rows<E, E, N, true>(a, st) : launch_rows<E, E, 1, true>(a, st);
}

template <typename E>
hipError_t quantize_typed(const RowArgs& a, hipStream_t st) {
    constexpr int N = Pack<E>::N;
    const bool vec = a.d % N == 0 && aligned_to(a.x, 16) && aligned_to(a.w, 16) && aligned_to(a.q, N);
    return vec ? launch_rows<E, float, N, false>(a, st) : launch_rows<E, float, 1, false>(a, st);
}

// Workgroups of the backward pass, each with its own row of dw partials.
constexpr int kBwdParts = 512;

int bwd_parts(int64_t rows) { return (int)(rows < kBwdParts ? rows : kBwdParts); }

template <typename E, int N>
bool launch_bwd_regs(const BwdArgs& a, int parts, hipStream_t st) {
    const RowShape s = row_shape(a.d / N, a.rows);
    switch (s.p) {
        case 1: rms_bwd_regs<E, N, 1><<<parts, s.nt, 0, st>>>(a); break;
        case 2: rms_bwd_regs<E, N, 2><<<parts, s.nt, 0, st>>>(a); break;
        case 4: rms_bwd_regs<E, N, 4><<<parts, s.nt, 0, st>>>(a); break;
        case 8: rms_bwd_regs<E, N, 8><<<parts, s.nt, 0, st>>>(a); break;
        default: return false;
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
        if (!(vec ? launch_bwd_regs<E, N>(a, parts, st) : launch_bwd_regs<E, 1>(a, parts, st))) {
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
        dw_finalize<<<(unsigned)(g < 65536 ? g : 65536), 256, 0, st>>>(a.part, a.rows > 0 ? parts : 0, a.d, dw);
    }
    return hipGetLastError();
}

template <typename E>
hipError_t dequantize_typed(const int8_t* q, const float* scale, int64_t rows, int64_t d, void* out, hipStream_t st) {
    constexpr int N = Pack<E>::N;
    const bool vec = d % N == 0 && aligned_to(q, N) && aligned_to(out, 16);
    const int64_t n = vec ? d / N : d;
    int64_t gx = (n + 255) / 256;
    if (gx > 64) gx = 64;
    const dim3 grid((unsigned)gx, (unsigned)(rows < 65535 ? rows : 65535));
    if (vec)
        dequantize<E, N><<<grid, 256, 0, st>>>(q, scale, rows, d, static_cast<E*>(out));
    else
        dequantize<E, 1><<<grid, 256, 0, st>>>(q, scale, rows, d, static_cast<E*>(out));
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
