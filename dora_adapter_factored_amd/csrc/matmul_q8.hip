// Matrix product in 8-bit integers with a scale for each token and channel,
// for gfx950, with the DoRA composition in its epilogue.
//
//   acc_tn  = sum_k xq_tk wq_nk                    exact, int32
//   base_tn = acc_tn xs_t ws_n
//   y_tn    = base + (g_n - 1) base + (g_n s) lora_tn + bias_n   (terms as given)
// in fp32 after the sum, rounded once to y's type.
//
// Codes go through v_mfma_i32_16x16x64_i8.  The channels are the A operand
// and the tokens the B operand, so a lane's four results are four channels of
// one token.  Both operands use one map from lanes and registers to k, so any
// permutation of k inside an instruction is as good as another: the kernels
// choose the one whose loads are widest.
#include "dora_device.h"
#include "dora_gfx950.h"
#include "dora_launch.h"

namespace dora {
namespace {

constexpr int kWaves = 8;

// 16 bytes from any address.
__device__ __forceinline__ i32x4_t load16(const int8_t* p) {
    i32x4_t v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// The first `left` of 16 bytes, zeros after them.
__device__ __forceinline__ i32x4_t load16_tail(const int8_t* p, int64_t left) {
    if (left >= 16) return load16(p);
    i32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int b = 0; b < 16; ++b)
        if (b < left) v[b / 4] |= (int)(uint8_t)p[b] << (8 * (b % 4));
    return v;
}

// One result: its scales, the composition, the bias.  Contraction is off so
// that every form of the kernel rounds alike: with the sum exact, a token's
// result is then bitwise the same whatever batch it is in.
template <typename E>
__device__ __forceinline__ E finish(const MatmulQ8& a, int acc, int64_t t, int64_t n) {
#pragma clang fp contract(off)
    float v = (float)acc * a.xs[t];
    if (a.ws) v *= a.ws[n];
    if (a.g) {
        const float g = a.g[n];
        v += fmaf(g - 1.0f, v, (g * a.s) * Cvt<E>::to_f(static_cast<const E*>(a.lora)[t * a.N + n]));
    }
    if (a.bias) v += a.bias[n];
    return Cvt<E>::from_f(v);
}

// 16 channels x 16 C tokens per workgroup, the waves taking 128-byte columns
// of K in turn straight from memory into the MFMA operands; the waves' sums
// are added through LDS.
template <typename E, int C>
__global__ __launch_bounds__(kWaves * 64) void q8_direct(MatmulQ8 a) {
    __shared__ int red[kWaves][C][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * 16 * C;
    // rows past the end repeat the last one; their results are not stored
    const int64_t nr = n0 + (lane & 15) < a.N ? n0 + (lane & 15) : a.N - 1;
    const int kl = (lane >> 4) * 32;
    const int8_t* wp = a.wq + nr * a.K + kl;
    const int8_t* xp[C];
    i32x4_t acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t t = t0 + c * 16 + (lane & 15);
        xp[c] = a.xq + (t < a.T ? t : a.T - 1) * a.K + kl;
        acc[c] = {0, 0, 0, 0};
    }
    const int64_t full = a.K / 128;
    for (int64_t kb = wave; kb < full; kb += kWaves) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const i32x4_t w = load16(wp + kb * 128 + j * 16);
#pragma unroll
            for (int c = 0; c < C; ++c)
                acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, load16(xp[c] + kb * 128 + j * 16), acc[c], 0, 0, 0);
        }
    }
    if (full % kWaves == wave && full * 128 < a.K) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t k = full * 128 + j * 16, left = a.K - k - kl;
            const i32x4_t w = load16_tail(wp + k, left);
#pragma unroll
            for (int c = 0; c < C; ++c)
                acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, load16_tail(xp[c] + k, left), acc[c], 0, 0, 0);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) *reinterpret_cast<i32x4_t*>(&red[wave][c][lane * 4]) = acc[c];
    __syncthreads();
    for (int o = threadIdx.x; o < C * 256; o += kWaves * 64) {
        const int c = o >> 8, tok = (o >> 4) & 15, ch = o & 15;
        const int64_t t = t0 + c * 16 + tok, n = n0 + ch;
        if (t >= a.T || n >= a.N) continue;
        const int src = ((ch >> 2) * 16 + tok) * 4 + (ch & 3);
        int v = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += red[w][c][src];
        static_cast<E*>(a.y)[t * a.N + n] = finish<E>(a, v, t, n);
    }
}

template <typename E>
hipError_t launch_typed(MatmulQ8 a, hipStream_t st) {
    const unsigned gx = (unsigned)((a.N + 15) / 16);
    constexpr int64_t kMaxTokens = (int64_t)65535 * 16;   // of one launch: a grid's rows
    const MatmulQ8 all = a;
    for (int64_t t = 0; t < all.T; t += kMaxTokens) {
        a.T = all.T - t < kMaxTokens ? all.T - t : kMaxTokens;
        a.xq = all.xq + t * all.K;
        a.xs = all.xs + t;
        a.lora = all.lora ? static_cast<const E*>(all.lora) + t * all.N : nullptr;
        a.y = static_cast<E*>(all.y) + t * all.N;
        if (a.T <= 16)
            q8_direct<E, 1><<<dim3(gx, 1), kWaves * 64, 0, st>>>(a);
        else
            q8_direct<E, 4><<<dim3(gx, (unsigned)((a.T + 63) / 64)), kWaves * 64, 0, st>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t matmul_q8_workspace_bytes(int64_t T, int64_t N, int64_t K) { return 0; }

hipError_t launch_matmul_q8(const MatmulQ8& a, int dtype, void* workspace, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    switch (dtype) {
        case kF32: return launch_typed<float>(a, stream);
        case kBF16: return launch_typed<bf16_t>(a, stream);
        default: return launch_typed<f16_t>(a, stream);
    }
}

}  // namespace dora
