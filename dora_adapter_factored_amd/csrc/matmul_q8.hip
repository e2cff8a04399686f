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
#include <type_traits>

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
// Scales or bias that are not given are ones or zeros, which change nothing.
struct Channel {   // what a channel brings
    float ws, gm1, gs, bias;
};

// Channels n .. n + C - 1, those past the end repeating the last one.
template <int C>
__device__ __forceinline__ void load_channels(const MatmulQ8& a, int64_t n, Channel (&c)[C]) {
    const int64_t left = a.N - 1 - n;
    auto at = [&](int j) __attribute__((always_inline)) { return n + (j < left ? j : left); };
#pragma unroll
    for (int j = 0; j < C; ++j) c[j] = {1.0f, 0.0f, 0.0f, 0.0f};
    if (a.ws) {
#pragma unroll
        for (int j = 0; j < C; ++j) c[j].ws = a.ws[at(j)];
    }
    if (a.g) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const float g = a.g[at(j)];
            c[j].gm1 = g - 1.0f;
            c[j].gs = g * a.s;
        }
    }
    if (a.bias) {
#pragma unroll
        for (int j = 0; j < C; ++j) c[j].bias = a.bias[at(j)];
    }
}

template <bool ADAPTER>
__device__ __forceinline__ float finish(int acc, float xs, const Channel& c, float lora) {
#pragma clang fp contract(off)
    float v = ((float)acc * xs) * c.ws;
    if (ADAPTER) v = v + fmaf(c.gm1, v, c.gs * lora);
    return v + c.bias;
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
        Channel cc[1];
        load_channels(a, n, cc);
        const float r = a.g ? finish<true>(v, a.xs[t], cc[0], Cvt<E>::to_f(static_cast<const E*>(a.lora)[t * a.N + n]))
                            : finish<false>(v, a.xs[t], cc[0], 0.0f);
        static_cast<E*>(a.y)[t * a.N + n] = Cvt<E>::from_f(r);
    }
}

// ------------------------------------------------------------- tiles through LDS

constexpr int kNumXCD = 8;

// BM tokens x BN channels per workgroup, k-tiles of 128 codes (whole 128-byte
// rows) of both operands in a two-stage LDS ring, filled by LDS DMA.
//
// Rows of an LDS tile keep their order; a 16-row MFMA block b of a 64-row
// group takes rows 16 (r / 4) + 4 b + r % 4, r = 0..15.  Lane l's results of
// the group's four channel blocks are then the 16 consecutive channels 16 (l /
// 16) + 0..15 of one token, so that results go from registers to memory in
// runs of 64 channels per token, without a pass through LDS.
//
// Row r's chunk c (16 bytes) is kept in slot c ^ swz(r), swz(r) = the bits
// (r0 ^ r5, r1, r4): the 16 rows of a fragment read then fill all slots of even
// and of odd rows, free of bank conflicts.
template <int BM_, int BN_, int WT_, int WC_>
struct Q8Tile {
    static constexpr int BM = BM_, BN = BN_;       // tokens, channels
    static constexpr int WT = WT_, WC = WC_;       // waves along each
    static constexpr int NW = WT * WC, NTH = NW * 64;
    static constexpr int MT = BM / WT / 16, NC = BN / WC / 16;   // 16-row blocks per wave
    static constexpr int XBYTES = BM * 128, WBYTES = BN * 128;
    static constexpr int STAGE = XBYTES + WBYTES;
    static constexpr int XG = BM / 8 / NW, WG = BN / 8 / NW;     // DMA instructions (8 rows) per wave and tile
    static_assert(MT % 4 == 0 && NC % 4 == 0, "whole 64-row groups per wave");
    static_assert(NW % 8 == 0, "a wave's DMA groups share their swizzle");
    static_assert(BM / 8 % NW == 0 && BN / 8 % NW == 0, "DMA groups split evenly across waves");
};

__device__ __forceinline__ int swz_tile(int row) {
    return ((row ^ (row >> 5)) & 1) | (row & 2) | (((row >> 4) & 1) << 2);
}

struct TileGrid {
    int tm, tn;   // tiles along the tokens and the channels
};

// Workgroup id -> tile.  Ids go round the XCDs, so XCD x takes the x-th
// contiguous part of the tile order, in which kGroupM token tiles share a
// channel tile before the next one: the tiles an XCD works on at one time are
// a block, whose operands' rows meet in its L2.
constexpr int kGroupM = 8;

__device__ __forceinline__ void tile_of(int id, const TileGrid& g, int& m, int& n) {
    const int total = g.tm * g.tn, q = total / kNumXCD, r = total % kNumXCD;
    const int x = id % kNumXCD;
    const int i = x * q + (x < r ? x : r) + id / kNumXCD;
    const int per = kGroupM * g.tn, grp = i / per, rest = i % per;
    const int h = g.tm - grp * kGroupM < kGroupM ? g.tm - grp * kGroupM : kGroupM;
    m = grp * kGroupM + rest % h;
    n = rest / h;
}

template <typename E, typename G, bool VEC>
__global__ __launch_bounds__(G::NTH, 1) void q8_tiles(MatmulQ8 a, TileGrid grid) {
    __shared__ __attribute__((aligned(1024))) char smem[2 * G::STAGE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wt = wave / G::WC, wc = wave % G::WC;
    int tm, tn;
    tile_of(blockIdx.x, grid, tm, tn);
    const int64_t t0 = (int64_t)tm * G::BM, n0 = (int64_t)tn * G::BN;
    const int K = (int)a.K;
    const int nk = (K + 127) / 128;

    // DMA: lane l moves slot l % 8 of row l / 8 of an 8-row group; the wave's
    // groups are wave, wave + NW, ...  Rows past the end repeat the last one
    // (their results are not stored); chunks past K read zeros.
    const int chunk = ((lane & 7) ^ swz_tile(wave * 8 + (lane >> 3))) * 16;
    int xoff[G::XG], woff[G::WG];
#pragma unroll
    for (int i = 0; i < G::XG; ++i) {
        const int r = (wave + i * G::NW) * 8 + (lane >> 3);
        xoff[i] = (int)(t0 + r < a.T ? r : a.T - 1 - t0) * K + chunk;
    }
#pragma unroll
    for (int i = 0; i < G::WG; ++i) {
        const int r = (wave + i * G::NW) * 8 + (lane >> 3);
        woff[i] = (int)(n0 + r < a.N ? r : a.N - 1 - n0) * K + chunk;
    }
    auto resource = [](const void* p) __attribute__((always_inline)) {
        const uint64_t v = reinterpret_cast<uint64_t>(p);
        i32x4_t rs;
        rs[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
        rs[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
        rs[2] = 0x7fffffff;
        rs[3] = kRsrcWord3;
        return rs;
    };
    const i32x4_t xr = resource(a.xq + t0 * K), wr = resource(a.wq + n0 * K);
    auto issue = [&](int kt) __attribute__((always_inline)) {
        // past the last k-tile: zeros, into a stage that no one reads
        const bool in = kt * 128 + chunk < K;
        char* dst = smem + (kt & 1) * G::STAGE + wave * 1024;
#pragma unroll
        for (int i = 0; i < G::XG; ++i)
            raw_buffer_load_lds(xr, (lds_void_t*)(dst + i * G::NW * 1024), 16, in ? xoff[i] : kOutOfRange, kt * 128, 0, 0);
#pragma unroll
        for (int i = 0; i < G::WG; ++i)
            raw_buffer_load_lds(wr, (lds_void_t*)(dst + G::XBYTES + i * G::NW * 1024), 16, in ? woff[i] : kOutOfRange,
                                kt * 128, 0, 0);
    };

    // fragments: lane l reads row 16 ((l % 16) / 4) + l % 4 of a group (+ 4 b
    // for block b), chunk 4 ks + l / 16
    const int fr = ((lane & 12) << 2) | (lane & 3), fs = swz_tile(fr);
    const int fo = fr * 128 + (((lane >> 4) ^ fs) << 4);   // ks = 0; ks = 1 is fo ^ 64
    const int xbase = wt * G::MT * 16 * 128, wbase = G::XBYTES + wc * G::NC * 16 * 128;
    i32x4_t acc[G::MT][G::NC];
#pragma unroll
    for (int m = 0; m < G::MT; ++m)
#pragma unroll
        for (int c = 0; c < G::NC; ++c) acc[m][c] = {0, 0, 0, 0};

    auto read = [&](int kt, int ks, i32x4_t (&x)[G::MT], i32x4_t (&w)[G::NC]) __attribute__((always_inline)) {
        const char* st = smem + (kt & 1) * G::STAGE + (fo ^ (ks * 64));
#pragma unroll
        for (int c = 0; c < G::NC; ++c)
            w[c] = *reinterpret_cast<const i32x4_t*>(st + wbase + (c / 4) * 64 * 128 + (c % 4) * 4 * 128);
#pragma unroll
        for (int m = 0; m < G::MT; ++m)
            x[m] = *reinterpret_cast<const i32x4_t*>(st + xbase + (m / 4) * 64 * 128 + (m % 4) * 4 * 128);
    };
    auto mma = [&](const i32x4_t (&x)[G::MT], const i32x4_t (&w)[G::NC]) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < G::MT; ++m)
#pragma unroll
            for (int c = 0; c < G::NC; ++c) acc[m][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[c], x[m], acc[m][c], 0, 0, 0);
    };
    // one read for every two MFMAs, so that the reads run under the matrix pipe
    auto interleave = []() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < G::MT + G::NC; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);   // MFMA
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
        }
        __builtin_amdgcn_sched_group_barrier(0x008, G::MT * G::NC, 0);
        __builtin_amdgcn_sched_barrier(0);
    };

    // A k-tile is two steps of 64 codes.  While one step's MFMAs run the next
    // step's fragments are read.  Between them, once per tile: this wave's DMA
    // of the next tile has landed and its reads of this tile are done; barrier;
    // then the tile after the next is enqueued into this tile's stage.
    i32x4_t x0[G::MT], w0[G::NC], x1[G::MT], w1[G::NC];
    issue(0);
    issue(1);
    wait_vmcnt<G::XG + G::WG>();
    __builtin_amdgcn_s_barrier();
    read(0, 0, x0, w0);
    for (int kt = 0; kt < nk; ++kt) {
        read(kt, 1, x1, w1);
        mma(x0, w0);
        interleave();
        wait_vmcnt<0>();
        wait_lgkmcnt0();
        __builtin_amdgcn_s_barrier();
        issue(kt + 2);
        read(kt + 1, 0, x0, w0);   // past the last tile: zeros or an old tile, unused
        mma(x1, w1);
        interleave();
    }
    wait_vmcnt<0>();

    // epilogue: token block m of the wave, channels ch .. ch + 15 per lane
    auto epilogue = [&](auto adapter) __attribute__((always_inline)) {
        constexpr bool ADAPTER = decltype(adapter)::value;
        constexpr int P = VEC ? Pack<E>::N : 1;
#pragma unroll
        for (int cg = 0; cg < G::NC / 4; ++cg) {
            const int64_t ch = n0 + (wc * G::NC + cg * 4) * 16 + (lane >> 4) * 16;
            if (ch >= a.N) continue;
            Channel cc[16];
            load_channels(a, ch, cc);
#pragma unroll
            for (int m = 0; m < G::MT; ++m) {
                const int r = lane & 15;
                const int64_t t = t0 + (wt * G::MT + (m & ~3)) * 16 + (r >> 2) * 16 + (m & 3) * 4 + (r & 3);
                if (t >= a.T) continue;
                const float xs = a.xs[t];
                const int64_t at = t * a.N + ch;
#pragma unroll
                for (int h = 0; h < 16; h += P) {
                    if (ch + h >= a.N) continue;
                    if (VEC) {
                        Pack<E> l, o;
                        if (ADAPTER) l = load_pack(static_cast<const E*>(a.lora) + at + h);
#pragma unroll
                        for (int e = 0; e < P; ++e)
                            o.e[e] = Cvt<E>::from_f(finish<ADAPTER>(acc[m][cg * 4 + (h + e) / 4][(h + e) % 4], xs, cc[h + e],
                                                                    ADAPTER ? Cvt<E>::to_f(l.e[e]) : 0.0f));
                        *reinterpret_cast<u32x4_t*>(static_cast<E*>(a.y) + at + h) = o.u;
                    } else {
                        const float l = ADAPTER ? Cvt<E>::to_f(static_cast<const E*>(a.lora)[at + h]) : 0.0f;
                        static_cast<E*>(a.y)[at + h] =
                            Cvt<E>::from_f(finish<ADAPTER>(acc[m][cg * 4 + h / 4][h % 4], xs, cc[h], l));
                    }
                }
            }
        }
    };
    if (a.g)
        epilogue(std::true_type{});
    else
        epilogue(std::false_type{});
}

// ------------------------------------------------------------- launches

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename E, typename G>
hipError_t launch_tiles(const MatmulQ8& a, hipStream_t st) {
    const TileGrid g{(int)((a.T + G::BM - 1) / G::BM), (int)((a.N + G::BN - 1) / G::BN)};
    const bool vec = a.N % Pack<E>::N == 0 && aligned16(a.y) && aligned16(a.lora);
    auto k = vec ? q8_tiles<E, G, true> : q8_tiles<E, G, false>;
    k<<<(unsigned)(g.tm * g.tn), G::NTH, 0, st>>>(a, g);
    return hipGetLastError();
}

template <typename E>
hipError_t launch_direct(MatmulQ8 a, hipStream_t st) {
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

template <typename E>
hipError_t launch_typed(const MatmulQ8& a, hipStream_t st) {
    const bool dma = a.K % 16 == 0 && aligned16(a.xq) && aligned16(a.wq);
    if (a.T > 64 && dma) return launch_tiles<E, Q8Tile<256, 256, 2, 4>>(a, st);
    return launch_direct<E>(a, st);
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
