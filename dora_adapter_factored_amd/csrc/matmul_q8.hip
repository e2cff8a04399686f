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

// Bytes k .. k + 15 of a row of K, zeros past its end: the last 16 bytes of
// the row moved down, so that nothing outside the row is read.
__device__ __forceinline__ i32x4_t load16_tail(const int8_t* row, int k, int K) {
    i32x4_t v = {0, 0, 0, 0};
    if (K < 16) {
        for (int b = 0; b < 16; ++b)
            if (k + b < K) v[b / 4] |= (int)(uint8_t)row[k + b] << (8 * (b % 4));
        return v;
    }
    const int at = k < K - 16 ? k : K - 16, skip = 8 * (k - at);   // bits
    const i32x4_t r = load16(row + at);
    uint64_t lo = (uint32_t)r[0] | (uint64_t)(uint32_t)r[1] << 32, hi = (uint32_t)r[2] | (uint64_t)(uint32_t)r[3] << 32;
    if (skip >= 128) lo = hi = 0;
    else if (skip >= 64) lo = hi >> (skip - 64), hi = 0;
    else if (skip > 0) lo = lo >> skip | hi << (64 - skip), hi >>= skip;
    v[0] = (int)(uint32_t)lo;
    v[1] = (int)(uint32_t)(lo >> 32);
    v[2] = (int)(uint32_t)hi;
    v[3] = (int)(uint32_t)(hi >> 32);
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
    const int K = (int)a.K;
    const int8_t* wp = a.wq + nr * K;
    const int8_t* xp[C];
    i32x4_t acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t t = t0 + c * 16 + (lane & 15);
        xp[c] = a.xq + (t < a.T ? t : a.T - 1) * K;
        acc[c] = {0, 0, 0, 0};
    }
    const int full = K / 128;
    for (int kb = wave; kb < full; kb += kWaves) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = kb * 128 + kl + j * 16;
            const i32x4_t w = load16(wp + k);
#pragma unroll
            for (int c = 0; c < C; ++c)
                acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, load16(xp[c] + k), acc[c], 0, 0, 0);
        }
    }
    if (full % kWaves == wave && full * 128 < K) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = full * 128 + kl + j * 16;
            const i32x4_t w = load16_tail(wp, k, K);
#pragma unroll
            for (int c = 0; c < C; ++c)
                acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, load16_tail(xp[c], k, K), acc[c], 0, 0, 0);
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

constexpr int kNumCU = 256;
constexpr int kNumXCD = 8;

// BM tokens x BN channels per workgroup of 8 waves, k-tiles of 128 codes
// (whole 128-byte rows) of both operands in an LDS ring of S stages.  The
// waves form KG groups: one, or two that each take 64 codes of every k-tile
// and add their sums at the end, for tiles too small to feed eight waves.
//
// Rows of an LDS tile keep their order.  Of a 64-channel group, the 16-row
// MFMA block b takes rows 16 (r / 4) + 4 b + r % 4, r = 0..15: lane l's
// results of the group's four blocks are then the 16 consecutive channels
// 16 (l / 16) + 0..15 of one token, and results go from registers to memory in
// runs of 64 channels per token, without a pass through LDS.  Token blocks
// take 16 rows in order.
//
// Row r's chunk c (16 bytes) is kept in slot c ^ swizzle(r).  A 16-byte read
// of a wave goes in four phases of 16 lanes, each of all 64 banks (two rows of
// slots); a phase joins quads of lanes of two neighbouring chunks (0-3, 12-15,
// 20-23, 24-27 and so on).  With a quad's number q = (q1 q0) in row bits 4 and
// 5 (channels) or 2 and 3 (tokens), the swizzle bits (q1, row bit 1, q0 ^ q1)
// from the lowest take both these and 16 lanes in a row to 16 different slots.
//
// D > 0: tiles come through registers, D of them on their way at a time, for
// codes whose rows are not 4-byte aligned; otherwise by LDS DMA.
template <int BM_, int BN_, int WT_, int KG_, int S_, int D_ = 0>
struct Q8Tile {
    static constexpr int BM = BM_, BN = BN_;       // tokens, channels
    static constexpr int NW = 8, NTH = NW * 64;
    static constexpr int KG = KG_;
    static constexpr int WT = WT_, WC = NW / KG / WT;            // waves of a group along each
    static constexpr int S = S_, D = D_;
    static constexpr int MT = BM / WT / 16, NC = BN / WC / 16;   // 16-row blocks per wave
    static constexpr int XROWS = (BM + 63) / 64 * 64;            // whole rounds of the waves' 8-row loads
    static constexpr int XBYTES = XROWS * 128, WBYTES = BN * 128;
    static constexpr int STAGE = XBYTES + WBYTES;
    static constexpr int LDS = S * STAGE;
    static constexpr int XG = XROWS / 8 / NW, WG = BN / 8 / NW;  // loads (8 rows) per wave and tile
    static constexpr int LOADS = XG + WG, FRAGS = MT + NC;
    static_assert(MT * 16 * WT == BM && NC * 16 * WC == BN && NC % 4 == 0, "whole blocks and 64-channel groups per wave");
    static_assert(BN % 64 == 0 && LDS <= 160 * 1024 && S >= 2 && (S - 1) * LOADS < 64, "ring");
    static_assert(KG == 1 || (KG == 2 && BM * BN * 4 <= LDS), "the second group's sums pass through the ring");
    static_assert(D == 0 || S == 2, "tiles through registers wait there, not in LDS");
};

__device__ __forceinline__ int swizzle(int row, int q0) {   // q0: the position of the quad's bits
    const int lo = (row >> q0) & 1, hi = (row >> (q0 + 1)) & 1;
    return hi | (row & 2) | (lo ^ hi) << 2;
}

struct TileGrid {
    int tm, tn;    // tiles along the tokens and the channels
    int ks;        // parts of K
    int* part;     // int32 sums [ks][T][N] where ks > 1
};

// Workgroup id -> part of K and tile.  Ids go round the XCDs, so XCD x takes
// the x-th contiguous part of the order, in which kGroupM token tiles share a
// channel tile before the next one: the tiles an XCD works on at one time are
// a block, whose operands' rows meet in its L2.
constexpr int kGroupM = 8;

__device__ __forceinline__ void tile_of(int id, const TileGrid& g, int& part, int& m, int& n) {
    const int tiles = g.tm * g.tn, total = tiles * g.ks, q = total / kNumXCD, r = total % kNumXCD;
    const int x = id % kNumXCD;
    int i = x * q + (x < r ? x : r) + id / kNumXCD;
    part = i / tiles;
    i -= part * tiles;
    const int per = kGroupM * g.tn, grp = i / per, rest = i % per;
    const int h = g.tm - grp * kGroupM < kGroupM ? g.tm - grp * kGroupM : kGroupM;
    m = grp * kGroupM + rest % h;
    n = rest / h;
}

// VEC: rows of y (and lora) are 16-byte aligned.  PART: the sums of a part of
// K go to the workspace.
template <typename E, typename G, bool VEC, bool PART>
__global__ __launch_bounds__(G::NTH, 1) void q8_tiles(MatmulQ8 a, TileGrid grid) {
    __shared__ __attribute__((aligned(1024))) char smem[G::LDS];
    constexpr int S = G::S, D = G::D, LOADS = G::LOADS, FRAGS = G::FRAGS;
    constexpr bool DMA = D == 0;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = wave / (G::WT * G::WC), wt = wave / G::WC % G::WT, wc = wave % G::WC;
    int part, tm, tn;
    tile_of(blockIdx.x, grid, part, tm, tn);
    const int64_t t0 = (int64_t)tm * G::BM, n0 = (int64_t)tn * G::BN;
    const int K = (int)a.K, tiles = (K + 127) / 128;
    const int k_begin = PART ? (int)((int64_t)tiles * part / grid.ks) : 0;
    const int nk = (PART ? (int)((int64_t)tiles * (part + 1) / grid.ks) : tiles) - k_begin;

    // Loads: lane l moves slot l % 8 of row l / 8 of an 8-row group; the wave's
    // groups are wave, wave + 8, ..., whose swizzles agree.  Rows past the end
    // repeat the last one (their results are not stored); chunks past K read
    // zeros.  A chunk that crosses K holds the next row's first codes (past
    // the operand's end: zeros, by the buffer's size), which mask() removes.
    const int lrow = wave * 8 + (lane >> 3);
    const int xchunk = ((lane & 7) ^ swizzle(lrow, 2)) * 16, wchunk = ((lane & 7) ^ swizzle(lrow, 4)) * 16;
    int xoff[G::XG], woff[G::WG];
#pragma unroll
    for (int i = 0; i < G::XG; ++i) {
        const int r = lrow + i * G::NW * 8;
        xoff[i] = (int)(t0 + r < a.T ? r : a.T - 1 - t0) * K + (DMA ? xchunk : 0);
    }
#pragma unroll
    for (int i = 0; i < G::WG; ++i) {
        const int r = lrow + i * G::NW * 8;
        woff[i] = (int)(n0 + r < a.N ? r : a.N - 1 - n0) * K + (DMA ? wchunk : 0);
    }
    const int8_t* xbase_p = a.xq + t0 * K;
    const int8_t* wbase_p = a.wq + n0 * K;
    auto resource = [](const void* p, int64_t bytes) __attribute__((always_inline)) {
        const uint64_t v = reinterpret_cast<uint64_t>(p);
        i32x4_t rs;
        rs[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
        rs[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
        rs[2] = __builtin_amdgcn_readfirstlane((int)(bytes < 0x7fffffff ? bytes : 0x7fffffff));
        rs[3] = kRsrcWord3;
        return rs;
    };
    const i32x4_t xr = resource(xbase_p, (a.T - t0) * K), wr = resource(wbase_p, (a.N - n0) * K);
    i32x4_t held[DMA ? 1 : D][DMA ? 1 : LOADS];   // tiles on their way through registers
    // Each XCD starts its walk over K at its own place, so that rows of one
    // pitch are not all asked for the same columns at once; within an XCD the
    // walks stay together, which its L2 lives on.
    const int rot = (int)((unsigned)(blockIdx.x % kNumXCD) * (unsigned)nk / kNumXCD);
    auto tile_at = [&](int j) __attribute__((always_inline)) {   // the j-th k-tile of the walk
        return k_begin + (j + rot < nk ? j + rot : j + rot - nk);
    };
    // load i of the walk's tile j; past the last one: nothing that anyone reads
    auto issue_one = [&](int j, int stage, int slot, int i) __attribute__((always_inline)) {
        const int k = tile_at(j) * 128;
        if constexpr (DMA) {
            const bool in = j < nk && k + (i < G::XG ? xchunk : wchunk) < K;
            char* dst = smem + stage + wave * 1024 + i * G::NW * 1024;   // the channels' rows follow the tokens'
            if (i < G::XG)
                raw_buffer_load_lds(xr, (lds_void_t*)dst, 16, in ? xoff[i < G::XG ? i : 0] : kOutOfRange, k, 0, 0);
            else
                raw_buffer_load_lds(wr, (lds_void_t*)dst, 16, in ? woff[i < G::XG ? 0 : i - G::XG] : kOutOfRange, k, 0, 0);
        } else if (j < nk) {
            const int8_t* row = i < G::XG ? xbase_p + xoff[i < G::XG ? i : 0] : wbase_p + woff[i < G::XG ? 0 : i - G::XG];
            const int at = k + (i < G::XG ? xchunk : wchunk);
            held[slot][i] = k + 128 <= K ? load16(row + at) : load16_tail(row, at, K);
        }
    };
    auto issue = [&](int j, int stage, int slot) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) issue_one(j, stage, slot, i);
    };
    auto land = [&](int stage, int slot) __attribute__((always_inline)) {   // registers to LDS
        if constexpr (!DMA) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                *reinterpret_cast<i32x4_t*>(smem + stage + wave * 1024 + i * G::NW * 1024 + lane * 16) = held[slot][i];
        }
    };

    // fragments: lane l reads chunk 4 ks + l / 16 of its row
    const int xrow = lane & 15, wrow = ((lane & 12) << 2) | (lane & 3);
    const int xfo = (wt * G::MT * 16 + xrow) * 128 + (((lane >> 4) ^ swizzle(xrow, 2)) << 4);   // ks = 0; ks = 1 is ^ 64
    const int wfo = G::XBYTES + (wc * G::NC * 16 + wrow) * 128 + (((lane >> 4) ^ swizzle(wrow, 4)) << 4);
    i32x4_t acc[G::MT][G::NC];
#pragma unroll
    for (int m = 0; m < G::MT; ++m)
#pragma unroll
        for (int c = 0; c < G::NC; ++c) acc[m][c] = {0, 0, 0, 0};

    auto read_one = [&](int stage, int ks, int i, i32x4_t (&x)[G::MT], i32x4_t (&w)[G::NC]) __attribute__((always_inline)) {
        if (i < G::NC)
            w[i < G::NC ? i : 0] = *reinterpret_cast<const i32x4_t*>(smem + stage + (wfo ^ (ks * 64)) + (i / 4) * 64 * 128 + (i % 4) * 4 * 128);
        else
            x[i < G::NC ? 0 : i - G::NC] = *reinterpret_cast<const i32x4_t*>(smem + stage + (xfo ^ (ks * 64)) + (i - G::NC) * 16 * 128);
    };
    // the last k-tile's codes past K out of the channels' fragments
    const bool ragged = DMA && K % 16 != 0;
    auto mask = [&](int j, int ks, i32x4_t (&w)[G::NC]) __attribute__((always_inline)) {
        if (DMA && ragged && tile_at(j) == tiles - 1) {
            const int left = K - (tiles - 1) * 128 - (ks * 4 + (lane >> 4)) * 16;   // a multiple of 4
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int keep = 4 * d < left ? -1 : 0;
#pragma unroll
                for (int c = 0; c < G::NC; ++c) w[c][d] &= keep;
            }
        }
    };
    auto mma = [&](const i32x4_t (&x)[G::MT], const i32x4_t (&w)[G::NC]) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < G::MT; ++m)
#pragma unroll
            for (int c = 0; c < G::NC; ++c) acc[m][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[c], x[m], acc[m][c], 0, 0, 0);
    };
    // Reads, and the second step's loads, are spread over the MFMAs: the reads
    // run under the matrix pipe, and a wave's loads wait their turn at the
    // CU's one address unit without holding up its MFMAs.
    constexpr int PER = G::MT * G::NC < FRAGS ? 1 : G::MT * G::NC / FRAGS;   // MFMAs per fragment read
    auto interleave = [](bool loads) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FRAGS; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);   // MFMA
            if (loads && DMA && i < LOADS) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // load
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // LDS read
        }
        __builtin_amdgcn_sched_group_barrier(0x008, G::MT * G::NC, 0);
        __builtin_amdgcn_sched_barrier(0);
    };

    // A k-tile is two steps of 64 codes (with two groups: one step of each).
    // While one step's MFMAs run the next step's fragments are read.  Once per
    // tile, before its last step: this wave's loads of the next tile have
    // landed and its reads of this tile are done; barrier; then tile j + S (in
    // registers: j + 1 + D) is enqueued into what this tile (tile j + 1) held.
    i32x4_t x0[G::MT], w0[G::NC], x1[G::MT], w1[G::NC];
    constexpr int UNROLL = DMA ? 1 : D;   // registers are indexed by constants
    if (nk > 0) {
        if constexpr (DMA) {
#pragma unroll
            for (int s = 0; s < S; ++s) issue(s, s * G::STAGE, 0);
            wait_vmcnt<(S - 1) * LOADS>();
            __builtin_amdgcn_s_barrier();
        } else {
#pragma unroll
            for (int s = 0; s < D; ++s) issue(s, 0, s);
            land(0, 0);
            issue(D, 0, 0);
            __syncthreads();
        }
        const int ks0 = G::KG == 1 ? 0 : kg;
#pragma unroll
        for (int i = 0; i < FRAGS; ++i) read_one(0, ks0, i, x0, w0);
        mask(0, ks0, w0);
        int here = 0;   // this tile's stage
        for (int j0 = 0; j0 < nk; j0 += UNROLL) {
#pragma unroll
            for (int d = 0; d < UNROLL; ++d) {
                const int j = j0 + d;
                if (UNROLL > 1 && j >= nk) break;
                const int next = here + G::STAGE == G::LDS ? 0 : here + G::STAGE, slot = (d + 1) % UNROLL;
                if constexpr (G::KG == 1) {
#pragma unroll
                    for (int i = 0; i < FRAGS; ++i) read_one(here, 1, i, x1, w1);
                    mma(x0, w0);
                    interleave(false);
                    mask(j, 1, w1);
                } else {
#pragma unroll
                    for (int m = 0; m < G::MT; ++m) x1[m] = x0[m];
#pragma unroll
                    for (int c = 0; c < G::NC; ++c) w1[c] = w0[c];
                }
                if constexpr (DMA) {
                    wait_vmcnt<(S - 2) * LOADS>();
                    wait_lgkmcnt0();
                    __builtin_amdgcn_s_barrier();
                } else {
                    land(next, slot);   // the readers of that stage's last tile passed the last barrier
                    __syncthreads();
                }
#pragma unroll
                for (int i = 0; i < (FRAGS > LOADS ? FRAGS : LOADS); ++i) {
                    if (i < LOADS) issue_one(DMA ? j + S : j + 1 + D, here, slot, i);
                    if (i < FRAGS) read_one(next, ks0, i, x0, w0);   // past the last tile: unused
                }
                mma(x1, w1);
                interleave(true);
                mask(j + 1, ks0, w0);
                here = next;
            }
        }
        wait_vmcnt<0>();
    }
    if constexpr (G::KG == 2) {   // the second group's sums to the first
        __syncthreads();
        char* sums = smem + (wt * G::WC + wc) * G::MT * G::NC * 1024 + lane * 16;
        if (kg == 1) {
#pragma unroll
            for (int m = 0; m < G::MT; ++m)
#pragma unroll
                for (int c = 0; c < G::NC; ++c) *reinterpret_cast<i32x4_t*>(sums + (m * G::NC + c) * 1024) = acc[m][c];
        }
        __syncthreads();
        if (kg == 1) return;
#pragma unroll
        for (int m = 0; m < G::MT; ++m)
#pragma unroll
            for (int c = 0; c < G::NC; ++c) {
                const i32x4_t v = *reinterpret_cast<const i32x4_t*>(sums + (m * G::NC + c) * 1024);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][c][e] += v[e];
            }
    }

    // epilogue: token block m of the wave, channels ch .. ch + 15 per lane
    auto epilogue = [&](auto adapter) __attribute__((always_inline)) {
        constexpr bool ADAPTER = decltype(adapter)::value;
        constexpr int P = VEC ? Pack<E>::N : 1;
#pragma unroll
        for (int cg = 0; cg < G::NC / 4; ++cg) {
            const int64_t ch = n0 + (wc * G::NC + cg * 4) * 16 + (lane >> 4) * 16;
            if (ch >= a.N) continue;
            Channel cc[16];
            if (!PART) load_channels(a, ch, cc);
#pragma unroll
            for (int m = 0; m < G::MT; ++m) {
                const int64_t t = t0 + (wt * G::MT + m) * 16 + (lane & 15);
                if (t >= a.T) continue;
                const int64_t at = t * a.N + ch;
                if (PART) {
                    int* dst = grid.part + (int64_t)part * a.T * a.N + at;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (a.N % 4 == 0) {
                            if (ch + 4 * b < a.N) *reinterpret_cast<i32x4_t*>(dst + 4 * b) = acc[m][cg * 4 + b];
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (ch + 4 * b + e < a.N) dst[4 * b + e] = acc[m][cg * 4 + b][e];
                        }
                    }
                    continue;
                }
                const float xs = a.xs[t];
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
    if (!PART && a.g)
        epilogue(std::true_type{});
    else
        epilogue(std::false_type{});
}

// The parts of K joined, and the epilogue: 4 channels of one token per thread
// (one where N is not a multiple of 4).  Integer sums: any order is exact.
template <typename E, int P>
__global__ __launch_bounds__(256) void q8_join(MatmulQ8 a, const int* __restrict__ part, int ks) {
    const int64_t per = a.N / P, all = a.T * a.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.T * per; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / per, n = (i - t * per) * P, at = t * a.N + n;
        int v[P];
#pragma unroll
        for (int e = 0; e < P; ++e) v[e] = 0;
        for (int k = 0; k < ks; ++k) {
            const int* src = part + k * all + at;
            if (P == 4) {
                const i32x4_t q = *reinterpret_cast<const i32x4_t*>(src);
#pragma unroll
                for (int e = 0; e < P; ++e) v[e] += q[e];
            } else {
                v[0] += *src;
            }
        }
        Channel cc[P];
        load_channels(a, n, cc);
        const float xs = a.xs[t];
        E l[P], o[P];
        if (a.g) __builtin_memcpy(l, static_cast<const E*>(a.lora) + at, sizeof(l));
#pragma unroll
        for (int e = 0; e < P; ++e)
            o[e] = Cvt<E>::from_f(a.g ? finish<true>(v[e], xs, cc[e], Cvt<E>::to_f(l[e])) : finish<false>(v[e], xs, cc[e], 0.0f));
        __builtin_memcpy(static_cast<E*>(a.y) + at, o, sizeof(o));
    }
}

// ------------------------------------------------------------- choice of form

constexpr int kDirect = -1;

struct Q8Plan {
    int form;   // kDirect, or a tile form
    int ks;     // parts of K
};

Q8Plan plan_q8(int64_t T, int64_t N, int64_t K, bool dma) {
    if (T <= 64 || K < 16) return {kDirect, 1};
    if (!dma) return {T * N > 512 * 4096 ? 4 : 6, 1};
    return {0, 1};
}

size_t plan_bytes(const Q8Plan& p, int64_t T, int64_t N) { return p.ks > 1 ? (size_t)p.ks * T * N * sizeof(int) : 0; }

// ------------------------------------------------------------- launches

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <typename E, typename G>
hipError_t launch_form(const MatmulQ8& a, int ks, void* workspace, hipStream_t st) {
    const TileGrid g{(int)((a.T + G::BM - 1) / G::BM), (int)((a.N + G::BN - 1) / G::BN), ks, static_cast<int*>(workspace)};
    const unsigned wgs = (unsigned)(g.tm * g.tn * ks);
    if (ks > 1) {
        q8_tiles<float, G, false, true><<<wgs, G::NTH, 0, st>>>(a, g);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int p = a.N % 4 == 0 ? 4 : 1;
        int64_t blocks = (a.T * (a.N / p) + 255) / 256;
        if (blocks > 65536) blocks = 65536;
        if (p == 4)
            q8_join<E, 4><<<(unsigned)blocks, 256, 0, st>>>(a, g.part, ks);
        else
            q8_join<E, 1><<<(unsigned)blocks, 256, 0, st>>>(a, g.part, ks);
    } else if (a.N % Pack<E>::N == 0 && aligned_to(a.y, 16) && aligned_to(a.lora, 16)) {
        q8_tiles<E, G, true, false><<<wgs, G::NTH, 0, st>>>(a, g);
    } else {
        q8_tiles<E, G, false, false><<<wgs, G::NTH, 0, st>>>(a, g);
    }
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
hipError_t launch_typed(const MatmulQ8& a, void* workspace, hipStream_t st) {
    const bool dma = a.K % 4 == 0 && aligned_to(a.xq, 4) && aligned_to(a.wq, 4);
    const Q8Plan p = plan_q8(a.T, a.N, a.K, dma);
    if (p.form == kDirect) return launch_direct<E>(a, st);
    if (!dma) {
        if (p.form == 4) return launch_form<E, Q8Tile<128, 128, 4, 1, 2, 3>>(a, p.ks, workspace, st);
        return launch_form<E, Q8Tile<64, 64, 4, 2, 2, 8>>(a, p.ks, workspace, st);
    }
    switch (p.form) {
        case 0: return launch_form<E, Q8Tile<256, 256, 2, 1, 2>>(a, p.ks, workspace, st);
        case 1: return launch_form<E, Q8Tile<192, 256, 2, 1, 2>>(a, p.ks, workspace, st);
        case 2: return launch_form<E, Q8Tile<128, 256, 2, 1, 3>>(a, p.ks, workspace, st);
        case 3: return launch_form<E, Q8Tile<64, 256, 2, 1, 4>>(a, p.ks, workspace, st);
        case 4: return launch_form<E, Q8Tile<128, 128, 4, 1, 5>>(a, p.ks, workspace, st);
        case 5: return launch_form<E, Q8Tile<64, 128, 4, 1, 6>>(a, p.ks, workspace, st);
        case 6: return launch_form<E, Q8Tile<64, 64, 4, 2, 8>>(a, p.ks, workspace, st);
        case 7: return launch_form<E, Q8Tile<128, 64, 4, 2, 6>>(a, p.ks, workspace, st);
        default: return launch_form<E, Q8Tile<64, 64, 4, 2, 4>>(a, p.ks, workspace, st);
    }
}

}  // namespace

size_t matmul_q8_workspace_bytes(int64_t T, int64_t N, int64_t K) {
    // the codes' alignment is known only at the call
    size_t most = 0;
    for (int dma = 0; dma < 2; ++dma) {
        if (dma && K % 4 != 0) continue;
        const size_t b = plan_bytes(plan_q8(T, N, K, dma), T, N);
        most = b > most ? b : most;
    }
    return align_up(most, 256);
}

hipError_t launch_matmul_q8(const MatmulQ8& a, int dtype, void* workspace, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    switch (dtype) {
        case kF32: return launch_typed<float>(a, workspace, stream);
        case kBF16: return launch_typed<bf16_t>(a, workspace, stream);
        default: return launch_typed<f16_t>(a, workspace, stream);
    }
}

}  // namespace dora
