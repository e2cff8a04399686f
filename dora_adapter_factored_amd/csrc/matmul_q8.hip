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
#include "dora_q8_plan.h"

namespace dora {
namespace {

constexpr int kWaves = 8;

// 16 bytes from any address.
__device__ __forceinline__ i32x4_t load16(const int8_t* p) {
    i32x4_t v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// The same by whole dwords, for scattered rows: lanes that each read 16 bytes
// of another row at odd addresses are split into bytes' worth of requests (4 x
// 5120 x 27649 took 138 us, 27648 30).  The dwords read are those that hold
// the 16 bytes, so nothing is touched that shares no aligned dword with them.
struct Odd16 {
    i32x4_t lo;
    int hi, shift;
};

__device__ __forceinline__ Odd16 load16_dwords(const int8_t* p) {
    Odd16 v;
    v.shift = (int)(reinterpret_cast<uintptr_t>(p) & 3);
    const int* d = reinterpret_cast<const int*>(p - v.shift);
    __builtin_memcpy(&v.lo, __builtin_assume_aligned(d, 4), 16);
    v.hi = d[v.shift ? 4 : 3];
    return v;
}

__device__ __forceinline__ i32x4_t join(const Odd16& v) {
    i32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = (int)__builtin_amdgcn_alignbyte((uint32_t)(i < 3 ? v.lo[i < 3 ? i + 1 : 3] : v.hi), (uint32_t)v.lo[i], (uint32_t)v.shift);
    return r;
}

// v without its first n bytes, zeros after them.
__device__ __forceinline__ i32x4_t drop_bytes(const i32x4_t& v, int n) {
    uint64_t lo = (uint32_t)v[0] | (uint64_t)(uint32_t)v[1] << 32, hi = (uint32_t)v[2] | (uint64_t)(uint32_t)v[3] << 32;
    const int bits = 8 * n;
    if (n >= 16) lo = hi = 0;
    else if (n >= 8) lo = hi >> (bits - 64), hi = 0;
    else if (n > 0) lo = lo >> bits | hi << (64 - bits), hi >>= bits;
    return i32x4_t{(int)(uint32_t)lo, (int)(uint32_t)(lo >> 32), (int)(uint32_t)hi, (int)(uint32_t)(hi >> 32)};
}

// Bytes k .. k + 15 of a row of K, zeros past its end: the last 16 bytes of
// the row moved down, so that nothing outside the row is read.
__device__ __forceinline__ i32x4_t load16_tail(const int8_t* row, int k, int K) {
    if (K < 16) {
        i32x4_t v = {0, 0, 0, 0};
        for (int b = 0; b < 16; ++b)
            if (k + b < K) v[b / 4] |= (int)(uint8_t)row[k + b] << (8 * (b % 4));
        return v;
    }
    const int at = k < K - 16 ? k : K - 16;
    return drop_bytes(load16(row + at), k - at);
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

// One token: kRows channels per workgroup on the vector units.  The weight's
// bytes are all that counts, and a load takes 1 KB of one channel's row, whole
// lines only, where the MFMA layout of q8_direct asks for 64 bytes of each of
// 16 rows, which holds a CU to about 22 GB/s.  Wave w takes every eighth KB of
// the rows from the w-th; lanes, then waves are summed at the end.  8192 x
// 8192: 13.6 us, 4.9 TB/s (q8_direct 15.1); 28672 x 8192: 39.1 us, 6.0 TB/s
// (42.6); 5120 x 27648: 27.5 us (39.5); two channels per workgroup 46.8 us and
// eight 43.4 at 28672 x 8192.
constexpr int kRows = 4;

template <typename E>
__global__ __launch_bounds__(kWaves * 64) void q8_one_token(MatmulQ8 a) {
    __shared__ int red[kWaves][kRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * kRows;
    const int K = (int)a.K;
    int acc[kRows] = {};
    auto step = [&](int k, auto tail) __attribute__((always_inline)) {
        constexpr bool TAIL = decltype(tail)::value;
        i32x4_t w[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {   // channels past the end repeat the last one; their results are not stored
            const int8_t* row = a.wq + (n0 + r < a.N ? n0 + r : a.N - 1) * K;
            w[r] = TAIL ? load16_tail(row, k, K) : load16(row + k);
        }
        const i32x4_t x = TAIL ? load16_tail(a.xq, k, K) : load16(a.xq + k);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int d = 0; d < 4; ++d) acc[r] = __builtin_amdgcn_sdot4(w[r][d], x[d], acc[r], false);
    };
    int k0 = wave * 1024;
#pragma unroll 2
    for (; k0 + 1024 <= K; k0 += kWaves * 1024) step(k0 + lane * 16, std::false_type{});
    if (k0 < K) step(k0 + lane * 16, std::true_type{});
    // the lanes' sums: two steps in which a lane hands half of its values over
    // and keeps the others, after which lane l holds channel l / 16
    const bool up5 = lane & 32, up4 = lane & 16;
    int v0 = (up5 ? acc[2] : acc[0]) + __shfl_xor(up5 ? acc[0] : acc[2], 32);
    const int v1 = (up5 ? acc[3] : acc[1]) + __shfl_xor(up5 ? acc[1] : acc[3], 32);
    v0 = (up4 ? v1 : v0) + __shfl_xor(up4 ? v0 : v1, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v0 += __shfl_xor(v0, o);
    if (lane % 16 == 0) red[wave][lane / 16] = v0;
    __syncthreads();
    const int64_t n = n0 + threadIdx.x;
    if (threadIdx.x >= kRows || n >= a.N) return;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += red[w][threadIdx.x];
    Channel cc[1];
    load_channels(a, n, cc);
    const float y = a.g ? finish<true>(sum, a.xs[0], cc[0], Cvt<E>::to_f(static_cast<const E*>(a.lora)[n]))
                        : finish<false>(sum, a.xs[0], cc[0], 0.0f);
    static_cast<E*>(a.y)[n] = Cvt<E>::from_f(y);
}

// 16 channels x 16 tokens per workgroup, the waves taking 128-byte columns of
// K in turn straight from memory into the MFMA operands; the waves' sums are
// added through LDS.  For few tokens and channels, where tiles through LDS
// would leave most CUs without work (12 x 1024 x 5120: 7.0 us, 64 x 64 tiles
// in 4 parts 10.4), for rows of fewer than 16 codes, and for few tokens of
// codes whose rows are not 4-byte aligned.  8 x 8192 x 8192: 16.5 us, 4.1 TB/s;
// 64-byte requests hold a CU to 22.5 GB/s.
template <typename E, bool DWORDS>   // DWORDS: rows are 4-byte aligned
__global__ __launch_bounds__(kWaves * 64) void q8_direct(MatmulQ8 a) {
    __shared__ int red[kWaves][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * 16;
    // rows past the end repeat the last one; their results are not stored
    const int64_t nr = n0 + (lane & 15) < a.N ? n0 + (lane & 15) : a.N - 1;
    const int64_t tr = t0 + (lane & 15) < a.T ? t0 + (lane & 15) : a.T - 1;
    const int kl = (lane >> 4) * 32;
    const int K = (int)a.K;
    const int8_t* wp = a.wq + nr * K;
    const int8_t* xp = a.xq + tr * K;
    i32x4_t acc = {0, 0, 0, 0};
    const int full = K / 128;
    // U columns at a time, all their loads before the first MFMA
    auto columns = [&](int kb, auto u) __attribute__((always_inline)) {
        constexpr int U = decltype(u)::value;
        typedef typename std::conditional<DWORDS, i32x4_t, Odd16>::type Codes;
        Codes w[U][2], x[U][2];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = (kb + i * kWaves) * 128 + kl + j * 16;
                if constexpr (DWORDS) {
                    w[i][j] = load16(wp + k);
                    x[i][j] = load16(xp + k);
                } else {
                    w[i][j] = load16_dwords(wp + k);
                    x[i][j] = load16_dwords(xp + k);
                }
            }
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (DWORDS)
                    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[i][j], x[i][j], acc, 0, 0, 0);
                else
                    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(join(w[i][j]), join(x[i][j]), acc, 0, 0, 0);
            }
    };
    int kb = wave;
    for (; kb + 3 * kWaves < full; kb += 4 * kWaves) columns(kb, std::integral_constant<int, 4>{});
    for (; kb < full; kb += kWaves) columns(kb, std::integral_constant<int, 1>{});
    if (full % kWaves == wave && full * 128 < K) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = full * 128 + kl + j * 16;
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(load16_tail(wp, k, K), load16_tail(xp, k, K), acc, 0, 0, 0);
        }
    }
    *reinterpret_cast<i32x4_t*>(&red[wave][lane * 4]) = acc;
    __syncthreads();
    if (threadIdx.x >= 256) return;
    const int tok = threadIdx.x >> 4, ch = threadIdx.x & 15;
    const int64_t t = t0 + tok, n = n0 + ch;
    if (t >= a.T || n >= a.N) return;
    const int src = ((ch >> 2) * 16 + tok) * 4 + (ch & 3);
    int v = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += red[w][src];
    Channel cc[1];
    load_channels(a, n, cc);
    const float r = a.g ? finish<true>(v, a.xs[t], cc[0], Cvt<E>::to_f(static_cast<const E*>(a.lora)[t * a.N + n]))
                        : finish<false>(v, a.xs[t], cc[0], 0.0f);
    static_cast<E*>(a.y)[t * a.N + n] = Cvt<E>::from_f(r);
}

// ------------------------------------------------------------- tiles through LDS

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
    int* part;     // where ks > 1: the parts' int32 sums, as part_at() lays them out
};

// The sums of one MFMA block of one part, 16 bytes a lane: blocks of a wave,
// waves of a tile, tiles, parts.
template <typename G>
__device__ __forceinline__ i32x4_t* part_at(const TileGrid& g, int part, int tm, int tn, int wave, int m, int c) {
    const int64_t tile = ((int64_t)part * g.tn + tn) * g.tm + tm;
    return reinterpret_cast<i32x4_t*>(g.part) + (((tile * (G::NW / G::KG) + wave) * G::MT + m) * G::NC + c) * 64;
}

// Workgroup id -> part of K and tile.  Ids go round the XCDs, so XCD x takes
// the x-th contiguous part of the order, in which kGroupM token tiles share a
// channel tile before the next one: the tiles an XCD works on at one time are
// a block, whose operands' rows meet in its L2.  In turn on one card at 4096 x
// 28672 x 8192, 256 x 256 tiles: 4 x 8 tiles 736 us, 8 x 4 739; 2 x 16, 3 x 11 and
// 16 x 2 3 to 5% more.  (The card's power sets the level, 695 to 736 us in
// several runs; only runs in turn compare.)
constexpr int kGroupM = 4;

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

// What bounds the tile forms, on MI355X.  256 x 256 over the whole chip: power
// and the operands' way to the CU.  Of the cycles at 4096 x 28672 x 8192 the
// matrix units are busy in 66% (SQ_VALU_MFMA_BUSY_CYCLES), at 1.85 GHz of
// 2.4; with every load a hit in L2 the product is 6 to 9% faster, LDS has no
// bank conflicts (with them: 1% slower), and 4 waves of 128 x 128 with a third
// fewer LDS reads are no faster.  The small forms: the latency of a k-tile's
// barrier, fragment reads and loads in one workgroup (290 ns for 64 x 64),
// which a second workgroup on the CU hides.

// Results of wave (wt, wc) of the tile at (t0, n0), token blocks m_begin ..
// m_end - 1: lane l has token l % 16 of a block and the 16 channels from 16 (l
// / 16) of each 64-channel group, four of them in sums(m, group, 0 .. 3) each.
// Rows of y (and lora) that are not 16-byte aligned (VEC false) are written in
// the same packs at their elements' alignment, the last one element by
// element: all of them so took 68 us at 2000 x 4097 x 4096 where this takes 47
// (4096 channels: 35).
template <typename E, typename G, bool VEC, bool ADAPTER, typename Sums>
__device__ __forceinline__ void store_results(const MatmulQ8& a, int64_t t0, int64_t n0, int wt, int wc, int m_begin, int m_end,
                                              Sums sums) {
    constexpr int P = Pack<E>::N;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int cg = 0; cg < G::NC / 4; ++cg) {
        const int64_t ch = n0 + (wc * G::NC + cg * 4) * 16 + (lane >> 4) * 16;
        if (ch >= a.N) continue;
        Channel cc[16];
        load_channels(a, ch, cc);
#pragma unroll
        for (int m = m_begin; m < m_end; ++m) {
            const int64_t t = t0 + (wt * G::MT + m) * 16 + (lane & 15);
            if (t >= a.T) continue;
            const int64_t at = t * a.N + ch;
            const float xs = a.xs[t];
#pragma unroll
            for (int h = 0; h < 16; h += P) {
                const int64_t left = a.N - ch - h;
                if (left <= 0) continue;
                const E* lora = static_cast<const E*>(a.lora) + at + h;
                E* y = static_cast<E*>(a.y) + at + h;
                Pack<E> l, o;
                if (ADAPTER) {
                    if (VEC) {
                        l = load_pack(lora);
                    } else if (left >= P) {
                        __builtin_memcpy(&l.u, lora, 16);
                    } else {
#pragma unroll
                        for (int e = 0; e < P; ++e) l.e[e] = lora[e < left ? e : left - 1];
                    }
                }
#pragma unroll
                for (int e = 0; e < P; ++e)
                    o.e[e] = Cvt<E>::from_f(finish<ADAPTER>(sums(m, cg, (h + e) / 4)[(h + e) % 4], xs, cc[h + e],
                                                            ADAPTER ? Cvt<E>::to_f(l.e[e]) : 0.0f));
                if (VEC) {
                    *reinterpret_cast<u32x4_t*>(y) = o.u;
                } else if (left >= P) {
                    __builtin_memcpy(y, &o.u, 16);
                } else {
#pragma unroll
                    for (int e = 0; e < P; ++e)
                        if (e < left) y[e] = o.e[e];
                }
            }
        }
    }
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
    // through registers the walk is over whole tiles, and a ragged last one follows it
    const int nk = DMA ? (PART ? (int)((int64_t)tiles * (part + 1) / grid.ks) : tiles) - k_begin : K / 128;

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
    Odd16 held[DMA ? 1 : D][DMA ? 1 : LOADS];   // tiles on their way through registers
    // Each XCD starts its walk over K at its own place, so that rows of one
    // pitch are not all asked for the same columns at once; within an XCD the
    // walks stay together, which its L2 lives on.
    const int rot = (int)((unsigned)(blockIdx.x % kNumXCD) * (unsigned)nk / kNumXCD);
    auto tile_at = [&](int j) __attribute__((always_inline)) {   // the j-th k-tile of the walk
        return k_begin + (j + rot < nk ? j + rot : j + rot - nk);
    };
    auto row_of = [&](int i) __attribute__((always_inline)) {
        return i < G::XG ? xbase_p + xoff[i < G::XG ? i : 0] : wbase_p + woff[i < G::XG ? 0 : i - G::XG];
    };
    // load i of the walk's tile j; past the last one: nothing that anyone reads
    auto issue_one = [&](int j, int stage, int slot, int i) __attribute__((always_inline)) {
        const int k = j < nk ? tile_at(j) * 128 : 0;   // a buffer's scalar offset stays inside it
        if constexpr (DMA) {
            const bool in = j < nk && k + (i < G::XG ? xchunk : wchunk) < K;
            char* dst = smem + stage + wave * 1024 + i * G::NW * 1024;   // the channels' rows follow the tokens'
            if (i < G::XG)
                raw_buffer_load_lds(xr, (lds_void_t*)dst, 16, in ? xoff[i < G::XG ? i : 0] : kOutOfRange, k, 0, 0);
            else
                raw_buffer_load_lds(wr, (lds_void_t*)dst, 16, in ? woff[i < G::XG ? 0 : i - G::XG] : kOutOfRange, k, 0, 0);
        } else {   // past the last tile the first again, which land() turns to zeros: no branch round a load
            held[slot][i] = load16_dwords(row_of(i) + k + (i < G::XG ? xchunk : wchunk));
        }
    };
    auto issue = [&](int j, int stage, int slot) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) issue_one(j, stage, slot, i);
    };
    auto put = [&](int stage, int i, const i32x4_t& v) __attribute__((always_inline)) {
        *reinterpret_cast<i32x4_t*>(smem + stage + wave * 1024 + i * G::NW * 1024 + lane * 16) = v;
    };
    auto land = [&](int j, int stage, int slot) __attribute__((always_inline)) {   // registers to LDS
        if constexpr (!DMA) {
            const int keep = j < nk ? -1 : 0;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) put(stage, i, join(held[slot][i]) & keep);
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
    // back and forth, so that each MFMA has an operand of the one before it: the
    // full chip runs against its power limit (1.85 GHz at 4096 x 28672 x 8192,
    // 4.0 POP/s with operands in registers and nothing else, 4.9 with zeros in
    // them), and fewer toggled inputs are 0.6 to 1% of the time at sizes that
    // fill it (735.7 against 742.0 us in turn; 104.1 against 104.8 at 2048 x 8192 x
    // 8192)
    auto mma = [&](const i32x4_t (&x)[G::MT], const i32x4_t (&w)[G::NC]) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < G::MT; ++m)
#pragma unroll
            for (int i = 0; i < G::NC; ++i) {
                const int c = m % 2 ? G::NC - 1 - i : i;
                acc[m][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[c], x[m], acc[m][c], 0, 0, 0);
            }
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
    i32x4_t last[DMA ? 1 : LOADS];   // through registers: the ragged last tile, at hand from the start
    if (!DMA) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int at = K / 128 * 128 + (i < G::XG ? xchunk : wchunk);
            last[DMA ? 0 : i] = load16(row_of(i) + (at < K - 16 ? at : K - 16));
        }
    }
    const int ks0 = G::KG == 1 ? 0 : kg;
    int here = 0;   // this tile's stage
    if (nk > 0) {
        if constexpr (DMA) {
#pragma unroll
            for (int s = 0; s < S; ++s) issue(s, s * G::STAGE, 0);
            wait_vmcnt<(S - 1) * LOADS>();
            lds_barrier();
        } else {
#pragma unroll
            for (int s = 0; s < D; ++s) issue(s, 0, s);
            land(0, 0, 0);
            issue(D, 0, 0);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < FRAGS; ++i) read_one(0, ks0, i, x0, w0);
        mask(0, ks0, w0);
        for (int j0 = 0; j0 < nk; j0 += UNROLL) {
#pragma unroll
            for (int d = 0; d < UNROLL; ++d) {
                const int j = j0 + d;   // past the last tile: zeros
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
                    lds_barrier();
                } else {
                    land(j + 1, next, slot);   // the readers of that stage's last tile passed the last barrier
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
        if (DMA) wait_vmcnt<0>();
    }
    if (!DMA && K % 128 != 0) {
        const int other = G::STAGE - here;   // its readers passed the last barrier
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int at = K / 128 * 128 + (i < G::XG ? xchunk : wchunk);
            put(other, i, drop_bytes(last[DMA ? 0 : i], at > K - 16 ? at - (K - 16) : 0));
        }
        __syncthreads();
#pragma unroll
        for (int ks = ks0; ks < (G::KG == 1 ? 2 : ks0 + 1); ++ks) {
#pragma unroll
            for (int i = 0; i < FRAGS; ++i) read_one(other, ks, i, x0, w0);
            mma(x0, w0);
        }
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

    if constexpr (PART) {
#pragma unroll
        for (int m = 0; m < G::MT; ++m)
#pragma unroll
            for (int c = 0; c < G::NC; ++c) part_at<G>(grid, part, tm, tn, wt * G::WC + wc, m, c)[lane] = acc[m][c];
    } else {
        if (a.g)
            store_results<E, G, VEC, true>(a, t0, n0, wt, wc, 0, G::MT, [&](int m, int cg, int b) { return acc[m][cg * 4 + b]; });
        else
            store_results<E, G, VEC, false>(a, t0, n0, wt, wc, 0, G::MT, [&](int m, int cg, int b) { return acc[m][cg * 4 + b]; });
    }
}

// The parts of K joined, and the epilogue: a wave for each token block of a
// tile's wave.  Integer sums: any order is exact.  Bound by the parts' bytes
// (134 MB of 2048 x 8192 x 8192 in two parts: 35 us more than one part's
// epilogue; in row order, 16 bytes of 64 rows at a time, it took 150).
template <typename E, typename G, bool VEC>
__global__ __launch_bounds__(256) void q8_join(MatmulQ8 a, TileGrid grid) {
    const int lane = threadIdx.x & 63;
    constexpr int PER = G::NW / G::KG * G::MT;   // waves per tile
    const int id = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
    const int tile = id / PER, rest = id % PER, wave = rest / G::MT, m = rest % G::MT;
    const int tm = tile % grid.tm, tn = tile / grid.tm;
    if (tn >= grid.tn) return;
    i32x4_t sum[G::NC];
#pragma unroll
    for (int c = 0; c < G::NC; ++c) sum[c] = {0, 0, 0, 0};
#pragma unroll 4
    for (int p = 0; p < grid.ks; ++p) {
#pragma unroll
        for (int c = 0; c < G::NC; ++c) sum[c] += part_at<G>(grid, p, tm, tn, wave, m, c)[lane];
    }
    const int64_t t0 = (int64_t)tm * G::BM, n0 = (int64_t)tn * G::BN;
    if (a.g)
        store_results<E, G, VEC, true>(a, t0, n0, wave / G::WC, wave % G::WC, m, m + 1, [&](int, int cg, int b) { return sum[cg * 4 + b]; });
    else
        store_results<E, G, VEC, false>(a, t0, n0, wave / G::WC, wave % G::WC, m, m + 1, [&](int, int cg, int b) { return sum[cg * 4 + b]; });
}

// Rows of K codes to rows of Kp, a multiple of 16, zeros after the codes: x's T
// rows, then w's N.
__global__ __launch_bounds__(256) void q8_pad(MatmulQ8 a, int Kp, int8_t* __restrict__ xp, int8_t* __restrict__ wp) {
    const int K = (int)a.K;
    for (int64_t row = blockIdx.x; row < a.T + a.N; row += gridDim.x) {
        const bool x = row < a.T;
        const int64_t r = x ? row : row - a.T;
        const int8_t* src = (x ? a.xq : a.wq) + r * K;
        int8_t* dst = (x ? xp : wp) + r * Kp;
        for (int k = threadIdx.x * 16; k < Kp; k += 256 * 16)
            *reinterpret_cast<i32x4_t*>(dst + k) = k + 16 <= K ? load16(src + k) : load16_tail(src, k, K);
    }
}

// ------------------------------------------------------------- the forms of the plan

typedef Q8Tile<256, 256, 2, 1, 2> Form0;
typedef Q8Tile<192, 256, 2, 1, 2> Form1;
typedef Q8Tile<128, 256, 2, 1, 3> Form2;
typedef Q8Tile<128, 128, 4, 1, 5> Form3;
typedef Q8Tile<64, 128, 4, 1, 3> Form4;
typedef Q8Tile<64, 64, 4, 2, 4> Form5;
// through registers
typedef Q8Tile<128, 128, 4, 1, 2, 3> FormR0;
typedef Q8Tile<64, 64, 4, 2, 2, 4> FormR1;

template <typename G>
constexpr bool is_form(int f) { return kForms[f].bm == G::BM && kForms[f].bn == G::BN; }
static_assert(is_form<Form0>(0) && is_form<Form1>(1) && is_form<Form2>(2) && is_form<Form3>(3) && is_form<Form4>(4) &&
              is_form<Form5>(5) && kNumForms == 6, "the plan's sizes are the kernels'");

// ------------------------------------------------------------- launches

inline bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <typename E, typename G>
hipError_t launch_form(const MatmulQ8& a, int ks, void* workspace, hipStream_t st) {
    const TileGrid g{(int)((a.T + G::BM - 1) / G::BM), (int)((a.N + G::BN - 1) / G::BN), ks, static_cast<int*>(workspace)};
    const unsigned wgs = (unsigned)(g.tm * g.tn * ks);
    const bool vec = a.N % Pack<E>::N == 0 && aligned_to(a.y, 16) && aligned_to(a.lora, 16);
    if constexpr (G::D == 0) {
        if (ks > 1) {
            q8_tiles<float, G, false, true><<<wgs, G::NTH, 0, st>>>(a, g);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            const unsigned blocks = (unsigned)((g.tm * g.tn * (G::NW / G::KG * G::MT) + 3) / 4);
            if (vec)
                q8_join<E, G, true><<<blocks, 256, 0, st>>>(a, g);
            else
                q8_join<E, G, false><<<blocks, 256, 0, st>>>(a, g);
            return hipGetLastError();
        }
    }
    if (vec)
        q8_tiles<E, G, true, false><<<wgs, G::NTH, 0, st>>>(a, g);
    else
        q8_tiles<E, G, false, false><<<wgs, G::NTH, 0, st>>>(a, g);
    return hipGetLastError();
}

template <typename E>
hipError_t launch_tiles(const MatmulQ8& a, const Q8Plan& p, void* workspace, hipStream_t st) {
    switch (p.form) {
        case 0: return launch_form<E, Form0>(a, p.ks, workspace, st);
        case 1: return launch_form<E, Form1>(a, p.ks, workspace, st);
        case 2: return launch_form<E, Form2>(a, p.ks, workspace, st);
        case 3: return launch_form<E, Form3>(a, p.ks, workspace, st);
        case 4: return launch_form<E, Form4>(a, p.ks, workspace, st);
        case 5: return launch_form<E, Form5>(a, p.ks, workspace, st);
        case kRegsBig: return launch_form<E, FormR0>(a, 1, workspace, st);
        default: return launch_form<E, FormR1>(a, 1, workspace, st);
    }
}

template <typename E>
hipError_t launch_piece(const MatmulQ8& a, void* workspace, hipStream_t st) {
    const bool dma = a.K % 4 == 0 && aligned_to(a.xq, 4) && aligned_to(a.wq, 4);
    const Q8Plan p = plan_q8(a.T, a.N, a.K, dma);
    if (p.form >= 0) return launch_tiles<E>(a, p, workspace, st);
    if (p.form == kPadded) {
        const PadPlan pad = plan_pad(a.T, a.N, a.K);
        int8_t* ws = static_cast<int8_t*>(workspace);
        MatmulQ8 b = a;
        b.K = padded(a.K);
        b.xq = ws;
        b.wq = ws + pad.w;
        const int64_t rows = a.T + a.N;
        q8_pad<<<(unsigned)(rows < (1 << 20) ? rows : 1 << 20), 256, 0, st>>>(a, (int)b.K, ws, ws + pad.w);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        return launch_tiles<E>(b, pad.plan, ws + pad.parts, st);
    }
    if (p.form == kOneToken) {
        q8_one_token<E><<<(unsigned)((a.N + kRows - 1) / kRows), kWaves * 64, 0, st>>>(a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.T + 15) / 16));
    if (dma)
        q8_direct<E, true><<<grid, kWaves * 64, 0, st>>>(a);
    else
        q8_direct<E, false><<<grid, kWaves * 64, 0, st>>>(a);
    return hipGetLastError();
}

template <typename E>
hipError_t launch_typed(const MatmulQ8& a, void* workspace, hipStream_t st) {
    MatmulQ8 b = a;
    for (int64_t t = 0; t < a.T; t += kPieceTokens) {
        b.T = a.T - t < kPieceTokens ? a.T - t : kPieceTokens;
        b.xq = a.xq + t * a.K;
        b.xs = a.xs + t;
        b.lora = a.lora ? static_cast<const E*>(a.lora) + t * a.N : nullptr;
        b.y = static_cast<E*>(a.y) + t * a.N;
        const hipError_t e = launch_piece<E>(b, workspace, st);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t matmul_q8_workspace_bytes(int64_t T, int64_t N, int64_t K) { return q8_workspace_bytes(T, N, K); }

hipError_t launch_matmul_q8(const MatmulQ8& a, int dtype, void* workspace, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    switch (dtype) {
        case kF32: return launch_typed<float>(a, workspace, stream);
        case kBF16: return launch_typed<bf16_t>(a, workspace, stream);
        default: return launch_typed<f16_t>(a, workspace, stream);
    }
}

}  // namespace dora
