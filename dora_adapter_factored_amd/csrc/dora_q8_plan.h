// The choice of a form for an 8-bit product, and the workspace that it needs.
//
// Plain host code: the library and a host compiler alone can build it, so the
// choice is checked without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace dora {

// The tile forms, by what they cost: a workgroup's time per k-tile in ns where
// it has the chip nearly to itself and where `slots` of them fill it (two of
// the small ones fit a CU; up to one a CU they do not slow each other).
// Measured on MI355X at K = 8192, T = 64 .. 2048, N = 4096 .. 28672.
struct Q8Form {
    int bm, bn, slots, ns_empty, ns_full;
};
constexpr Q8Form kForms[] = {
    {256, 256, 256, 1240, 1700}, {192, 256, 256, 1080, 1330}, {128, 256, 256, 740, 970},
    {128, 128, 256, 470, 660},   {64, 128, 512, 440, 780},    {64, 64, 512, 286, 520},
};
constexpr int kNumForms = sizeof(kForms) / sizeof(kForms[0]);
constexpr int kRegsBig = kNumForms, kRegsSmall = kNumForms + 1;   // 128 x 128 and 64 x 64 through registers

constexpr int kDirect = -1, kOneToken = -2, kPadded = -3;
constexpr int kMaxParts = 16;

struct Q8Plan {
    int form;   // a tile form, kDirect, kOneToken or kPadded
    int ks;     // parts of K
};

inline size_t plan_bytes(const Q8Plan& p, int64_t T, int64_t N) {   // of a tile form
    if (p.ks == 1) return 0;
    const Q8Form& f = kForms[p.form];
    return (size_t)((T + f.bm - 1) / f.bm) * ((N + f.bn - 1) / f.bn) * f.bm * f.bn * sizeof(int) * p.ks;
}

// The form and number of parts of least cost.  A round of workgroups costs its
// k-tiles; a launch about 5 us, of which the loads' first latency and the
// epilogue are most; parts that have to be joined one more launch (3 us, and
// for a short call as much again on the host: 4.5) and their bytes written and
// read again (0.23 us for each MB).  At 333 x 5120 x 27648 this takes 192 x 256
// tiles in 6 parts (73 us; 128 x 256 in 4 69, every form without parts over
// 92), at 2048 x 5120 x 5120 192 x 256 tiles (58 us; 256 x 256 67, 128 x 256
// 81), at 512 x 8192 x 8192 128 x 128 (45 us; 128 x 256 in 2 parts 49, 64 x 128
// 55).
inline int64_t cost_q8(int form, int ks, int64_t T, int64_t N, int64_t K) {
    const Q8Form& f = kForms[form];
    const int64_t wgs = ((T + f.bm - 1) / f.bm) * ((N + f.bn - 1) / f.bn) * ks, nk = ((K + 127) / 128 + ks - 1) / ks;
    const int64_t full = wgs / f.slots, rest = wgs % f.slots;
    int64_t ns = full * f.ns_full;
    if (rest > 0) ns += f.slots > 256 ? (rest > 256 ? f.ns_full : f.ns_empty) : f.ns_empty + (f.ns_full - f.ns_empty) * rest / 256;
    ns *= nk;
    const int64_t read = N * K / 6300;   // the weight at 6.3 TB/s
    ns = 5000 + (ns > read ? ns : read);
    if (ks > 1) ns += 4500 + (int64_t)plan_bytes({form, ks}, T, N) / 4400;
    return ns;
}

// 16 channels and tokens a workgroup straight from memory: what a CU's
// workgroups read at 22.5 GB/s, more with x's rows.
inline int64_t cost_direct(int64_t T, int64_t N, int64_t K) {
    const int64_t rounds = ((N + 15) / 16 * ((T + 15) / 16) + 255) / 256, t = T < 16 ? T : 16;
    return 2500 + rounds * 16 * K * (420 + t * t) / 420 * 2 / 45;
}

// The same for rows that are not 4-byte aligned, by whole dwords: 13.3 GB/s a
// CU at one token, 9.1 at 16.
inline int64_t cost_direct_odd(int64_t T, int64_t N, int64_t K) {
    const int64_t rounds = ((N + 15) / 16 * ((T + 15) / 16) + 255) / 256, t = T < 16 ? T : 16;
    return 2500 + rounds * 16 * K * (28 + t) / 400;
}

// The tile form and parts of least cost.
inline int64_t plan_tiles(int64_t T, int64_t N, int64_t K, Q8Plan& best) {
    int64_t least = INT64_MAX;
    for (int f = 0; f < kNumForms; ++f)
        for (int ks = 1; ks <= kMaxParts && ks * 2 <= (K + 127) / 128 + 1; ++ks) {
            // parts are for tiles that leave CUs idle
            if (ks > 1 && ((T + kForms[f].bm - 1) / kForms[f].bm) * ((N + kForms[f].bn - 1) / kForms[f].bn) * ks > kForms[f].slots * 2) break;
            const int64_t c = cost_q8(f, ks, T, N, K);
            if (c < least) {
                least = c;
                best = {f, ks};
            }
        }
    return least;
}

inline int64_t padded(int64_t K) { return (K + 15) / 16 * 16; }

inline size_t round_up_256(size_t x) { return (x + 255) / 256 * 256; }

inline Q8Plan make_plan_q8(int64_t T, int64_t N, int64_t K, bool dma) {
    if (T == 1) return {kOneToken, 1};
    if (K < 16) return {kDirect, 1};
    Q8Plan best{kDirect, 1};
    if (dma) {
        const int64_t tiles = plan_tiles(T, N, K, best);
        return T <= 16 && cost_direct(T, N, K) <= tiles ? Q8Plan{kDirect, 1} : best;
    }
    // Rows that are not 4-byte aligned, by rounds of 256 workgroups: 64 x 64
    // tiles through registers cost 0.43 us a k-tile, 128 x 128 1.22.  Up to 64
    // tokens may go straight from memory.  Where d_in is no multiple of 4, rows
    // may be padded to 16 bytes first, for a launch and their bytes both ways
    // (written at 5.3 TB/s, and read again in part from the MALL).  Measured, GPU
    // time with weights that are not in the MALL, straight / padded / 64 x 64 /
    // 128 x 128 in us: 24 x 5120 x 27649 149 / 80 / 98 / 210, 64 x 300 x 1001
    // 4.3 / 9.2 / 8.8 / 16, 64 x 4099 x 4099 30 / 21 / 19 / 36, 64 x 8193 x 8193
    // 113 / 45 / 45 / 81, 333 x 8193 x 8193 - / 71 / 116 / 86, 1000 x 515 x 16385
    // - / 35 / 54 / 128, 100 x 28673 x 2049 - / 46 / 46 / 34, 2000 x 4099 x 4099
    // - / 68 / 128 / 121.  Over 266 such sizes the form that this takes is 0.4% slower
    // than the fastest one in the mean, and 18% at most.
    auto rounds = [&](int64_t b) { return (((T + b - 1) / b) * ((N + b - 1) / b) + 255) / 256; };
    const int64_t nk = (K + 127) / 128, small = 5000 + rounds(64) * 430 * nk, big = 5000 + rounds(128) * 1220 * nk;
    const int64_t direct = T <= 64 ? cost_direct_odd(T, N, K) : INT64_MAX;
    const int64_t pad = K % 4 == 0 ? INT64_MAX : 4500 + (T + N) * 2 * K / 6000 + plan_tiles(T, N, padded(K), best);
    if (pad < direct && pad < small && pad < big) return {kPadded, 1};
    return {direct < small && direct < big ? kDirect : small <= big ? kRegsSmall : kRegsBig, 1};
}

// A call asks twice, for its workspace's size and for the launch: the thread's
// last plan is kept (making one takes 0.3 to 0.7 us at few tokens).
inline Q8Plan plan_q8(int64_t T, int64_t N, int64_t K, bool dma) {
    struct Last {
        int64_t T, N, K;
        bool dma;
        Q8Plan plan;
    };
    static thread_local Last last{0, 0, 0, false, {kDirect, 1}};   // T is never 0
    if (last.T != T || last.N != N || last.K != K || last.dma != dma) last = {T, N, K, dma, make_plan_q8(T, N, K, dma)};
    return last.plan;
}

// Workspace of a padded product: x's rows, w's rows, and what their product needs.
struct PadPlan {
    Q8Plan plan;
    size_t w, parts, bytes;   // offsets, and all
};

inline PadPlan plan_pad(int64_t T, int64_t N, int64_t K) {
    PadPlan p;
    const int64_t Kp = padded(K);
    plan_tiles(T, N, Kp, p.plan);
    p.w = round_up_256((size_t)(T * Kp));
    p.parts = p.w + round_up_256((size_t)(N * Kp));
    p.bytes = p.parts + plan_bytes(p.plan, T, N);
    return p;
}

// Tokens of one launch: a grid has at most 65535 rows (16 tokens each straight
// from memory), and with at most 2^24 channels its threads stay below 2^32.
constexpr int64_t kPieceTokens = (int64_t)1 << 19;

inline size_t q8_workspace_bytes(int64_t T, int64_t N, int64_t K) {
    // the largest of the pieces'; of d_in that is a multiple of 4 only codes at
    // 4-byte aligned addresses need any, which is known at the call
    size_t most = 0;
    const int64_t pieces[2] = {T < kPieceTokens ? T : kPieceTokens, T % kPieceTokens};
    for (int64_t t : pieces) {
        if (t == 0) continue;
        const Q8Plan p = plan_q8(t, N, K, K % 4 == 0);
        const size_t b = p.form == kPadded ? plan_pad(t, N, K).bytes : p.form >= 0 ? plan_bytes(p, t, N) : 0;
        most = b > most ? b : most;
    }
    return round_up_256(most);
}

}  // namespace dora
