// attend_kernel.h -- attention of drafted blocks over the paged 4-bit cache, for
// MI355X (gfx950): the kernels, how their work is cut, and the host side of a
// call. Included by the entry points' files, which differ in what a row sees
// (Mode) and are compiled apart. Internal.
//
// The mathematics: row (t, h) of request b, t <= k_b, stands at position
// p = ctx_b + t and sees the positions j of [max(0, p - window + 1), p]:
//   o = sum_j 2^(z_j - m) v_j / sum_j 2^(z_j - m),  z_j = scale log2(e) q . k_j,
// over one pass, the reference m and the sums held in fp32. m is a maximum that
// lags behind: it follows the running one when a term would exceed 2^8, so the
// weights 2^(z - m) lie in [0, 2^8]. Keys and values are decoded to bf16 (exact);
// products accumulate in fp32 on the matrix cores. The weights are rounded to
// bf16 for the value product (at most 2^-8 relative each, the size of the
// output's own rounding: with it outputs are 2.3e-3 of their norm off, without
// it 1.7e-3); their sum is taken before that rounding.
//
// Layout: a wavefront takes tiles of 32 tokens of one kv head and all query
// rows that share it (up to 16 kMT rows of (t, head in the group), in
// registers). Scores are computed transposed, K Q^T, so that a lane holds one
// query row (lane % 16) and tokens {16 half + 4 (lane / 16) + r}: the row's
// statistics stay within 4 lanes, the probabilities are already the right
// operand of V^T P^T (whose contraction runs over tokens in that same order),
// and the accumulators' rescale is a per-lane factor. The cache's tile layout
// gives every lane its codes in 16-byte loads in these orders.
//
// What bounds it is the latency of a tile's loads and the work on the tile
// before, two wavefronts a SIMD: about 1.5 us a tile and wavefront, 6 TB/s with
// all of them in the loop, 54 % of a wavefront's time spent waiting. 128 blocks of
// 3..9 rows x 4 heads over 1,024..8,192 tokens (8 kv heads of 128): 155 us, 4.2
// TB/s, the join's 13 in it, and 197 with 9 rows each; single tokens over the same
// contexts 129; one block of 5 over 131,071 tokens 41; 64 blocks under a window of
// 1,024 (8 kv heads of 256) 33. 64 blocks over 2,000..4,000 tokens, 8 kv heads:
// 64 rows of 128 channels 101 us, 2.0 TB/s (that kernel spills 67 registers, six
// reloads in its loop over pairs of tiles), 48 rows of 64 channels 50, 2.1 TB/s.
#pragma once

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "cache_tile.h"
#include "lds_dma.h"

namespace {

using namespace svcache;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) unsigned u32x4;

// What a row sees of the positions up to its own: those of a window, or also some
// sinks in front of it; or, as partial results that are joined elsewhere, those
// behind a shared prefix.
enum Mode { kWindow, kSinks, kTail };

constexpr int kFew = 4, kMany = 8;      // wavefronts of a workgroup (see plan_of)
constexpr float kNegInf = -INFINITY;

// How the work is cut. A unit is a request's kv head and block of 16 kMT
// rows, its cost the tiles times (kTileCost plus their row tiles; measured
// times per tile grow like that, one unit about 0.05 us). Three cuts:
//  - direct: a workgroup per unit and nothing to join, where rows see at most
//    kDirectTiles tiles, or twice that if every workgroup that is resident at
//    once has a unit (searching and joining, about 8 us, would cost more: 64
//    requests under a window of 1,024 tokens 41 against 34 us; measured there
//    only), or kDirectTiles for each of kDirectUnits and more units that it has:
//    then they even out by themselves, even if one request is as long as the
//    page table allows and the others are short. (512 requests of 256..4,096
//    tokens, 2 rows x 3 heads of 128: 228 us direct, 244 cut; heads of 64 195
//    and 216; 18 rows of 256 channels, 128 requests of 2,016 tokens 175 and 173.
//    But one request of 131,000 tokens among 127 of 1,000 takes 1,815 us direct
//    and 195 cut, among 511 897 and 159: under page tables wider than that a
//    batch of many even requests pays the cut's 2 to 11 %.)
// Else the lengths, which are on the device, decide. Every workgroup adds up
// the requests for itself and finds its place by a prefix sum. With `groups`
// workgroups resident at once and share = (cost of all units) / groups:
//  - aligned: every unit is cut into round(cost / share) equal parts, at least
//    one, and a workgroup takes one part; if the longest part is no more than
//    kSlack over the share, about what the line's extra runs cost.
//  - line: all units lie on one line, each led by a stretch of kUnitCost for
//    starting and ending it, and each of `groups` workgroups takes an equal
//    stretch, so that ragged lengths and budgets load the chip evenly.
// Parts of a unit are put together by the join kernel.
constexpr int kTileCost = 5;
constexpr int kUnitCost = 120;
constexpr int kSlack = 400;
constexpr int kLeastShare = 48;     // a few tiles for each of a workgroup's wavefronts
constexpr int kDirectTiles = 32;
constexpr int kDirectUnits = 4;

struct AttendArgs {
    const uint16_t* q;
    long long q_stride;
    const uint8_t* cache;
    const int32_t* ctx_lens;
    const int32_t* budgets;
    uint16_t* out;
    int32_t* status;
    float* part_o;      // [slot][16 kMT rows][D], not normalised
    float2* part_ml;    // [slot][16 kMT rows]: reference exponent, sum
    int4* parts;        // [workgroup][2]: unit, its parts, which one this is, first slot (see slot_of)
    Pages pages;
    int B, K, Hq, group;
    int groups;         // workgroups resident at once
    int row_blocks;     // blocks of 16 kMT rows of a full block's (K + 1) group rows
    int window;
    int sinks;          // kSinks: positions that stay visible in front of the window
    const int* skip;    // kTail: [B], tiles of each request that are not its own
    int2* units;        // kTail: [unit]: first slot (see slot_of) and parts
    int whole;          // kTail: the slot of unit 0, for units that are not cut
    bool direct;        // a workgroup per unit
    bool negate;        // scale < 0: queries are negated and |scale| is used
    float c;            // |scale| * log2(e)
};

// A request's block, and in kTail where its own tokens start.
template <Mode kMode>
struct Req : Block {};
template <>
struct Req<kTail> : Block {
    int tiles;          // of the shared prefix
};

// The tiles a request's block reads: [first, end), by numbers that are the tiles'
// own but in front of the window's whole tiles (see SinkTiles).
struct Span {
    int first, end;
    __device__ __forceinline__ int size() const { return end - first; }
};

// The first tile of the window, and the first that every row sees whole.
__device__ __forceinline__ int window_first(const Block& blk, int window) {
    return (window > 0 ? max(0, blk.ctx - window + 1) : 0) / kTile;
}
__device__ __forceinline__ int window_whole(const Block& blk, int window) {
    const int all_lo = window > 0 ? max(0, blk.ctx + blk.len - window) : 0;
    return (all_lo + kTile - 1) / kTile;
}

// The tiles in front of the window that hold sinks, and how they are numbered:
// a run takes tiles that some row does not see whole first, so the tile that
// sinks fill in part comes before the window's low edge, and the whole ones
// between that edge and the window's whole tiles, which keep their numbers:
//   [part][low edge][whole sinks][whole tiles of the window ...
struct SinkTiles {
    int whole, part;        // whole tiles of sinks; 1 if one more holds some
    int low, mid;           // first tile of the window, its first whole tile
    __device__ __forceinline__ SinkTiles(const Block& blk, int window, int sinks)
        : low(window_first(blk, window)), mid(window_whole(blk, window)) {
        whole = min(sinks / kTile, low);
        part = whole < low && sinks % kTile != 0 ? 1 : 0;
    }
    // The tile of number n.
    __device__ __forceinline__ int tile(int n) const {
        return n >= mid ? n : n >= mid - whole ? n - (mid - whole) : n >= low - whole ? n + whole : whole;
    }
};

template <Mode kMode>
__device__ __forceinline__ Span span_of(const Req<kMode>& blk, const AttendArgs& a) {
    const int end = (blk.ctx + blk.len + kTile - 1) / kTile;
    if constexpr (kMode == kTail) return Span{min(blk.tiles, end), end};
    if constexpr (kMode == kSinks) {
        const SinkTiles s(blk, a.window, a.sinks);
        return Span{s.low - s.whole - s.part, end};
    }
    return Span{window_first(blk, a.window), end};
}

// Whether a row at position p sees position j, as far as the window goes.
template <Mode kMode>
__device__ __forceinline__ bool in_window(const AttendArgs& a, int j, int p) {
    return a.window == 0 || j > p - a.window || (kMode == kSinks && j < a.sinks);
}

// A run of one unit's tiles: [t0, t1) of (b, h, row block rb); slot: where its
// partial result goes, or -1 when the run is the whole unit.
struct Work {
    int b, h, rb, t0, t1, slot;
};

// Slot of part i of a unit whose first part has slot `first`. On the line a
// workgroup g may end one unit (slot 2 g) and start another (slot 2 g + 1);
// aligned parts follow each other (first >= 0 there, ~first on the line).
__device__ __forceinline__ int slot_of(int first, int i) {
    return first >= 0 ? first + i : ~first + (i > 0 ? 2 * i - 1 : 0);
}

__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
    bf16x2 v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(unsigned, v);
}

// A value that is the same in every lane, as a scalar.
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ unsigned long long scalar(unsigned long long v) {
    return (unsigned long long)(unsigned)scalar((int)(v >> 32)) << 32 | (unsigned)scalar((int)v);
}
template <Mode kMode>
__device__ __forceinline__ Req<kMode> scalar(const Req<kMode>& k) {
    Req<kMode> r;
    r.ctx = scalar(k.ctx);
    r.len = scalar(k.len);
    if constexpr (kMode == kTail) r.tiles = scalar(k.tiles);
    return r;
}

// Maximum / sum over the four lanes that hold the same row (lane ^ 16, ^ 32).
__device__ __forceinline__ float quad_max(float v) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// A tile's bytes as one lane holds them.
template <int D>
struct Frag {
    using L = Tile<D>;
    unsigned k[L::kPlanes][2][L::U / 4];        // plane, half: a token's unit of channels
    unsigned v[L::kPlanes][2][L::C];            // plane, half: 4 tokens' pieces
    unsigned ks[L::kPlanes];                    // key scales of both halves
    unsigned vs[L::kPlanes][2];                 // value scales of 4 + 4 tokens

    // The tile is the same for the whole wavefront: one scalar base, a 32-bit
    // offset per lane.
    __device__ __forceinline__ void load(const uint8_t* tile, unsigned lane) {
        const unsigned x = lane & 15, quad = lane >> 4;
        #pragma unroll
        for (int p = 0; p < L::kPlanes; ++p) {
            #pragma unroll
            for (int half = 0; half < 2; ++half) {
                __builtin_memcpy(k[p][half], __builtin_assume_aligned(
                    tile + (half * 8 * D + p * 64 * L::U) + lane * L::U, L::U), L::U);
                __builtin_memcpy(v[p][half], __builtin_assume_aligned(
                    tile + (L::kVCodes + (p * 2 + half) * 256 * L::C) + lane * (4 * L::C), 4 * L::C), 4 * L::C);
            }
            const unsigned kg = D == 64 ? quad >> 1 : quad, vg = D == 64 ? x >> 3 : x >> 2;
            ks[p] = *reinterpret_cast<const uint16_t*>(tile + (L::kKScales + p * 128) + (kg * 32 + x * 2));
            __builtin_memcpy(vs[p], __builtin_assume_aligned(
                tile + (L::kVScales + p * 128) + (vg * 4 + quad) * 8, 8), 8);
        }
    }
};

// Registers of one wavefront over its tiles, for kAct row tiles.
template <int D, int kAct>
struct State {
    using L = Tile<D>;
    static constexpr int kPlanes = L::kPlanes;
    static constexpr int kUnitSteps = D == 64 ? 2 : 4;  // products of 32 channels in a key unit
    static constexpr int kSteps = D / 32;
    static constexpr int kChans = D == 64 ? 4 : 8;      // channels of a value piece
    f32x4 o[kAct][kPlanes][kChans];
    float ref[kAct];     // reference of the exponents; -inf: nothing seen
    float sum[kAct];     // this lane's share of the row's sum
    int pos[kAct];       // the row's position; -1 past the block
};

template <int D, int kMT, int kWaves>
struct Lds {
    static constexpr int kPieces = kMT * Tile<D>::kPlanes * (D == 64 ? 4 : 8) / 4;  // float4 per lane and component
    union {
        u32x4 q[kMT][D / 32][64];           // right operands of K Q^T
        f32x4 o[kWaves][2][kPieces][64];    // two components of the accumulators at a time
    };
    float ref[kWaves][kMT][16];
    float sum[kWaves][kMT][16];
    unsigned long long cost[kWaves], scan[kWaves], before;
    unsigned units[kWaves], longest[kWaves];
    int found;
};

// One tile. kMasked: some row does not see some token of it; positions outside
// [first, last] no row sees (but for sinks).
template <int D, int kMT, int kWaves, int kAct, Mode kMode, bool kMasked>
__device__ __forceinline__ void tile_step(State<D, kAct>& st, const Frag<D>& f,
                                          const Lds<D, kMT, kWaves>& sh, const AttendArgs& a, int lane,
                                          int tok0, int first, int last, const uint8_t* tile) {
    using L = Tile<D>;
    using S = State<D, kAct>;
    // These accumulators leave no registers for steps that overlap (D = 256, of
    // as many, has one wave per SIMD and so twice the registers).
    constexpr bool kTight = D == 128 && kAct == 4;
    // Opaque: the masks' token numbers are computed here, not kept in
    // registers throughout the loop over tiles.
    if (kMasked) asm volatile("" : "+v"(lane));
    const int quad = lane >> 4;
    // Scores of 2 x 16 tokens (lane: tokens 16 half + 4 quad + r).
    f32x4 z[kAct][2] = {};
    #pragma unroll
    for (int p = 0; p < S::kPlanes; ++p) {
        const float s[2] = {scale_of(f.ks[p] & 255u), scale_of(f.ks[p] >> 8)};
        #pragma unroll
        for (int j = 0; j < S::kUnitSteps; ++j) {
            if (kTight) __builtin_amdgcn_sched_barrier(0);
            bf16x8 kf[2];
            #pragma unroll
            for (int half = 0; half < 2; ++half) {
                const unsigned w = f.k[p][half][j];
                const u32x4 kw = {decode2<0>(w, s[half]), decode2<1>(w, s[half]),
                                  decode2<2>(w, s[half]), decode2<3>(w, s[half])};
                kf[half] = __builtin_bit_cast(bf16x8, kw);
            }
            #pragma unroll
            for (int mt = 0; mt < kAct; ++mt) {
                const bf16x8 qf = __builtin_bit_cast(bf16x8, sh.q[mt][p * S::kUnitSteps + j][lane]);
                #pragma unroll
                for (int half = 0; half < 2; ++half) {
                    z[mt][half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[half], qf, z[mt][half], 0, 0, 0);
                }
            }
        }
    }

    // Probabilities 2^(c z - ref). The reference follows the running maximum
    // only when a term exceeds 2^8: until then nothing has to be rescaled.
    if (kTight) __builtin_amdgcn_sched_barrier(0);
    bf16x8 pf[kAct];
    #pragma unroll
    for (int mt = 0; mt < kAct; ++mt) {
        if (kMasked) {
            const int lo = a.window > 0 ? st.pos[mt] - a.window : -1;
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = tok0 + 16 * (i >> 2) + 4 * quad + (i & 3);
                if (j > st.pos[mt] || (j <= lo && !(kMode == kSinks && j < a.sinks))) z[mt][i >> 2][i & 3] = kNegInf;
            }
        }
        // A row that has seen nothing yet has reference 0 here; what it does
        // not see is 2^(-inf) = 0.
        const bool fresh = st.ref[mt] == kNegInf;
        const float ref = fresh ? 0.0f : st.ref[mt];
        float s[8];
        #pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = __builtin_fmaf(z[mt][i >> 2][i & 3], a.c, -ref);
        float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])),
                          fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
        if (__ballot(top > (fresh ? kNegInf : 8.0f)) != 0) {
            // The four lanes of a row share its reference.
            top = quad_max(top);
            const float next = fresh ? top : fmaxf(ref, ref + top);
            const float keep = fresh ? 0.0f : exp2_fast(ref - next);
            const float off = next == kNegInf ? 0.0f : next;
            st.ref[mt] = next;
            st.sum[mt] *= keep;
            #pragma unroll
            for (int p = 0; p < S::kPlanes; ++p) {
                #pragma unroll
                for (int j = 0; j < S::kChans; ++j) st.o[mt][p][j] *= keep;
            }
            #pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = __builtin_fmaf(z[mt][i >> 2][i & 3], a.c, -off);
        }
        #pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = exp2_fast(s[i]);
        st.sum[mt] += ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
        const u32x4 pw = {pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]),
                          pack_bf16(s[6], s[7])};
        pf[mt] = __builtin_bit_cast(bf16x8, pw);
    }

    // Values: 8 tokens (4 quad + r of both halves) x kChans channels a plane.
    #pragma unroll
    for (int p = 0; p < S::kPlanes; ++p) {
        unsigned w[8];
        float vs[8];
        bool poison = false;
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int half = i >> 2, r = i & 3;
            if constexpr (D == 64) {
                w[i] = r & 1 ? f.v[p][half][r >> 1] >> 16 : f.v[p][half][r >> 1];
            } else {
                w[i] = f.v[p][half][r];
            }
            const unsigned sc = f.vs[p][half];
            unsigned bits = (r == 3 ? sc >> 1 : sc << (23 - 8 * r)) & 0x7f800000u;
            if (kMasked) {
                // What some row does not see must not reach it as 0 * NaN or
                // 0 * infinity: positions past the block and in front of every
                // row's window hold anything and are cleared; NaN groups of
                // tokens that other rows see are cleared here and put into
                // those rows below.
                const int j = tok0 + 16 * half + 4 * quad + r;
                const bool nan = bits == 0x7f800000u, some = (j >= first || (kMode == kSinks && j < a.sinks)) && j <= last;
                poison |= nan && some;
                if (nan || !some) {
                    bits = 0x3f800000u;
                    w[i] = 0;
                }
            }
            vs[i] = __uint_as_float(bits);
        }
        #pragma unroll
        for (int cb = 0; cb < S::kChans / 2; ++cb) {
            if (kTight) __builtin_amdgcn_sched_barrier(0);
            unsigned e[8];
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                e[i] = cb == 0   ? decode2<0>(w[i], vs[i])
                       : cb == 1 ? decode2<1>(w[i], vs[i])
                       : cb == 2 ? decode2<2>(w[i], vs[i])
                                 : decode2<3>(w[i], vs[i]);
            }
            u32x4 even, odd;
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                even[i] = __builtin_amdgcn_perm(e[2 * i + 1], e[2 * i], 0x05040100u);
                odd[i] = __builtin_amdgcn_perm(e[2 * i + 1], e[2 * i], 0x07060302u);
            }
            #pragma unroll
            for (int mt = 0; mt < kAct; ++mt) {
                st.o[mt][p][2 * cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, even), pf[mt], st.o[mt][p][2 * cb], 0, 0, 0);
                st.o[mt][p][2 * cb + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, odd), pf[mt], st.o[mt][p][2 * cb + 1], 0, 0, 0);
            }
        }
        if (kMasked && __ballot(poison) != 0) {
            // The accumulators of this lane hold channels of one group of each
            // plane (pieces 4 quad + r): NaN for the rows that see a NaN token
            // of that group.
            const int og = D == 64 ? quad >> 1 : p * 4 + quad;
            for (int tok = 0; tok < kTile; ++tok) {
                const int j = tok0 + tok;
                const bool nan = j <= last && tile[L::v_scale(tok, og)] == 255u;
                #pragma unroll
                for (int mt = 0; mt < kAct; ++mt) {
                    const bool seen = j <= st.pos[mt] && in_window<kMode>(a, j, st.pos[mt]);
                    const float add = nan && seen ? NAN : 0.0f;
                    #pragma unroll
                    for (int c = 0; c < S::kChans; ++c) st.o[mt][p][c] += add;
                }
            }
        }
    }
}

// This wavefront's share of a run: of the run's tiles, those that some row
// does not see whole first (the block's own, the windows' edges), then the
// others, every kWaves-th by number n = 0, 1, ... The next tile's bytes are asked
// for before one is worked on. Of the whole tiles only every other one's stay in
// flight meanwhile: the second load of a pair is conditional, and where its two
// paths meet the compiler waits for all of it but the last piece. (Two tiles
// ahead, or a ring in LDS filled by buffer-to-LDS loads, measured slower: 174-186
// against 153 us for 128 requests over 1,024..8,192 tokens.)
template <int D, int kMT, int kWaves, Mode kMode>
struct Stream {
    using L = Tile<D>;
    Frag<D> f[2];
    int wave, first, low, u0, u1, edges, count;     // tiles [u0, u1) are seen whole by every row
    SinkTiles sinks;
    // Page numbers of the next 64 tiles, one a lane. They come in one load: 157 us
    // for 128 requests over 1,024..8,192 tokens, 192 with a lookup per tile. (As
    // that load is conditional, taking a number out of the register still waits
    // for the loads before it.)
    int pages;
    bool bad;               // a page was outside the pool

    __device__ __forceinline__ Stream(const AttendArgs& a, const Block& blk)
        : sinks(blk, a.window, kMode == kSinks ? a.sinks : 0) {}
    __device__ __forceinline__ int tile_of(int n) const {
        const int i = wave + n * kWaves;
        const int tile = i < low ? first + i : i < edges ? u1 + (i - low) : u0 + (i - edges);
        return kMode == kSinks ? sinks.tile(tile) : tile;
    }
    // No branch in the loops over tiles depends on the lane: where one does,
    // the compiler may keep a second set of accumulators.
    template <int i>
    __device__ __forceinline__ const uint8_t* fetch(const AttendArgs& a, const Work& wk, int n, int lane) {
        if ((n & 63) == 0) {
            pages = a.pages.page(wk.b, tile_of(min(n + lane, count - 1)) * kTile);
        }
        long long at = a.pages.tile_in(__builtin_amdgcn_readlane(pages, n & 63), wk.h,
                                       tile_of(n) * kTile, L::kBytes);
        // The first tile of the cache stands in for one whose page is bad (the
        // request is flagged and its outputs are undefined).
        if (at < 0) {
            bad = true;
            at = 0;
        }
        const uint8_t* tile = a.cache + at;
        f[i].load(tile, lane);
        return tile;
    }
    __device__ __forceinline__ const uint8_t* start(const AttendArgs& a, const Work& wk,
                                                    const Block& blk, int lane, int its_wave) {
        wave = its_wave;
        // Tokens that every row of the block sees: from the window's first whole
        // tile to ctx, and whole tiles of sinks.
        first = wk.t0;
        const int whole = window_whole(blk, a.window), end = (blk.ctx + 1) / kTile;
        u0 = min(max(wk.t0, kMode == kSinks ? whole - sinks.whole : whole), wk.t1);
        u1 = max(u0, min(wk.t1, kMode == kSinks ? max(end, whole) : end));
        low = u0 - wk.t0;
        edges = low + wk.t1 - u1;
        count = (wk.t1 - wk.t0 - wave + kWaves - 1) / kWaves;
        bad = false;
        return count > 0 ? fetch<0>(a, wk, 0, lane) : a.cache;
    }
    template <int kAct>
    __device__ __forceinline__ void run(State<D, kAct>& st, const Lds<D, kMT, kWaves>& sh,
                                        const AttendArgs& a, const Work& wk, const Block& blk,
                                        const uint8_t* tile, int lane) {
        const int lo = a.window > 0 ? max(0, blk.ctx - a.window + 1) : 0;
        int n = 0;
        for (; wave + n * kWaves < edges; ++n) {
            const uint8_t* next = tile;
            if (n + 1 < count) next = fetch<1>(a, wk, n + 1, lane);
            tile_step<D, kMT, kWaves, kAct, kMode, true>(st, f[0], sh, a, lane, tile_of(n) * kTile, lo, blk.ctx + blk.len - 1, tile);
            f[0] = f[1];
            tile = next;
        }
        while (n < count) {
            if (n + 1 < count) fetch<1>(a, wk, n + 1, lane);
            tile_step<D, kMT, kWaves, kAct, kMode, false>(st, f[0], sh, a, lane, 0, 0, 0, nullptr);
            if (n + 1 < count) {
                if (n + 2 < count) fetch<0>(a, wk, n + 2, lane);
                tile_step<D, kMT, kWaves, kAct, kMode, false>(st, f[1], sh, a, lane, 0, 0, 0, nullptr);
            }
            n += 2;
        }
    }
};

template <Mode kMode>
__device__ __forceinline__ Req<kMode> plain_block(const AttendArgs& a, int b) {
    Req<kMode> r;
    static_cast<Block&>(r) = block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, nullptr, false);
    if constexpr (kMode == kTail) r.tiles = r.len > 0 ? a.skip[b] : 0;
    return r;
}
// The same, where there may be no request.
template <Mode kMode>
__device__ __forceinline__ Req<kMode> plain_block(const AttendArgs& a, int b, bool some) {
    Req<kMode> none{};
    return some ? plain_block<kMode>(a, b) : none;
}

// A request's share of the line.
template <int kMT, Mode kMode>
struct Share {
    Req<kMode> blk;
    Span span;
    int rows, blocks;           // rows, row blocks that hold some
    __device__ __forceinline__ Share(const AttendArgs& a, const Req<kMode>& k)
        : blk(k), span(span_of<kMode>(k, a)), rows(k.len * a.group),
          blocks((rows + 16 * kMT - 1) / (16 * kMT)) {}
    // Row tiles of row block rb, and what one tile of its units costs.
    __device__ __forceinline__ int act(int rb) const { return min((rows - rb * 16 * kMT + 15) / 16, kMT); }
    __device__ __forceinline__ int cost(int rb) const { return kTileCost + act(rb); }
    // Parts of a unit when the cut is aligned: tiles / share, rounded, at
    // least 1 and at most one a tile.
    __device__ __forceinline__ int parts(int rb, int share) const {
        return min(max((tiles(rb) + share / 2) / share, 1), max(span.size(), 1));
    }
    // Cost of all tiles of a unit of row block rb.
    __device__ __forceinline__ int tiles(int rb) const { return span.size() * cost(rb); }
    // Sum over all the request's units of f(row block).
    template <typename F>
    __device__ __forceinline__ unsigned long long sum(int heads, F f) const {
        if (blk.len == 0) return 0;
        return (unsigned long long)heads * ((unsigned long long)(blocks - 1) * f(0) + f(blocks - 1));
    }
};

// Waves per SIMD that the registers leave room for.
template <int D, int kMT>
constexpr int occupancy() {
    return D == 256 ? 3 - kMT : D * kMT <= 64 ? 4 : D * kMT <= 128 ? 3 : 2;
}

// A sum of partial results under its running reference.
struct Joined {
    float ref, sum;
    f32x4 acc;
    __device__ __forceinline__ void add(float other_ref, float other_sum, const f32x4& other) {
        const float top = fmaxf(ref, other_ref), base = top == kNegInf ? 0.0f : top;
        const float f = exp2_fast(ref - base), g = exp2_fast(other_ref - base);
        sum = sum * f + other_sum * g;
        acc = acc * f + other * g;
        ref = top;
    }
};

// One run of tiles, from the queries to the output or a partial result, for a
// row block of which kAct row tiles hold rows.
template <int D, int kMT, int kWaves, int kAct, Mode kMode>
__device__ __forceinline__ void attend_run(const AttendArgs& a, const Work& any, const Req<kMode>& its,
                                           Lds<D, kMT, kWaves>& sh, int lane, int wave) {
    // The same for the whole wavefront, and to be kept in scalar registers.
    const Work wk{scalar(any.b), scalar(any.h), scalar(any.rb), scalar(any.t0), scalar(any.t1), scalar(any.slot)};
    const Req<kMode> blk = scalar(its);
    using S = State<D, kAct>;
    constexpr int kPlanes = S::kPlanes, kChans = S::kChans, kPieces = kAct * kPlanes * kChans / 4;
    constexpr int kOwn = (kAct * S::kSteps + kWaves - 1) / kWaves;
    // Opaque: what derives from the lane is computed again for every run
    // rather than kept in registers across the loop over runs.
    asm volatile("" : "+v"(lane));
    const int x = lane & 15, quad = lane >> 4;
    const int rows = blk.len * a.group;

    // The queries as right operands: lane holds row x, 8 channels of its unit.
    u32x4 own[kOwn];
    #pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        const int i = k * kWaves + wave, mt = i / S::kSteps, s = i % S::kSteps;
        const int r = (wk.rb * kMT + mt) * 16 + x, t = r / a.group;
        own[k] = u32x4{0, 0, 0, 0};
        if (r < rows && mt < kAct) {
            const int ch = (s / S::kUnitSteps * 4 + quad) * (8 * S::kUnitSteps) + 8 * (s % S::kUnitSteps);
            own[k] = *reinterpret_cast<const u32x4*>(
                a.q + ((long long)wk.b * (a.K + 1) + t) * a.q_stride +
                (wk.h * a.group + (r - t * a.group)) * D + ch);
            if (a.negate) own[k] ^= u32x4{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
        }
    }
    Stream<D, kMT, kWaves, kMode> stream(a, blk);
    const uint8_t* tile = stream.start(a, wk, blk, lane, wave);
    S st;
    #pragma unroll
    for (int mt = 0; mt < kAct; ++mt) {
        const int r = (wk.rb * kMT + mt) * 16 + x;
        st.pos[mt] = r < rows ? blk.ctx + r / a.group : -1;
        st.ref[mt] = kNegInf;
        st.sum[mt] = 0.0f;
        #pragma unroll
        for (int p = 0; p < kPlanes; ++p) {
            #pragma unroll
            for (int j = 0; j < kChans; ++j) st.o[mt][p][j] = f32x4{0, 0, 0, 0};
        }
    }
    #pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        const int i = k * kWaves + wave;
        if (i < kAct * S::kSteps) sh.q[i / S::kSteps][i % S::kSteps][lane] = own[k];
    }
    svdma::ring_barrier();            // leaves the tiles in flight
    stream.run(st, sh, a, wk, blk, tile, lane);
    if (stream.bad && lane == 0) flag(a.status, SV_FLAG_BAD_PAGE);

    // Join the waves, two components of every accumulator in each of two
    // rounds; a wave adds up and writes every other piece of 4 channels of one.
    #pragma unroll
    for (int mt = 0; mt < kAct; ++mt) {
        const float sum = quad_sum(st.sum[mt]);
        if (quad == 0) {
            sh.ref[wave][mt][x] = st.ref[mt];
            sh.sum[wave][mt][x] = sum;
        }
    }
    svdma::ring_barrier();
    float total[kAct], top[kAct];
    #pragma unroll
    for (int mt = 0; mt < kAct; ++mt) {
        top[mt] = kNegInf;
        #pragma unroll
        for (int w = 0; w < kWaves; ++w) top[mt] = fmaxf(top[mt], sh.ref[w][mt][x]);
        const float ref = top[mt] == kNegInf ? 0.0f : top[mt];
        const float mine = exp2_fast(st.ref[mt] - ref);
        total[mt] = 0.0f;
        #pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            total[mt] += sh.sum[w][mt][x] * exp2_fast(sh.ref[w][mt][x] - ref);
        }
        #pragma unroll
        for (int p = 0; p < kPlanes; ++p) {
            #pragma unroll
            for (int j = 0; j < kChans; ++j) st.o[mt][p][j] *= mine;
        }
    }
    #pragma unroll
    for (int round = 0; round < 2; ++round) {
        #pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int mt = i / (kPieces / kAct), p = i / (kChans / 4) % kPlanes, c = i % (kChans / 4) * 4;
            #pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = 2 * round + k;
                sh.o[wave][k][i][lane] = f32x4{st.o[mt][p][c][r], st.o[mt][p][c + 1][r],
                                               st.o[mt][p][c + 2][r], st.o[mt][p][c + 3][r]};
            }
        }
        svdma::ring_barrier();
        const int k = wave & 1, m = 4 * quad + 2 * round + k;     // the lane's pieces of channels
        #pragma unroll
        for (int j = 0; j < (kPieces + kWaves / 2 - 1) / (kWaves / 2); ++j) {
            const int i = kWaves / 2 * j + (wave >> 1);
            if (i >= kPieces) continue;
            const int mt = i / (kPieces / kAct), p = i / (kChans / 4) % kPlanes, c = i % (kChans / 4) * 4;
            const int in = mt * 16 + x, row = wk.rb * (16 * kMT) + in;
            if (row >= rows) continue;
            f32x4 v = sh.o[0][k][i][lane] + sh.o[1][k][i][lane];
            #pragma unroll
            for (int w = 2; w < kWaves; w += 2) v += sh.o[w][k][i][lane] + sh.o[w + 1][k][i][lane];
            const int ch = p * 128 + m * kChans + c;
            // mt is the same for the whole wave but no constant.
            float sum = total[0], ref = top[0];
            #pragma unroll
            for (int n = 1; n < kAct; ++n) {
                sum = mt == n ? total[n] : sum;
                ref = mt == n ? top[n] : ref;
            }
            if (kMode != kTail && wk.slot < 0) {
                const int t = row / a.group;
                const float inv = 1.0f / sum;
                const unsigned w[2] = {pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv)};
                uint16_t* dst = a.out + (((long long)wk.b * (a.K + 1) + t) * a.Hq + wk.h * a.group +
                                         (row - t * a.group)) * D + ch;
                __builtin_memcpy(__builtin_assume_aligned(dst, 8), w, 8);
            } else {
                const long long part = (long long)wk.slot * (16 * kMT) + in;
                *reinterpret_cast<f32x4*>(a.part_o + part * D + ch) = v;
                if (ch == 0) a.part_ml[part] = make_float2(ref, sum);
            }
        }
        svdma::ring_barrier();
    }
}

// Workgroup g of `grid`.
template <int D, int kMT, int kWaves, Mode kMode>
__device__ __forceinline__ void attend_body(const AttendArgs& a, Lds<D, kMT, kWaves>& sh, int g, unsigned grid) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = scalar(tid >> 6);
    const int heads = a.pages.heads;

    if (g == 0) {                     // report bad budgets and lengths, once per call
        for (int b = tid; b < a.B; b += 64 * kWaves) {
            block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, a.status, true);
        }
    }
    // Where this workgroup is: unit (b, h, rb); on the line, its stretch
    // [lo, hi) and request b's first place; of an aligned unit, its part.
    int b = -1, h = 0, rb = 0, part = 0;
    unsigned long long at = 0, lo = 0, hi = 0, share = 1;
    bool aligned = false;
    Req<kMode> blk{};
    if (kWaves != kFew || a.direct) {
        rb = scalar(g % a.row_blocks);
        h = scalar(g / a.row_blocks % heads);
        const int mine = scalar(g / a.row_blocks / heads);
        blk = scalar(plain_block<kMode>(a, mine));
        if (rb < Share<kMT, kMode>(a, blk).blocks) b = mine;
    } else if constexpr (kWaves == kFew) {
        const int per = (a.B + 255) / 256;
        const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
        if (tid == 0) sh.found = -1;
        if (kMode != kTail && tid < 2) a.parts[2 * g + tid] = make_int4(0, 0, 0, 0);
        // The first of this thread's requests (the only one up to 256) is kept.
        const Share<kMT, kMode> first(a, plain_block<kMode>(a, b0, b0 < b1));
        unsigned long long cost = 0;
        unsigned units = 0;
        for (int i = b0; i < b1; ++i) {
            const Share<kMT, kMode> s = i == b0 ? first : Share<kMT, kMode>(a, plain_block<kMode>(a, i));
            cost += s.sum(heads, [&](int r) { return s.tiles(r); });
            units += s.blocks * heads;
        }
        #pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            cost += __shfl_xor(cost, o, 64);
            units += __shfl_xor(units, o, 64);
        }
        if (lane == 0) {
            sh.cost[wave] = cost;
            sh.units[wave] = units;
        }
        __syncthreads();
        cost = scalar((sh.cost[0] + sh.cost[1]) + (sh.cost[2] + sh.cost[3]));
        units = scalar((int)((sh.units[0] + sh.units[1]) + (sh.units[2] + sh.units[3])));
        share = scalar(max((cost + a.groups - 1) / a.groups, (unsigned long long)kLeastShare));
        // Aligned parts: no more than groups + units workgroups, which the
        // grid has room for or not.
        unsigned longest = 0;
        const int width = (int)min(share, 1ull << 30);
        for (int i = b0; i < b1; ++i) {
            const Share<kMT, kMode> s = i == b0 ? first : Share<kMT, kMode>(a, plain_block<kMode>(a, i));
            if (s.blocks > 0) longest = max(longest, (unsigned)(s.tiles(0) / s.parts(0, width)));
        }
        #pragma unroll
        for (int o = 1; o < 64; o <<= 1) longest = max(longest, (unsigned)__shfl_xor((int)longest, o, 64));
        if (lane == 0) sh.longest[wave] = longest;
        __syncthreads();
        longest = max(max(sh.longest[0], sh.longest[1]), max(sh.longest[2], sh.longest[3]));
        aligned = scalar((int)(a.groups + units <= grid && longest <= share + kSlack)) != 0;
        if (!aligned) {
            cost += (unsigned long long)units * kUnitCost;
            share = scalar(max((cost + a.groups - 1) / a.groups, (unsigned long long)kLeastShare));
        }
        auto length = [&](const Share<kMT, kMode>& s) {
            if (aligned) return s.sum(heads, [&](int r) { return s.parts(r, (int)share); });
            return s.sum(heads, [&](int r) { return kUnitCost + s.tiles(r); });
        };
        lo = aligned ? g : g * share;
        hi = aligned ? g + 1 : lo + share;
        unsigned long long mine = 0;
        for (int i = b0; i < b1; ++i) {
            mine += length(i == b0 ? first : Share<kMT, kMode>(a, plain_block<kMode>(a, i)));
        }
        unsigned long long upto = mine;
        #pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const unsigned long long u = __shfl_up(upto, o, 64);
            if (lane >= o) upto += u;
        }
        if (lane == 63) sh.scan[wave] = upto;
        __syncthreads();
        for (int w = 0; w < wave; ++w) upto += sh.scan[w];
        if (mine > 0 && upto - mine <= lo && lo < upto) {
            at = upto - mine;
            int i = b0;
            for (; i < b1 - 1; ++i) {
                const unsigned long long n = length(Share<kMT, kMode>(a, plain_block<kMode>(a, i)));
                if (lo < at + n) break;
                at += n;
            }
            sh.found = i;
            sh.before = at;
        }
        __syncthreads();
        b = scalar(sh.found);
        if (b >= 0 && (aligned || g < a.groups)) {
            at = scalar(sh.before);
            blk = scalar(plain_block<kMode>(a, b));
            if (aligned) {
                const Share<kMT, kMode> s(a, blk);
                const int full = heads * scalar(s.parts(0, (int)share));    // of a full row block
                part = (int)(lo - at);
                rb = scalar(min(part / full, s.blocks - 1));
                part -= rb * full;
                const int each = scalar(s.parts(rb, (int)share));
                h = scalar(part / each);
                part -= h * each;
            }
        } else {
            b = -1;
        }
    }

    while (b >= 0) {
        const Share<kMT, kMode> s(a, blk);
        const int unit = kUnitCost + s.tiles(rb), n = s.span.size();
        int i0 = 0, i1 = n, slot = -1;
        if (aligned) {
            const int parts = s.parts(rb, (int)share);
            i0 = (int)((long long)n * part / parts);
            i1 = (int)((long long)n * (part + 1) / parts);
            if (kMode == kTail || parts > 1) {
                slot = g;
                const int u = (b * heads + h) * a.row_blocks + rb;
                if (tid == 0) {
                    if (kMode != kTail) a.parts[2 * g] = make_int4(u, parts, part, g - part);
                    else if (part == 0) a.units[u] = make_int2(g, parts);
                }
            }
        } else if (!a.direct) {
            // Places relative to the unit's first tile; beyond it either way
            // is as good as 2^30.
            const unsigned cost = s.cost(rb);
            const long long start = (long long)(at + (unsigned long long)h * unit + kUnitCost);
            const int from = (int)min(max((long long)lo - start, -(1ll << 30)), 1ll << 30);
            const int to = (int)min(max((long long)hi - start, -(1ll << 30)), 1ll << 30);
            i0 = from > 0 ? min((int)((from + cost - 1) / cost), n) : 0;
            i1 = to > 0 ? min((int)((to + cost - 1) / cost), n) : 0;
            if (i0 < i1 && (i0 > 0 || i1 < n)) {
                slot = 2 * g + (i0 == 0);
                const unsigned width = (unsigned)min(share, 1ull << 31);
                const int before = from > 0 ? (int)((from + width - 1) / width) : 0;
                const int after = (int)((unsigned)((n - 1) * (int)cost - from) / width);
                if (tid == 0) {
                    const int u = (b * heads + h) * a.row_blocks + rb, from = ~(2 * (g - before) + 1);
                    if (kMode != kTail) a.parts[slot] = make_int4(u, before + after + 1, before, from);
                    else if (before == 0) a.units[u] = make_int2(from, after + 1);
                }
            }
        }
        if (kMode == kTail && slot < 0 && i0 < i1) {
            const int u = (b * heads + h) * a.row_blocks + rb;
            slot = a.whole + u;
            if (tid == 0) a.units[u] = make_int2(slot, 1);
        }
        if (i0 < i1) {
            const Work wk{b, h, rb, s.span.first + scalar(i0), s.span.first + scalar(i1), slot};
            const int act = scalar(s.act(rb));
            if (kMT >= 4 && act == 4) attend_run<D, kMT, kWaves, (kMT < 4 ? 1 : 4), kMode>(a, wk, blk, sh, lane, wave);
            else if (kMT >= 3 && act == 3) attend_run<D, kMT, kWaves, (kMT < 3 ? 1 : 3), kMode>(a, wk, blk, sh, lane, wave);
            else if (kMT >= 2 && act == 2) attend_run<D, kMT, kWaves, (kMT < 2 ? 1 : 2), kMode>(a, wk, blk, sh, lane, wave);
            else attend_run<D, kMT, kWaves, 1, kMode>(a, wk, blk, sh, lane, wave);
        }
        if (a.direct || aligned) break;
        // On to the next unit: heads, row blocks, requests.
        if (++h == heads) {
            at += (unsigned long long)heads * unit;
            h = 0;
            if (++rb == s.blocks) {
                rb = 0;
                int next = b + 1;
                b = -1;
                for (; next < a.B && b < 0; next += 64) {     // the next request that holds anything
                    const Req<kMode> k = plain_block<kMode>(a, next + lane, next + lane < a.B);
                    const unsigned long long some = __ballot(k.len > 0);
                    if (some != 0) {
                        const int i = __builtin_ctzll(some);
                        b = next + i;
                        blk.ctx = __builtin_amdgcn_readlane(k.ctx, i);
                        blk.len = __builtin_amdgcn_readlane(k.len, i);
                        if constexpr (kMode == kTail) blk.tiles = __builtin_amdgcn_readlane(k.tiles, i);
                    }
                }
            }
        }
        if (b >= 0 && at + (unsigned long long)h * (kUnitCost + Share<kMT, kMode>(a, blk).tiles(rb)) >= hi) b = -1;
    }
}

template <int D, int kMT, int kWaves, Mode kMode>
__global__ __launch_bounds__(64 * kWaves, (occupancy<D, kMT>())) void attend_kernel(AttendArgs a) {
    __shared__ Lds<D, kMT, kWaves> sh;
    attend_body<D, kMT, kWaves, kMode>(a, sh, blockIdx.x, gridDim.x);
}

// Joins the units that the first kernel left in parts. A workgroup here belongs
// to one there and to 16 rows of a row block. The 16 rows of a unit of fewer
// than 16 parts are dealt to the workgroups of its first four parts, a
// wavefront a row; those of a unit of more to the workgroups of its first 16
// parts, which take one row with all their wavefronts. Lanes
// hold 4 channels, 256 / D parts lie side by side in a wavefront, kDeep of them
// each are in flight. The order of the sums is fixed by the shapes and lengths
// of the call.
template <int D, int kMT>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
    constexpr int kSide = 256 / D, kLanes = 64 / kSide;     // parts side by side, lanes of each
    constexpr int kDeep = 8;
    __shared__ Joined sh[kFew][64];
    const int lane = threadIdx.x & 63, wave = scalar((int)threadIdx.x >> 6);
    const int side = lane / kLanes, ch = lane % kLanes * 4;
    const int g = blockIdx.x / kMT, in0 = blockIdx.x % kMT * 16;
    const int4 both[2] = {a.parts[2 * g], a.parts[2 * g + 1]};
    #pragma unroll
    for (int slot = 0; slot < 2; ++slot) {
        const int n = both[slot].y, s0 = both[slot].z, first = both[slot].w;
        const bool many = n >= 16;
        if (n == 0 || s0 >= (many ? 16 : 4)) continue;
        const int rb = both[slot].x % a.row_blocks, h = both[slot].x / a.row_blocks % a.pages.heads;
        const int b = both[slot].x / a.row_blocks / a.pages.heads;
        const int rows = plain_block<kWindow>(a, b).len * a.group - rb * (16 * kMT);
        const int by = many ? kFew * kSide : kSide;
        for (int i = many ? s0 : s0 * kFew + wave; i < 16 && in0 + i < rows; i += many ? 16 : min(n, 4) * kFew) {
            const int in = in0 + i;
            Joined j{kNegInf, 0.0f, {0, 0, 0, 0}};
            for (int s = (many ? wave * kSide : 0) + side; s < n; s += kDeep * by) {
                f32x4 v[kDeep];
                float2 ml[kDeep];
                #pragma unroll
                for (int k = 0; k < kDeep; ++k) {
                    const long long p = (long long)slot_of(first, min(s + k * by, n - 1)) * (16 * kMT) + in;
                    ml[k] = a.part_ml[p];
                    v[k] = *reinterpret_cast<const f32x4*>(a.part_o + p * D + ch);
                }
                #pragma unroll
                for (int k = 0; k < kDeep; ++k) {
                    if (s + k * by < n) j.add(ml[k].x, ml[k].y, v[k]);
                }
            }
            #pragma unroll
            for (int o = kLanes; o < 64; o <<= 1) {
                f32x4 other;
                #pragma unroll
                for (int c = 0; c < 4; ++c) other[c] = __shfl_xor(j.acc[c], o);
                j.add(__shfl_xor(j.ref, o), __shfl_xor(j.sum, o), other);
            }
            if (many) {
                __syncthreads();
                sh[wave][lane] = j;
                __syncthreads();
                j = sh[0][lane];
                #pragma unroll
                for (int w = 1; w < kFew; ++w) j.add(sh[w][lane].ref, sh[w][lane].sum, sh[w][lane].acc);
            }
            if (side == 0 && (!many || wave == 0)) {
                const int row = rb * (16 * kMT) + in;
                const int t = row / a.group, head = h * a.group + (row - t * a.group);
                const float inv = 1.0f / j.sum;
                const unsigned w[2] = {pack_bf16(j.acc[0] * inv, j.acc[1] * inv),
                                       pack_bf16(j.acc[2] * inv, j.acc[3] * inv)};
                uint16_t* dst = a.out + (((long long)b * (a.K + 1) + t) * a.Hq + head) * D + ch;
                __builtin_memcpy(__builtin_assume_aligned(dst, 8), w, 8);
            }
        }
    }
}

// What the host fixes of a call: rows per wavefront, row blocks, workgroups.
struct Plan {
    int mt, row_blocks;
    int groups;         // workgroups resident at once (and no more than there is work for)
    int grid, slots;
    bool direct;
    int waves;          // of a workgroup
};

template <int D>
int resident(int mt) {      // workgroups of a kernel that the 256 CUs hold at once
    return 256 * (mt == 1 ? occupancy<D, 1>() : mt == 2 ? occupancy<D, 2>()
                  : mt == 3 ? occupancy<D, 3>() : occupancy<D, 4>());
}

Plan plan_of(int B, int K, int Hq, int kv_heads, int D, int page_size, int max_pages, int window,
             int sinks = 0, int resident_groups = 0) {
    Plan p;
    const int rows = (K + 1) * (Hq / kv_heads);
    const int widest = D == 256 ? 2 : 4;     // accumulators: kMT D / 4 registers a lane
    p.mt = std::min((rows + 15) / 16, widest);
    p.row_blocks = (rows + 16 * p.mt - 1) / (16 * p.mt);
    const long long units = (long long)B * kv_heads * p.row_blocks;
    long long tokens = (long long)max_pages * page_size;
    if (window > 0) tokens = std::min(tokens, (long long)window + K + kTile + (sinks > 0 ? (long long)sinks + kTile : 0));
    const long long tiles = (tokens + kTile - 1) / kTile + 1;
    const long long most = (units * tiles * (kTileCost + p.mt) + kLeastShare - 1) / kLeastShare;
    const int held = resident_groups > 0 ? resident_groups
                     : D == 64 ? resident<64>(p.mt) : D == 128 ? resident<128>(p.mt) : resident<256>(p.mt);
    p.groups = (int)std::min<long long>(held, most);
    p.direct = tiles <= kDirectTiles || (units >= held && tiles <= 2 * kDirectTiles) ||
               (units >= (long long)kDirectUnits * held && tiles * held <= kDirectTiles * units);
    // Twice the wavefronts on a unit's tiles where a CU has no more than one unit
    // of one row tile: what is left is latency. (8 requests of up to 577 tokens, 8
    // kv heads of 128: 7.0 against 7.6 us, of 900 tokens 8.2 against 9.4, of 256
    // channels 11.3 against 14.4; 32 requests 9.4 against 10.8, but 64, two units
    // a CU, 15.9 against 15.2.)
    p.waves = p.direct && p.mt == 1 && units <= 256 ? kMany : kFew;
    p.grid = (int)(p.direct ? units : p.groups + std::min<long long>(units, held));
    p.slots = p.direct ? 0 : std::max(2 * p.groups, p.grid);
    return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t parts_of(const Plan& p) { return (size_t)p.slots * 16 * p.mt; }

bool shape_ok(int B, int K, int Hq, int kv_heads, int D, int page_size, int max_pages, int window) {
    return B >= 0 && B <= SV_MAX_BATCH && K >= 0 && K <= SV_MAX_K && window >= 0 &&
           geometry_ok(kv_heads, D, page_size, max_pages, 1) && Hq >= kv_heads &&
           Hq <= SV_MAX_HEADS && Hq % kv_heads == 0;
}

template <int D, int kMT, Mode kMode>
void launch(const AttendArgs& a, const Plan& p, hipStream_t s) {
    if constexpr (kMT == 1) {
        if (p.waves == kMany) {
            hipLaunchKernelGGL((attend_kernel<D, kMT, kMany, kMode>), dim3((unsigned)p.grid), dim3(64 * kMany), 0, s, a);
            return;
        }
    }
    hipLaunchKernelGGL((attend_kernel<D, kMT, kFew, kMode>), dim3((unsigned)p.grid), dim3(64 * kFew), 0, s, a);
    if (!p.direct) {
        const unsigned blocks = (unsigned)(p.grid * kMT);
        hipLaunchKernelGGL((attend_join_kernel<D, kMT>), dim3(blocks), dim3(256), 0, s, a);
    }
}

size_t workspace_of(const Plan& p, int head_dim) {
    if (p.direct) return 256;
    return round256((size_t)p.grid * 2 * sizeof(int4)) + round256(parts_of(p) * sizeof(float2)) +
           parts_of(p) * head_dim * sizeof(float);
}

// Whether a call's arguments are in order (an sv_status).
int check(const void* queries, int64_t query_stride, const void* cache, const int32_t* page_table,
          const int32_t* ctx_lens, const int32_t* budgets, int B, int K, int q_heads, int kv_heads,
          int head_dim, int page_size, int max_pages, int num_pages, float scale, int window,
          const void* out, const int32_t* out_status, const void* workspace) {
    if (!shape_ok(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, window) ||
        num_pages < 1 || !std::isfinite(scale)) {
        return SV_ERR_ARG;
    }
    if (B == 0) return SV_OK;
    if (query_stride < (int64_t)q_heads * head_dim || query_stride > SV_MAX_STRIDE) {
        return SV_ERR_ARG;
    }
    if (!queries || !cache || !page_table || !ctx_lens || !out || !workspace) return SV_ERR_NULL;
    if (!aligned(queries, 16) || query_stride % 8 != 0 || !aligned(cache, 16) ||
        !aligned(out, 16) || !aligned(workspace, 256) || !aligned(page_table, 4) ||
        !aligned(ctx_lens, 4) || !aligned(budgets, 4) || !aligned(out_status, 4)) {
        return SV_ERR_ALIGN;
    }
    return SV_OK;
}

// The kernels' arguments for a call that is in order.
AttendArgs args_of(const Plan& p, const void* queries, int64_t query_stride, const void* cache,
                   const int32_t* page_table, const int32_t* ctx_lens, const int32_t* budgets, int B,
                   int K, int q_heads, int kv_heads, int page_size, int max_pages, int num_pages,
                   float scale, void* out, int32_t* out_status, void* workspace) {
    AttendArgs a{};
    a.q = static_cast<const uint16_t*>(queries);
    a.q_stride = query_stride;
    a.cache = static_cast<const uint8_t*>(cache);
    a.ctx_lens = ctx_lens;
    a.budgets = budgets;
    a.out = static_cast<uint16_t*>(out);
    a.status = out_status;
    char* ws = static_cast<char*>(workspace);
    a.parts = reinterpret_cast<int4*>(ws);
    a.part_ml = reinterpret_cast<float2*>(ws + round256((size_t)p.grid * 2 * sizeof(int4)));
    a.part_o = reinterpret_cast<float*>(ws + round256((size_t)p.grid * 2 * sizeof(int4)) +
                                        round256(parts_of(p) * sizeof(float2)));
    a.pages = make_pages(page_table, kv_heads, page_size, max_pages, num_pages);
    a.B = B;
    a.K = K;
    a.Hq = q_heads;
    a.group = q_heads / kv_heads;
    a.groups = p.groups;
    a.row_blocks = p.row_blocks;
    a.direct = p.direct;
    a.negate = scale < 0.0f;
    // A scale of 0 becomes 2^-126, under which every seen score is as good as 0
    // and an unseen one (-inf) still is -inf; one too large for fp32 its largest
    // value, under which a score of 0 still is 0.
    a.c = (float)std::clamp(std::fabs((double)scale) * 1.4426950408889634, (double)FLT_MIN, (double)FLT_MAX);
    return a;
}

template <Mode kMode>
int launch_attend(const AttendArgs& a, const Plan& p, int head_dim, hipStream_t s) {
    switch (head_dim * 8 + p.mt) {
        case 64 * 8 + 1: launch<64, 1, kMode>(a, p, s); break;
        case 64 * 8 + 2: launch<64, 2, kMode>(a, p, s); break;
        case 64 * 8 + 3: launch<64, 3, kMode>(a, p, s); break;
        case 64 * 8 + 4: launch<64, 4, kMode>(a, p, s); break;
        case 128 * 8 + 1: launch<128, 1, kMode>(a, p, s); break;
        case 128 * 8 + 2: launch<128, 2, kMode>(a, p, s); break;
        case 128 * 8 + 3: launch<128, 3, kMode>(a, p, s); break;
        case 128 * 8 + 4: launch<128, 4, kMode>(a, p, s); break;
        case 256 * 8 + 1: launch<256, 1, kMode>(a, p, s); break;
        default: launch<256, 2, kMode>(a, p, s); break;
    }
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

// A call without a shared prefix.
template <Mode kMode>
int attend(const void* queries, int64_t query_stride, const void* cache, const int32_t* page_table,
           const int32_t* ctx_lens, const int32_t* budgets, int B, int K, int q_heads,
           int kv_heads, int head_dim, int page_size, int max_pages, int num_pages, float scale,
           int window, int sinks, void* out, int32_t* out_status, void* workspace,
           size_t workspace_bytes, void* stream) {
    const int rc = check(queries, query_stride, cache, page_table, ctx_lens, budgets, B, K, q_heads,
                         kv_heads, head_dim, page_size, max_pages, num_pages, scale, window, out,
                         out_status, workspace);
    if (rc != SV_OK || B == 0) return rc;
    const Plan p = plan_of(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, window, sinks);
    if (workspace_bytes < workspace_of(p, head_dim)) return SV_ERR_ARG;
    AttendArgs a = args_of(p, queries, query_stride, cache, page_table, ctx_lens, budgets, B, K, q_heads,
                           kv_heads, page_size, max_pages, num_pages, scale, out, out_status, workspace);
    a.window = window;
    a.sinks = sinks;
    return launch_attend<kMode>(a, p, head_dim, static_cast<hipStream_t>(stream));
}

}  // namespace
