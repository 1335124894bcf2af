// block_attention.hip -- attention of drafted blocks over the paged 4-bit
// cache, for MI355X (gfx950).
//
// The mathematics: row (t, h) of request b, t <= k_b, stands at position
// p = ctx_b + t and sees the positions j of [max(0, p - window + 1), p]:
//   o = sum_j 2^(z_j - m) v_j / sum_j 2^(z_j - m),  z_j = scale log2(e) q . k_j,
// with the running maximum m and the sums held in fp32 over one pass. Keys
// and values are decoded to bf16 (exact); products accumulate in fp32 on the
// matrix cores. The probabilities 2^(z - m), in [0, 1], are rounded to bf16
// for the value product (2^-9 relative each, the size of the output's own
// rounding); their sum is taken before that rounding.
//
// Layout: a wavefront takes tiles of 32 tokens of one kv head and all query
// rows that share it (up to 16 kMT rows of (t, head in the group), in
// registers). Scores are computed transposed, K Q^T, so that a lane holds one
// query row (lane % 16) and tokens {16 half + 4 (lane / 16) + r}: the row's
// statistics stay within 4 lanes, the probabilities are already the right
// operand of V^T P^T (whose contraction runs over tokens in that same order),
// and the accumulators' rescale is a per-lane factor. The cache's tile layout
// gives every lane its codes in 16-byte loads in these orders.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "cache_tile.h"

namespace {

using namespace svcache;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) unsigned u32x4;

constexpr int kWaves = 4;
constexpr float kNegInf = -INFINITY;

// How the work is cut. A unit is a request's kv head and block of 16 kMT
// rows. All units' tiles lie on one line, a tile as long as its cost (kTileCost
// plus its row tiles) and each unit led by a stretch for what starting and
// ending one takes; every workgroup takes an equal share of the line, so that
// ragged lengths and budgets load the chip evenly. The lengths are on the
// device, so every workgroup lays the line out for itself (sums over the
// requests and a prefix sum to find its place). A workgroup that ends inside a
// unit leaves a partial result, which the join kernel puts together.
// With page table rows of at most kDirectTiles tiles a workgroup per unit is
// launched instead and nothing is joined: a second launch and the search
// would cost more than the imbalance.
constexpr int kTileCost = 2;
constexpr int kUnitCost = 64;       // at most; a quarter of a share where shares are short
constexpr int kLeastShare = 32;     // a few tiles for each of a workgroup's wavefronts
constexpr int kDirectTiles = 32;

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
    int4* parts;        // [slot]: unit, its parts, which one this is, workgroup of the first
    Pages pages;
    int B, K, Hq, group;
    int row_blocks;     // blocks of 16 kMT rows of a full block's (K + 1) group rows
    int window;
    bool direct;        // a workgroup per unit
    bool negate;        // scale < 0: queries are negated and |scale| is used
    float c;            // |scale| * log2(e)
};

// The tiles a request's block reads: [first, end).
struct Span {
    int first, end;
    __device__ __forceinline__ int size() const { return end - first; }
};
__device__ __forceinline__ Span span_of(const Block& blk, int window) {
    const int lo = window > 0 ? max(0, blk.ctx - window + 1) : 0;
    return Span{lo / kTile, (blk.ctx + blk.len + kTile - 1) / kTile};
}

// A run of one unit's tiles: [t0, t1) of (b, h, row block rb); slot: where its
// partial result goes (slot 2 g + 1 of the workgroup g that starts the unit,
// 2 g of those that go on with it), or -1 when the run is the whole unit.
struct Work {
    int b, h, rb, t0, t1, slot;
};

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
__device__ __forceinline__ Block scalar(const Block& k) { return Block{scalar(k.ctx), scalar(k.len)}; }

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
    static constexpr int kWords = L::U / 4;             // words of a key unit
    unsigned k[2][L::kPlanes][kWords];                  // half, plane: a token's unit of channels
    unsigned v[2][L::kPlanes][L::C];                    // half, plane: 4 tokens' pieces
    unsigned ks[L::kPlanes];                            // key scales of both halves
    unsigned vs[L::kPlanes][2];                         // value scales of 4 + 4 tokens

    // The tile is the same for the whole wavefront: one scalar base, a 32-bit
    // offset per lane.
    __device__ __forceinline__ void load(const uint8_t* tile, unsigned lane) {
        const unsigned x = lane & 15, quad = lane >> 4;
        #pragma unroll
        for (int p = 0; p < L::kPlanes; ++p) {
            #pragma unroll
            for (int half = 0; half < 2; ++half) {
                __builtin_memcpy(k[half][p], __builtin_assume_aligned(
                    tile + (half * 8 * D + p * 64 * L::U) + lane * L::U, L::U), L::U);
                __builtin_memcpy(v[half][p], __builtin_assume_aligned(
                    tile + (L::kVCodes + (p * 2 + half) * 256 * L::C) + lane * (4 * L::C), 4 * L::C), 4 * L::C);
            }
            const unsigned kg = D == 64 ? quad >> 1 : quad, vg = D == 64 ? x >> 3 : x >> 2;
            ks[p] = *reinterpret_cast<const uint16_t*>(tile + (L::kKScales + p * 128) + (kg * 32 + x * 2));
            __builtin_memcpy(vs[p], __builtin_assume_aligned(
                tile + (L::kVScales + p * 128) + (vg * 4 + quad) * 8, 8), 8);
        }
    }
};

// Registers of one wavefront over its tiles.
template <int D, int kMT>
struct State {
    using L = Tile<D>;
    static constexpr int kPlanes = L::kPlanes;
    static constexpr int kUnitSteps = D == 64 ? 2 : 4;  // products of 32 channels in a key unit
    static constexpr int kSteps = D / 32;
    static constexpr int kChans = D == 64 ? 4 : 8;      // channels of a value piece
    f32x4 o[kMT][kPlanes][kChans];
    float ref[kMT];     // reference of the exponents; -inf: nothing seen
    float sum[kMT];     // this lane's share of the row's sum
    int pos[kMT];       // the row's position; -1 past the block
};

template <int D, int kMT>
struct Lds {
    static constexpr int kPieces = kMT * Tile<D>::kPlanes * (D == 64 ? 4 : 8) / 4;  // float4 per lane and component
    union {
        u32x4 q[kMT][D / 32][64];           // right operands of K Q^T
        f32x4 o[kWaves][2][kPieces][64];    // two components of the accumulators at a time
    };
    float ref[kWaves][kMT][16];
    float sum[kWaves][kMT][16];
    unsigned long long scan[kWaves], before;
    unsigned scan_units[kWaves];
    int found;
};

// One tile. kAct: row tiles that hold rows of the block. kMasked: some row
// does not see some token of the tile.
template <int D, int kMT, int kAct, bool kMasked>
__device__ __forceinline__ void tile_step(State<D, kMT>& st, const Frag<D>& f,
                                          const Lds<D, kMT>& sh, const AttendArgs& a, int lane,
                                          int tok0, int last, const uint8_t* tile) {
    using L = Tile<D>;
    using S = State<D, kMT>;
    const int quad = lane >> 4;
    // Scores of 2 x 16 tokens (lane: tokens 16 half + 4 quad + r).
    f32x4 z[kAct][2] = {};
    #pragma unroll
    for (int p = 0; p < S::kPlanes; ++p) {
        const float s[2] = {scale_of(f.ks[p] & 255u), scale_of(f.ks[p] >> 8)};
        #pragma unroll
        for (int j = 0; j < S::kUnitSteps; ++j) {
            __builtin_amdgcn_sched_barrier(0);
            bf16x8 kf[2];
            #pragma unroll
            for (int half = 0; half < 2; ++half) {
                const unsigned w = f.k[half][p][j];
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
    __builtin_amdgcn_sched_barrier(0);
    bf16x8 pf[kAct];
    #pragma unroll
    for (int mt = 0; mt < kAct; ++mt) {
        if (kMasked) {
            const int lo = a.window > 0 ? st.pos[mt] - a.window : -1;
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = tok0 + 16 * (i >> 2) + 4 * quad + (i & 3);
                if (j > st.pos[mt] || j <= lo) z[mt][i >> 2][i & 3] = kNegInf;
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
                w[i] = r & 1 ? f.v[half][p][r >> 1] >> 16 : f.v[half][p][r >> 1];
            } else {
                w[i] = f.v[half][p][r];
            }
            const unsigned sc = f.vs[p][half];
            unsigned bits = (r == 3 ? sc >> 1 : sc << (23 - 8 * r)) & 0x7f800000u;
            if (kMasked) {
                // What some row does not see must not reach it as 0 * NaN:
                // tokens past the block hold anything and are cleared; NaN
                // groups of tokens that other rows see are cleared here and
                // put into those rows below.
                const int j = tok0 + 16 * half + 4 * quad + r;
                const bool nan = bits == 0x7f800000u;
                poison |= nan && j <= last;
                if (nan || j > last) {
                    bits = 0x3f800000u;
                    w[i] = 0;
                }
            }
            vs[i] = __uint_as_float(bits);
        }
        #pragma unroll
        for (int cb = 0; cb < S::kChans / 2; ++cb) {
            __builtin_amdgcn_sched_barrier(0);
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
                if (j > last || tile[L::v_scale(tok, og)] != 255u) continue;
                #pragma unroll
                for (int mt = 0; mt < kAct; ++mt) {
                    if (j > st.pos[mt] || (a.window > 0 && j <= st.pos[mt] - a.window)) continue;
                    #pragma unroll
                    for (int c = 0; c < S::kChans; ++c) st.o[mt][p][c] *= NAN;
                }
            }
        }
    }
}

// This wavefront's share of the tiles [t0, t1). The tiles that every row sees
// whole come in a loop that keeps the next tile's bytes in flight; the few at the ends that some row does not see whole (the block's
// own, and the windows' edges) are worked on one by one while the loop's first
// bytes are on their way.
template <int D>
struct Stream {
    using L = Tile<D>;
    Frag<D> f[2];
    long long at[2];
    int t, u0, u1;
    // Page numbers of this wavefront's next 64 tiles, one a lane. They come in
    // one load: a lookup per tile would wait for every load before it, the
    // tiles in flight among them.
    int pages;

    // A tile whose page is bad is flagged and skipped; the first tile of the
    // cache stands in for its bytes, and past the end for the bytes of no tile.
    __device__ __forceinline__ long long locate(const AttendArgs& a, const Work& wk, int page,
                                                int tile, int lane) const {
        const long long p = a.pages.tile_in(page, wk.h, tile * kTile, L::kBytes);
        if (p < 0 && lane == 0) flag(a.status, SV_FLAG_BAD_PAGE);
        return p;
    }
    // The wavefront's tile number n = (tile - u0 - wave) / kWaves into f[i].
    template <int i>
    __device__ __forceinline__ void fetch(const AttendArgs& a, const Work& wk, int tile, int n,
                                          int lane) {
        at[i] = -1;
        if (tile < u1) {
            if ((n & 63) == 0) {
                const int mine = tile + lane * kWaves;
                pages = mine < u1 ? a.pages.page(wk.b, mine * kTile) : -1;
            }
            at[i] = locate(a, wk, __builtin_amdgcn_readlane(pages, n & 63), tile, lane);
        }
        f[i].load(a.cache + max(at[i], 0ll), lane);
    }
    __device__ __forceinline__ void start(const AttendArgs& a, const Work& wk, const Block& blk,
                                          int lane, int wave) {
        // Tiles [u0, u1) of this run lie wholly in [all_lo, ctx + 1), the
        // tokens that every row of the block sees.
        const int all_lo = a.window > 0 ? max(0, blk.ctx + blk.len - a.window) : 0;
        u0 = min(max(wk.t0, (all_lo + kTile - 1) / kTile), wk.t1);
        u1 = max(u0, min(wk.t1, (blk.ctx + 1) / kTile));
        t = u0 + wave;
        if (t < u1) fetch<0>(a, wk, t, 0, lane);
    }
    template <int kMT, int kAct>
    __device__ __forceinline__ void run(State<D, kMT>& st, const Lds<D, kMT>& sh,
                                        const AttendArgs& a, const Work& wk, const Block& blk,
                                        int lane, int wave) {
        const int last = blk.ctx + blk.len - 1;
        const int edges = (u0 - wk.t0) + (wk.t1 - u1);
        for (int i = kWaves - 1 - wave; i < edges; i += kWaves) {
            const int e = wk.t0 + i < u0 ? wk.t0 + i : u1 + (i - (u0 - wk.t0));
            const long long edge = locate(a, wk, scalar(a.pages.page(wk.b, e * kTile)), e, lane);
            if (edge < 0) continue;
            Frag<D> g;
            g.load(a.cache + edge, lane);
            tile_step<D, kMT, kAct, true>(st, g, sh, a, lane, e * kTile, last, a.cache + edge);
        }
        for (int n = 1; t < u1; n += 2) {
            step<kMT, kAct, 0>(st, sh, a, wk, n, lane);
            step<kMT, kAct, 1>(st, sh, a, wk, n + 1, lane);
        }
    }
    template <int kMT, int kAct, int i>
    __device__ __forceinline__ void step(State<D, kMT>& st, const Lds<D, kMT>& sh,
                                         const AttendArgs& a, const Work& wk, int n, int lane) {
        fetch<1 - i>(a, wk, t + kWaves, n, lane);
        if (at[i] >= 0) tile_step<D, kMT, kAct, false>(st, f[i], sh, a, lane, 0, 0, nullptr);
        t += kWaves;
    }
};

// A request's share of the line.
template <int kMT>
struct Share {
    Block blk;
    Span span;
    int rows, blocks;           // rows, row blocks that hold some
    __device__ __forceinline__ Share(const AttendArgs& a, const Block& k)
        : blk(k), span(span_of(k, a.window)), rows(k.len * a.group),
          blocks((rows + 16 * kMT - 1) / (16 * kMT)) {}
    // Row tiles of row block rb, and what one tile of its units costs.
    __device__ __forceinline__ int act(int rb) const { return min((rows - rb * 16 * kMT + 15) / 16, kMT); }
    __device__ __forceinline__ int cost(int rb) const { return kTileCost + act(rb); }
    // All tiles of a unit of row block rb, and of all the request's units.
    __device__ __forceinline__ int tiles(int rb) const { return span.size() * cost(rb); }
    __device__ __forceinline__ unsigned long long tiles_of_all(int heads) const {
        if (blk.len == 0) return 0;
        return (unsigned long long)heads * ((unsigned long long)(blocks - 1) * tiles(0) + tiles(blocks - 1));
    }
};

// Waves per SIMD that the registers leave room for.
template <int D, int kMT>
constexpr int occupancy() {
    return D == 256 || kMT == 4 ? 2 : D * kMT <= 128 ? 3 : 2;
}

// One run of tiles, from the queries to the output or a partial result.
template <int D, int kMT>
__device__ __forceinline__ void attend_run(const AttendArgs& a, const Work& wk, const Block& blk,
                                           Lds<D, kMT>& sh, int lane, int wave) {
    using S = State<D, kMT>;
    constexpr int kPlanes = S::kPlanes, kChans = S::kChans, kPieces = Lds<D, kMT>::kPieces;
    constexpr int kOwn = (kMT * S::kSteps + kWaves - 1) / kWaves;
    // Opaque: what derives from the lane is computed again for every run
    // rather than kept in registers across the loop over runs.
    asm volatile("" : "+v"(lane));
    const int x = lane & 15, quad = lane >> 4;
    const int rows = blk.len * a.group;
    const int act = min((rows - wk.rb * 16 * kMT + 15) / 16, kMT);

    // The queries as right operands: lane holds row x, 8 channels of its unit.
    u32x4 own[kOwn];
    #pragma unroll
    for (int k = 0; k < kOwn; ++k) {
        const int i = k * kWaves + wave, mt = i / S::kSteps, s = i % S::kSteps;
        const int r = (wk.rb * kMT + mt) * 16 + x, t = r / a.group;
        own[k] = u32x4{0, 0, 0, 0};
        if (r < rows && mt < kMT) {
            const int ch = (s / S::kUnitSteps * 4 + quad) * (8 * S::kUnitSteps) + 8 * (s % S::kUnitSteps);
            own[k] = *reinterpret_cast<const u32x4*>(
                a.q + ((long long)wk.b * (a.K + 1) + t) * a.q_stride +
                (wk.h * a.group + (r - t * a.group)) * D + ch);
            if (a.negate) own[k] ^= u32x4{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
        }
    }
    Stream<D> stream;
    stream.start(a, wk, blk, lane, wave);
    S st;
    #pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
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
        if (i < kMT * S::kSteps) sh.q[i / S::kSteps][i % S::kSteps][lane] = own[k];
    }
    __syncthreads();

    if (kMT >= 4 && act == 4) stream.template run<kMT, (kMT < 4 ? 1 : 4)>(st, sh, a, wk, blk, lane, wave);
    else if (kMT >= 3 && act == 3) stream.template run<kMT, (kMT < 3 ? 1 : 3)>(st, sh, a, wk, blk, lane, wave);
    else if (kMT >= 2 && act == 2) stream.template run<kMT, (kMT < 2 ? 1 : 2)>(st, sh, a, wk, blk, lane, wave);
    else stream.template run<kMT, 1>(st, sh, a, wk, blk, lane, wave);

    // Join the waves, two components of every accumulator in each of two
    // rounds; a wave adds up and writes every other piece of 4 channels of one.
    #pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
        const float sum = quad_sum(st.sum[mt]);
        if (quad == 0) {
            sh.ref[wave][mt][x] = st.ref[mt];
            sh.sum[wave][mt][x] = sum;
        }
    }
    __syncthreads();
    float total[kMT], top[kMT];
    #pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
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
            const int mt = i / (kPieces / kMT), p = i / (kChans / 4) % kPlanes, c = i % (kChans / 4) * 4;
            if (mt >= act) continue;
            #pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = 2 * round + k;
                sh.o[wave][k][i][lane] = f32x4{st.o[mt][p][c][r], st.o[mt][p][c + 1][r],
                                               st.o[mt][p][c + 2][r], st.o[mt][p][c + 3][r]};
            }
        }
        __syncthreads();
        const int k = wave & 1, m = 4 * quad + 2 * round + k;     // the lane's pieces of channels
        #pragma unroll
        for (int j = 0; j < (kPieces + 1) / 2; ++j) {
            const int i = 2 * j + (wave >> 1);
            if (i >= kPieces) continue;
            const int mt = i / (kPieces / kMT), p = i / (kChans / 4) % kPlanes, c = i % (kChans / 4) * 4;
            const int in = mt * 16 + x, row = wk.rb * (16 * kMT) + in;
            if (row >= rows) continue;
            const f32x4 v = (sh.o[0][k][i][lane] + sh.o[1][k][i][lane]) +
                            (sh.o[2][k][i][lane] + sh.o[3][k][i][lane]);
            const int ch = p * 128 + m * kChans + c;
            // mt is the same for the whole wave but no constant.
            float sum = total[0], ref = top[0];
            #pragma unroll
            for (int n = 1; n < kMT; ++n) {
                sum = mt == n ? total[n] : sum;
                ref = mt == n ? top[n] : ref;
            }
            if (wk.slot < 0) {
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
        __syncthreads();
    }
}

__device__ __forceinline__ Block plain_block(const AttendArgs& a, int b) {
    return block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, nullptr, false);
}
template <int D, int kMT>
__global__ __launch_bounds__(256, (occupancy<D, kMT>())) void attend_kernel(AttendArgs a) {
    __shared__ Lds<D, kMT> sh;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = scalar(tid >> 6);
    const int heads = a.pages.heads, g = blockIdx.x;

    if (g == 0) {                     // report bad budgets and lengths, once per call
        for (int b = tid; b < a.B; b += 256) {
            block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, a.status, true);
        }
    }
    // Where this workgroup is: unit (b, h, rb), request b's first place on the
    // line, and its stretch [lo, hi).
    int b = -1, h = 0, rb = 0, lead = 0;
    unsigned long long at = 0, lo = 0, hi = 0, share = 1;
    Block blk{0, 0};
    if (a.direct) {
        rb = g % a.row_blocks;
        h = g / a.row_blocks % heads;
        const int mine = g / a.row_blocks / heads;
        blk = scalar(plain_block(a, mine));
        if (rb < Share<kMT>(a, blk).blocks) b = mine;
    } else {
        const int per = (a.B + 255) / 256;
        const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
        if (tid == 0) sh.found = -1;
        if (tid < 2) a.parts[2 * g + tid] = make_int4(0, 0, 0, 0);
        unsigned long long mine = 0;
        unsigned units = 0;
        for (int i = b0; i < b1; ++i) {
            const Share<kMT> s(a, plain_block(a, i));
            mine += s.tiles_of_all(heads);
            units += s.blocks * heads;
        }
        unsigned long long upto = mine;
        unsigned units_upto = units;
        #pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const unsigned long long u = __shfl_up(upto, o, 64);
            const unsigned v = __shfl_up(units_upto, o, 64);
            if (lane >= o) {
                upto += u;
                units_upto += v;
            }
        }
        if (lane == 63) {
            sh.scan[wave] = upto;
            sh.scan_units[wave] = units_upto;
        }
        __syncthreads();
        unsigned long long all = 0;
        unsigned all_units = 0;
        #pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) {
                upto += sh.scan[w];
                units_upto += sh.scan_units[w];
            }
            all += sh.scan[w];
            all_units += sh.scan_units[w];
        }
        lead = scalar((int)min(all / (4 * gridDim.x), (unsigned long long)kUnitCost));
        all += (unsigned long long)all_units * lead;
        share = scalar(max((all + gridDim.x - 1) / gridDim.x, (unsigned long long)kLeastShare));
        lo = g * share;
        hi = lo + share;
        upto += (unsigned long long)units_upto * lead;
        mine += (unsigned long long)units * lead;
        if (mine > 0 && upto - mine <= lo && lo < upto) {
            at = upto - mine;
            int i = b0;
            for (; i < b1 - 1; ++i) {
                const Share<kMT> s(a, plain_block(a, i));
                const unsigned long long n = s.tiles_of_all(heads) + (unsigned long long)(s.blocks * heads) * lead;
                if (lo < at + n) break;
                at += n;
            }
            sh.found = i;
            sh.before = at;
        }
        __syncthreads();
        b = scalar(sh.found);
        if (b >= 0) {
            at = scalar(sh.before);
            blk = scalar(plain_block(a, b));
        }
    }

    while (b >= 0) {
        const Share<kMT> s(a, blk);
        Work wk{b, h, rb, s.span.first, s.span.end, -1};
        const int unit = lead + s.tiles(rb);
        if (!a.direct) {
            const int cost = s.cost(rb), n = s.span.size();
            const unsigned long long start = at + (unsigned long long)h * unit + lead;
            const int i0 = lo > start ? (int)min((lo - start + cost - 1) / cost, (unsigned long long)n) : 0;
            const int i1 = hi > start ? (int)min((hi - start + cost - 1) / cost, (unsigned long long)n) : 0;
            wk.t0 = s.span.first + i0;
            wk.t1 = s.span.first + i1;
            if (i0 < i1 && (i0 > 0 || i1 < n)) {
                wk.slot = 2 * g + (i0 == 0);
                const int from = (int)(start / share);
                const int to = (int)((start + (unsigned long long)(n - 1) * cost) / share);
                if (tid == 0) {
                    a.parts[wk.slot] = make_int4((b * heads + h) * a.row_blocks + rb, to - from + 1, g - from, from);
                }
            }
        }
        if (wk.t0 < wk.t1) attend_run<D, kMT>(a, wk, blk, sh, lane, wave);
        if (a.direct) break;
        // On to the next unit: heads, row blocks, requests.
        if (++h == heads) {
            at += (unsigned long long)heads * unit;
            h = 0;
            if (++rb == s.blocks) {
                rb = 0;
                int next = b + 1;
                b = -1;
                for (; next < a.B && b < 0; next += 64) {     // the next request that holds anything
                    Block k{0, 0};
                    if (next + lane < a.B) k = plain_block(a, next + lane);
                    const unsigned long long some = __ballot(k.len > 0);
                    if (some != 0) {
                        const int i = __builtin_ctzll(some);
                        b = next + i;
                        blk = Block{__builtin_amdgcn_readlane(k.ctx, i), __builtin_amdgcn_readlane(k.len, i)};
                    }
                }
            }
        }
        if (b >= 0 && at + (unsigned long long)h * (lead + Share<kMT>(a, blk).tiles(rb)) >= hi) b = -1;
    }
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

// Joins the units that workgroups of the first kernel left in parts: the part
// of workgroup `from` that starts the unit is in slot 2 from + 1, those of the
// next ones in slots 2 (from + 1), 2 (from + 2), ... A workgroup here belongs
// to one workgroup g there and four rows. A unit of fewer than four parts is
// joined by the workgroups of its first part, a wavefront a row; of more, by
// those of its first four parts, each taking one of the four rows with all its
// wavefronts. Lanes hold 4 channels, 256 / D parts lie side by side in a
// wavefront, kDeep of them each are in flight. The order of the sums is fixed
// by the shapes and lengths of the call.
template <int D, int kMT>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
    constexpr int kSide = 256 / D, kLanes = 64 / kSide;     // parts side by side, lanes of each
    constexpr int kDeep = 8;
    __shared__ Joined sh[kWaves][64];
    const int lane = threadIdx.x & 63, wave = scalar((int)threadIdx.x >> 6);
    const int side = lane / kLanes, ch = lane % kLanes * 4;
    const int g = blockIdx.x / (4 * kMT), in0 = blockIdx.x % (4 * kMT) * 4;
    const int4 both[2] = {a.parts[2 * g], a.parts[2 * g + 1]};
    #pragma unroll
    for (int slot = 0; slot < 2; ++slot) {
        const int n = both[slot].y, s0 = both[slot].z, from = both[slot].w;
        const bool many = n >= 4;
        if (n == 0 || s0 >= (many ? 4 : 1)) continue;
        const int rb = both[slot].x % a.row_blocks, h = both[slot].x / a.row_blocks % a.pages.heads;
        const int b = both[slot].x / a.row_blocks / a.pages.heads;
        const int in = in0 + (many ? s0 : wave);
        const int row = rb * (16 * kMT) + in;
        const Block blk = plain_block(a, b);
        const bool live = row < blk.len * a.group;
        const int by = many ? kWaves * kSide : kSide;

        Joined j{kNegInf, 0.0f, {0, 0, 0, 0}};
        for (int s = (many ? wave * kSide : 0) + side; live && s < n; s += kDeep * by) {
            f32x4 v[kDeep];
            float2 ml[kDeep];
            #pragma unroll
            for (int k = 0; k < kDeep; ++k) {
                const int i = min(s + k * by, n - 1);
                const long long p = (long long)(2 * (from + i) + (i == 0)) * (16 * kMT) + in;
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
            for (int w = 1; w < kWaves; ++w) j.add(sh[w][lane].ref, sh[w][lane].sum, sh[w][lane].acc);
        }
        if (live && side == 0 && (!many || wave == 0)) {
            const int t = row / a.group, head = h * a.group + (row - t * a.group);
            const float inv = 1.0f / j.sum;
            const unsigned w[2] = {pack_bf16(j.acc[0] * inv, j.acc[1] * inv),
                                   pack_bf16(j.acc[2] * inv, j.acc[3] * inv)};
            uint16_t* dst = a.out + (((long long)b * (a.K + 1) + t) * a.Hq + head) * D + ch;
            __builtin_memcpy(__builtin_assume_aligned(dst, 8), w, 8);
        }
    }
}

// What the host fixes of a call: rows per wavefront, row blocks, workgroups.
struct Plan {
    int mt, row_blocks, groups;
    bool direct;
};

template <int D>
int resident(int mt) {      // workgroups of a kernel that the 256 CUs hold at once
    return 256 * (mt == 1 ? occupancy<D, 1>() : mt == 2 ? occupancy<D, 2>()
                  : mt == 3 ? occupancy<D, 3>() : occupancy<D, 4>());
}

Plan plan_of(int B, int K, int Hq, int kv_heads, int D, int page_size, int max_pages, int window) {
    Plan p;
    const int rows = (K + 1) * (Hq / kv_heads);
    const int most = D == 256 ? 2 : 4;       // accumulators: kMT D / 4 registers a lane
    p.mt = (rows + 15) / 16 < most ? (rows + 15) / 16 : most;
    p.row_blocks = (rows + 16 * p.mt - 1) / (16 * p.mt);
    const long long units = (long long)B * kv_heads * p.row_blocks;
    long long tokens = (long long)max_pages * page_size;
    if (window > 0 && tokens > (long long)window + K + kTile) tokens = (long long)window + K + kTile;
    const long long tiles = (tokens + kTile - 1) / kTile + 1;
    p.direct = tiles <= kDirectTiles;
    // No more workgroups than the longest line has shares for.
    const long long most_shares = (units * (kUnitCost + tiles * (kTileCost + p.mt)) + kLeastShare - 1) / kLeastShare;
    const int held = D == 64 ? resident<64>(p.mt) : D == 128 ? resident<128>(p.mt) : resident<256>(p.mt);
    p.groups = (int)(p.direct ? units : std::min<long long>(held, most_shares));
    return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t parts_of(const Plan& p) { return (size_t)p.groups * 2 * 16 * p.mt; }

bool shape_ok(int B, int K, int Hq, int kv_heads, int D, int page_size, int max_pages, int window) {
    return B >= 0 && B <= SV_MAX_BATCH && K >= 0 && K <= SV_MAX_K && window >= 0 &&
           geometry_ok(kv_heads, D, page_size, max_pages, 1) && Hq >= kv_heads &&
           Hq <= SV_MAX_HEADS && Hq % kv_heads == 0;
}

template <int D, int kMT>
void launch(const AttendArgs& a, const Plan& p, hipStream_t s) {
    hipLaunchKernelGGL((attend_kernel<D, kMT>), dim3((unsigned)p.groups), dim3(256), 0, s, a);
    if (!p.direct) {
        const unsigned blocks = (unsigned)(p.groups * 4 * kMT);
        hipLaunchKernelGGL((attend_join_kernel<D, kMT>), dim3(blocks), dim3(256), 0, s, a);
    }
}

}  // namespace

extern "C" size_t spec_verify_attention_workspace_bytes(int B, int K, int q_heads, int kv_heads,
                                                        int head_dim, int page_size, int max_pages,
                                                        int window) {
    if (B < 1 || !shape_ok(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, window)) {
        return 0;
    }
    const Plan p = plan_of(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, window);
    if (p.direct) return 256;
    return round256((size_t)p.groups * 2 * sizeof(int4)) + round256(parts_of(p) * sizeof(float2)) +
           parts_of(p) * head_dim * sizeof(float);
}

extern "C" int spec_verify_attention(const void* queries, int64_t query_stride, const void* cache,
                                     const int32_t* page_table, const int32_t* ctx_lens,
                                     const int32_t* budgets, int B, int K, int q_heads,
                                     int kv_heads, int head_dim, int page_size, int max_pages,
                                     int num_pages, float scale, int window, void* out,
                                     int32_t* out_status, void* workspace, size_t workspace_bytes,
                                     void* stream) {
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
    const Plan p = plan_of(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, window);
    if (workspace_bytes < spec_verify_attention_workspace_bytes(B, K, q_heads, kv_heads, head_dim,
                                                                page_size, max_pages, window)) {
        return SV_ERR_ARG;
    }
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
    a.part_ml = reinterpret_cast<float2*>(ws + round256((size_t)p.groups * 2 * sizeof(int4)));
    a.part_o = reinterpret_cast<float*>(ws + round256((size_t)p.groups * 2 * sizeof(int4)) +
                                        round256(parts_of(p) * sizeof(float2)));
    a.pages = make_pages(page_table, kv_heads, page_size, max_pages, num_pages);
    a.B = B;
    a.K = K;
    a.Hq = q_heads;
    a.group = q_heads / kv_heads;
    a.row_blocks = p.row_blocks;
    a.window = window;
    a.direct = p.direct;
    a.negate = scale < 0.0f;
    // A scale of 0 becomes 2^-126, under which every seen score is as good as 0
    // and an unseen one (-inf) still is -inf.
    a.c = std::max((float)(std::fabs((double)scale) * 1.4426950408889634), FLT_MIN);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (head_dim * 8 + p.mt) {
        case 64 * 8 + 1: launch<64, 1>(a, p, s); break;
        case 64 * 8 + 2: launch<64, 2>(a, p, s); break;
        case 64 * 8 + 3: launch<64, 3>(a, p, s); break;
        case 64 * 8 + 4: launch<64, 4>(a, p, s); break;
        case 128 * 8 + 1: launch<128, 1>(a, p, s); break;
        case 128 * 8 + 2: launch<128, 2>(a, p, s); break;
        case 128 * 8 + 3: launch<128, 3>(a, p, s); break;
        case 128 * 8 + 4: launch<128, 4>(a, p, s); break;
        case 256 * 8 + 1: launch<256, 1>(a, p, s); break;
        default: launch<256, 2>(a, p, s); break;
    }
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
