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
// rows; its tiles are cut into splits of `chunk` tiles, a workgroup each. The
// lengths are on the device, so the cut is made there: every workgroup adds
// up the tiles of all requests, takes
//   chunk = max(total / kManySplits, min(total / kFewSplits, kChunk))
// (rounded up, at least kLeastChunk), and finds its own split by a prefix sum
// over the requests. kFewSplits workgroups are resident at once; chunks are
// cut below kChunk tiles only to fill them, and above kChunk only when more
// than kManySplits splits would come of it. With kDirectUnits units or more,
// or page table rows of fewer than kDirectTiles tiles, every unit is one
// workgroup and nothing is cut.
constexpr int kFewSplits = 512;
constexpr int kManySplits = 2048;
constexpr int kChunk = 64;
constexpr int kLeastChunk = 8;
constexpr int kDirectUnits = 4096;
constexpr int kDirectTiles = 32;

struct AttendArgs {
    const uint16_t* q;
    long long q_stride;
    const uint8_t* cache;
    const int32_t* ctx_lens;
    const int32_t* budgets;
    uint16_t* out;
    int32_t* status;
    float* part_o;      // [unit][16 kMT rows][split][D], not normalised
    float2* part_ml;    // [unit][16 kMT rows][split]: reference exponent, sum
    int2* cut;          // [B]: the request's first slot, and chunk
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

// What a workgroup works on: tiles [t0, t1) of (b, h, row block rb), one of
// the unit's n splits; slot: the unit's first.
struct Work {
    int b, h, rb, t0, t1;
    int n, split, slot;
    // Where the partial of the unit's row `in` lies: a row's splits follow
    // each other, so that the join reads one run.
    __device__ __forceinline__ long long part(int rows, int in) const {
        return (long long)slot * rows + in * n + split;
    }
};

__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
    bf16x2 v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(unsigned, v);
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
    static constexpr int kPieces = kMT * Tile<D>::kPlanes * (D == 64 ? 4 : 8) / 4;  // float4 per lane and round
    u32x4 q[kMT][D / 32][64];           // right operands of K Q^T
    f32x4 o[kWaves][kPieces][64];
    float ref[kWaves][kMT][16];
    float sum[kWaves][kMT][16];
    unsigned scan[kWaves];
    int found[7];
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
// whole come in a loop that keeps the bytes of the next kAhead tiles in
// flight; the few at the ends that some row does not see whole (the block's
// own, and the windows' edges) are worked on one by one while the loop's first
// bytes are on their way.
template <int D, int kAhead>
struct Stream {
    using L = Tile<D>;
    Frag<D> f[kAhead + 1];
    long long at[kAhead + 1];
    int t, u0, u1;

    // A tile whose page is bad is flagged and skipped; the first tile of the
    // cache stands in for its bytes, and past the end for the bytes of no tile.
    __device__ __forceinline__ long long locate(const AttendArgs& a, const Work& wk, int tile,
                                                int lane) const {
        const long long p = a.pages.tile<true>(wk.b, wk.h, tile * kTile, L::kBytes);
        if (p < 0 && lane == 0) flag(a.status, SV_FLAG_BAD_PAGE);
        return p;
    }
    template <int i>
    __device__ __forceinline__ void fetch(const AttendArgs& a, const Work& wk, int tile, int lane) {
        at[i] = tile < u1 ? locate(a, wk, tile, lane) : -1;
        f[i].load(a.cache + max(at[i], 0ll), lane);
    }
    __device__ __forceinline__ void start(const AttendArgs& a, const Work& wk, const Block& blk,
                                          int lane, int wave) {
        // Tiles [u0, u1) of this split lie wholly in [all_lo, ctx + 1), the
        // tokens that every row of the block sees.
        const int all_lo = a.window > 0 ? max(0, blk.ctx + blk.len - a.window) : 0;
        u0 = min(max(wk.t0, (all_lo + kTile - 1) / kTile), wk.t1);
        u1 = max(u0, min(wk.t1, (blk.ctx + 1) / kTile));
        t = u0 + wave;
        if (t < u1) {
            fetch<0>(a, wk, t, lane);
            if constexpr (kAhead == 2) fetch<1>(a, wk, t + kWaves, lane);
        }
    }
    template <int kMT, int kAct>
    __device__ __forceinline__ void run(State<D, kMT>& st, const Lds<D, kMT>& sh,
                                        const AttendArgs& a, const Work& wk, const Block& blk,
                                        int lane, int wave) {
        const int last = blk.ctx + blk.len - 1;
        const int edges = (u0 - wk.t0) + (wk.t1 - u1);
        for (int i = kWaves - 1 - wave; i < edges; i += kWaves) {
            const int e = wk.t0 + i < u0 ? wk.t0 + i : u1 + (i - (u0 - wk.t0));
            const long long edge = locate(a, wk, e, lane);
            if (edge < 0) continue;
            Frag<D> g;
            g.load(a.cache + edge, lane);
            tile_step<D, kMT, kAct, true>(st, g, sh, a, lane, e * kTile, last, a.cache + edge);
        }
        while (t < u1) {
            step<kMT, kAct, 0>(st, sh, a, wk, lane);
            step<kMT, kAct, 1>(st, sh, a, wk, lane);
            if constexpr (kAhead == 2) step<kMT, kAct, 2>(st, sh, a, wk, lane);
        }
    }
    template <int kMT, int kAct, int i>
    __device__ __forceinline__ void step(State<D, kMT>& st, const Lds<D, kMT>& sh,
                                         const AttendArgs& a, const Work& wk, int lane) {
        fetch<(i + kAhead) % (kAhead + 1)>(a, wk, t + kAhead * kWaves, lane);
        if (at[i] >= 0) tile_step<D, kMT, kAct, false>(st, f[i], sh, a, lane, 0, 0, nullptr);
        t += kWaves;
    }
};

// Finds the split of workgroup `slot`; false when there is none.
template <int D, int kMT>
__device__ bool find_work(const AttendArgs& a, Lds<D, kMT>& sh, Work& wk) {
    const int slot = blockIdx.x;
    if (a.direct) {
        wk.rb = slot % a.row_blocks;
        wk.h = slot / a.row_blocks % a.pages.heads;
        wk.b = slot / a.row_blocks / a.pages.heads;
        const Block blk = block_of(a.ctx_lens, a.budgets, wk.b, a.K + 1, a.pages, nullptr, false);
        if (wk.rb * 16 * kMT >= blk.len * a.group) return false;
        const Span s = span_of(blk, a.window);
        wk.t0 = s.first;
        wk.t1 = s.end;
        wk.n = 1;
        return true;
    }
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (a.B + 255) / 256;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    // Tiles of a request (0: nothing to do) and its units.
    auto tiles_of = [&](int b, int& units, int& first) {
        const Block blk = block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, nullptr, false);
        units = (blk.len * a.group + 16 * kMT - 1) / (16 * kMT) * a.pages.heads;
        if (blk.len == 0) return 0;
        const Span s = span_of(blk, a.window);
        first = s.first;
        return s.size();
    };
    auto block_total = [&](unsigned v, unsigned& before) {      // inclusive scan over threads
        unsigned incl = v;
        #pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const unsigned u = __shfl_up(incl, o, 64);
            if (lane >= o) incl += u;
        }
        __syncthreads();
        if (lane == 63) sh.scan[wave] = incl;
        __syncthreads();
        before = incl - v;
        unsigned total = 0;
        #pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) before += sh.scan[w];
            total += sh.scan[w];
        }
        return total;
    };
    if (tid == 0) sh.found[0] = -1;
    // The first of this thread's requests (the only one up to 256) is kept.
    int units0 = 0, first0 = 0, n0 = 0;
    unsigned mine = 0, before;
    if (b0 < b1) n0 = tiles_of(b0, units0, first0);
    mine = n0 * units0;
    for (int b = b0 + 1; b < b1; ++b) {
        int units, first = 0;
        const int n = tiles_of(b, units, first);
        mine += n * units;
    }
    const unsigned total = block_total(mine, before);
    unsigned chunk = max((total + kManySplits - 1) / kManySplits,
                         min((total + kFewSplits - 1) / kFewSplits, (unsigned)kChunk));
    chunk = max(chunk, (unsigned)kLeastChunk);
    mine = 0;
    for (int b = b0; b < b1; ++b) {
        int units = units0, first, n = n0;
        if (b > b0) n = tiles_of(b, units, first);
        mine += (n + chunk - 1) / chunk * units;
    }
    block_total(mine, before);
    for (int b = b0; b < b1; ++b) {
        int units = units0, first = first0, n = n0;
        if (b > b0) n = tiles_of(b, units, first);
        const unsigned count = (n + chunk - 1) / chunk * units;
        if ((unsigned)slot >= before && (unsigned)slot < before + count) {
            const int in = slot - before, split = in / units;
            sh.found[0] = b;
            sh.found[1] = in % units;
            sh.found[2] = first + split * chunk;
            sh.found[3] = min(first + (split + 1) * (int)chunk, first + n);
            sh.found[4] = count / units;
            sh.found[5] = split;
            sh.found[6] = before + in % units * (count / units);
            if (in == 0) a.cut[b] = make_int2(before, chunk);
        }
        before += count;
    }
    __syncthreads();
    if (sh.found[0] < 0) return false;
    wk.b = __builtin_amdgcn_readfirstlane(sh.found[0]);
    const int unit = __builtin_amdgcn_readfirstlane(sh.found[1]);
    wk.h = unit % a.pages.heads;
    wk.rb = unit / a.pages.heads;
    wk.t0 = __builtin_amdgcn_readfirstlane(sh.found[2]);
    wk.t1 = __builtin_amdgcn_readfirstlane(sh.found[3]);
    wk.n = __builtin_amdgcn_readfirstlane(sh.found[4]);
    wk.split = __builtin_amdgcn_readfirstlane(sh.found[5]);
    wk.slot = __builtin_amdgcn_readfirstlane(sh.found[6]);
    return true;
}

// Waves per SIMD that the registers leave room for, and tiles in flight.
template <int D, int kMT>
constexpr int occupancy() {
    return D == 256 || kMT == 4 ? 2 : D * kMT <= 128 ? 4 : D * kMT <= 256 ? 3 : 2;
}
template <int D, int kMT>
constexpr int ahead() {
    return D * kMT == 384 || (D == 256 && kMT == 1) ? 2 : 1;
}

template <int D, int kMT>
__global__ __launch_bounds__(256, (occupancy<D, kMT>())) void attend_kernel(AttendArgs a) {
    using S = State<D, kMT>;
    constexpr int kPlanes = S::kPlanes, kChans = S::kChans;
    __shared__ Lds<D, kMT> sh;
    const int lane = threadIdx.x & 63, x = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    if (blockIdx.x == 0) {            // report bad budgets and lengths, once per call
        for (int b = threadIdx.x; b < a.B; b += 256) {
            block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, a.status, true);
        }
    }
    Work wk;
    if (!find_work<D, kMT>(a, sh, wk)) return;
    const Block blk = block_of(a.ctx_lens, a.budgets, wk.b, a.K + 1, a.pages, nullptr, false);
    const int rows = blk.len * a.group;

    Stream<D, ahead<D, kMT>()> stream;
    stream.start(a, wk, blk, lane, wave);

    // The queries as right operands: lane holds row x, 8 channels of its unit.
    for (int i = wave; i < kMT * S::kSteps; i += kWaves) {
        const int mt = i / S::kSteps, s = i % S::kSteps;
        const int r = (wk.rb * kMT + mt) * 16 + x, t = r / a.group;
        u32x4 w = {0, 0, 0, 0};
        if (r < rows) {
            const int ch = (s / S::kUnitSteps * 4 + quad) * (8 * S::kUnitSteps) + 8 * (s % S::kUnitSteps);
            w = *reinterpret_cast<const u32x4*>(a.q + ((long long)wk.b * (a.K + 1) + t) * a.q_stride +
                                                (wk.h * a.group + (r - t * a.group)) * D + ch);
            if (a.negate) w ^= u32x4{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
        }
        sh.q[mt][s][lane] = w;
    }
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
    __syncthreads();

    const int act = min((rows - wk.rb * 16 * kMT + 15) / 16, kMT);
    if (kMT >= 4 && act == 4) stream.template run<kMT, (kMT < 4 ? 1 : 4)>(st, sh, a, wk, blk, lane, wave);
    else if (kMT >= 3 && act == 3) stream.template run<kMT, (kMT < 3 ? 1 : 3)>(st, sh, a, wk, blk, lane, wave);
    else if (kMT >= 2 && act == 2) stream.template run<kMT, (kMT < 2 ? 1 : 2)>(st, sh, a, wk, blk, lane, wave);
    else stream.template run<kMT, 1>(st, sh, a, wk, blk, lane, wave);

    // Join the waves: component r of every accumulator in round r, of which
    // wave r writes kChans consecutive channels per (row, plane).
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
    for (int r = 0; r < 4; ++r) {
        #pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
            #pragma unroll
            for (int p = 0; p < kPlanes; ++p) {
                #pragma unroll
                for (int c = 0; c < kChans; c += 4) {
                    const f32x4 v = {st.o[mt][p][c][r], st.o[mt][p][c + 1][r],
                                     st.o[mt][p][c + 2][r], st.o[mt][p][c + 3][r]};
                    sh.o[wave][((mt * kPlanes + p) * kChans + c) / 4][lane] = v;
                }
            }
        }
        __syncthreads();
        if (wave == r) {
            #pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
                const int row = (wk.rb * kMT + mt) * 16 + x;
                if (row >= rows) continue;
                const int t = row / a.group;
                const long long part = wk.part(16 * kMT, mt * 16 + x);
                if (wk.n > 1 && r == 0 && quad == 0) {
                    a.part_ml[part] = make_float2(top[mt], total[mt]);
                }
                const float inv = 1.0f / total[mt];
                uint16_t* dst = a.out + (((long long)wk.b * (a.K + 1) + t) * a.Hq + wk.h * a.group +
                                         (row - t * a.group)) * D;
                #pragma unroll
                for (int p = 0; p < kPlanes; ++p) {
                    const int ch = p * 128 + (4 * quad + r) * kChans;
                    f32x4 v[kChans / 4];
                    #pragma unroll
                    for (int c = 0; c < kChans / 4; ++c) {
                        const int i = (mt * kPlanes + p) * (kChans / 4) + c;
                        v[c] = (sh.o[0][i][lane] + sh.o[1][i][lane]) +
                               (sh.o[2][i][lane] + sh.o[3][i][lane]);
                    }
                    if (wk.n == 1) {
                        unsigned w[kChans / 2];
                        #pragma unroll
                        for (int c = 0; c < kChans; c += 2) {
                            w[c / 2] = pack_bf16(v[c / 4][c % 4] * inv, v[c / 4][c % 4 + 1] * inv);
                        }
                        __builtin_memcpy(__builtin_assume_aligned(dst + ch, 2 * kChans), w, 2 * kChans);
                    } else {
                        #pragma unroll
                        for (int c = 0; c < kChans / 4; ++c) {
                            *reinterpret_cast<f32x4*>(a.part_o + part * D + ch + 4 * c) = v[c];
                        }
                    }
                }
            }
        }
        __syncthreads();
    }
}

// Joins the splits of a unit's rows: a workgroup per unit and four rows, a
// wavefront each. Lanes hold 4 channels, 256 / D splits lie side by side in a
// wavefront, and the partials of kDeep of them each are in flight. The running
// reference keeps this to one pass; the order of the sums is fixed by the
// shapes and lengths.
template <int D, int kMT>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
    constexpr int kSide = 256 / D, kLanes = 64 / kSide;     // splits side by side, lanes of each
    constexpr int kDeep = 8;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int side = lane / kLanes, ch = lane % kLanes * 4;
    int id = blockIdx.x;
    const int in = id % (4 * kMT) * kWaves + wave;          // row of the row block
    id /= 4 * kMT;
    const int rb = id % a.row_blocks;
    id /= a.row_blocks;
    const int h = id % a.pages.heads, b = id / a.pages.heads;
    const Block blk = block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, nullptr, false);
    const int rows = blk.len * a.group, row = rb * (16 * kMT) + in;
    if (row >= rows) return;
    const int2 cut = a.cut[b];
    const int n = (span_of(blk, a.window).size() + cut.y - 1) / cut.y;
    if (n == 1) return;
    const long long part = (long long)(cut.x + (rb * a.pages.heads + h) * n) * (16 * kMT) + in * n;

    float ref = kNegInf, sum = 0.0f;
    f32x4 acc = {0, 0, 0, 0};
    for (int s0 = side; s0 < n; s0 += kDeep * kSide) {
        f32x4 v[kDeep];
        float2 ml[kDeep];
        #pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const long long p = part + min(s0 + k * kSide, n - 1);
            ml[k] = a.part_ml[p];
            v[k] = *reinterpret_cast<const f32x4*>(a.part_o + p * D + ch);
        }
        float top = ref;
        #pragma unroll
        for (int k = 0; k < kDeep; ++k) top = fmaxf(top, ml[k].x);
        const float base = top == kNegInf ? 0.0f : top;
        const float keep = exp2_fast(ref - base);
        sum *= keep;
        acc *= keep;
        ref = top;
        #pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            if (s0 + k * kSide >= n) break;
            const float f = exp2_fast(ml[k].x - base);
            sum += ml[k].y * f;
            acc += v[k] * f;
        }
    }
    #pragma unroll
    for (int o = kLanes; o < 64; o <<= 1) {
        const float other = __shfl_xor(ref, o), top = fmaxf(ref, other);
        const float base = top == kNegInf ? 0.0f : top;
        const float f = exp2_fast(ref - base), g = exp2_fast(other - base);
        sum = sum * f + __shfl_xor(sum, o) * g;
        #pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = acc[c] * f + __shfl_xor(acc[c], o) * g;
        ref = top;
    }
    if (side == 0) {
        const int t = row / a.group, head = h * a.group + (row - t * a.group);
        const float inv = 1.0f / sum;
        const unsigned w[2] = {pack_bf16(acc[0] * inv, acc[1] * inv),
                               pack_bf16(acc[2] * inv, acc[3] * inv)};
        uint16_t* dst = a.out + (((long long)b * (a.K + 1) + t) * a.Hq + head) * D + ch;
        __builtin_memcpy(__builtin_assume_aligned(dst, 8), w, 8);
    }
}

// What the host fixes of a call: rows per wavefront, row blocks, workgroups.
struct Plan {
    int mt, row_blocks;
    bool direct;
    long long slots;
};

Plan plan_of(int B, int K, int Hq, int kv_heads, int D, int page_size, int max_pages, int window) {
    Plan p;
    const int rows = (K + 1) * (Hq / kv_heads);
    const int most = D == 256 ? 2 : 4;       // accumulators: kMT D / 4 registers a lane
    p.mt = (rows + 15) / 16 < most ? (rows + 15) / 16 : most;
    p.row_blocks = (rows + 16 * p.mt - 1) / (16 * p.mt);
    const long long units = (long long)B * kv_heads * p.row_blocks;
    // Splits: every unit's last one, and no more than kManySplits full ones
    // or than the page table row can hold.
    long long tokens = (long long)max_pages * page_size;
    if (window > 0 && tokens > (long long)window + K + kTile) tokens = (long long)window + K + kTile;
    const long long tiles = (tokens + kTile - 1) / kTile + 1;
    p.direct = units >= kDirectUnits || tiles <= kDirectTiles;
    const long long per_unit = (tiles + kLeastChunk - 1) / kLeastChunk;
    p.slots = p.direct ? units : std::min(units + kManySplits, units * per_unit);
    return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t parts_of(const Plan& p) { return (size_t)p.slots * 16 * p.mt; }

bool shape_ok(int B, int K, int Hq, int kv_heads, int D, int page_size, int max_pages, int window) {
    return B >= 0 && B <= SV_MAX_BATCH && K >= 0 && K <= SV_MAX_K && window >= 0 &&
           geometry_ok(kv_heads, D, page_size, max_pages, 1) && Hq >= kv_heads &&
           Hq <= SV_MAX_HEADS && Hq % kv_heads == 0;
}

template <int D, int kMT>
void launch(const AttendArgs& a, const Plan& p, hipStream_t s) {
    hipLaunchKernelGGL((attend_kernel<D, kMT>), dim3((unsigned)p.slots), dim3(256), 0, s, a);
    if (!p.direct) {
        const unsigned blocks = (unsigned)(a.B * a.pages.heads * p.row_blocks * 4 * kMT);
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
    return round256((size_t)B * sizeof(int2)) + round256(parts_of(p) * sizeof(float2)) +
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
    a.cut = reinterpret_cast<int2*>(ws);
    a.part_ml = reinterpret_cast<float2*>(ws + round256((size_t)B * sizeof(int2)));
    a.part_o = reinterpret_cast<float*>(ws + round256((size_t)B * sizeof(int2)) +
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
