// shared_attention.hip -- attention of drafted blocks for requests that share a
// long prefix, for MI355X (gfx950).
//
// The mathematics: a softmax over positions [0, p] is joined from its parts over
// [0, s) and [s, p]. The requests of a group hold the same tokens up to s, so the
// part in front of s is a product of all their rows with one set of keys and
// values, which no row masks: it is computed once a group, from the pages of the
// group's first request. Every request's own tokens go through the kernels of
// attend_kernel.h.
//
// Three launches:
//  - plan (one workgroup): for every group the tokens that are shared and whose
//    tiles are whole (up to the shortest context), the list of its rows, and into
//    how many parts of the prefix its work is cut;
//  - work: workgroups that take kRows rows of one head and a part of a prefix, then
//    workgroups for the requests' own tokens, which fill the chip where the
//    former end. All leave partial results;
//  - join: every row's partial results, a row's channels over D / 4 lanes.
//
// Prefix part. With many rows a tile's keys and values serve many products, so
// tiles are decoded once a workgroup into LDS, as the operands of 32x32x16
// matrix instructions: keys [8 channels' chunk][token][8], values transposed,
// [8 tokens' chunk][channel][8], every read and write of a wavefront a run without
// bank conflicts. Scores are formed transposed, K Q^T: a lane holds one row and
// 16 of a tile's 32 tokens, in the order in which the value product contracts
// them, so probabilities go from one product to the next in registers. The
// values' channels lie in an order (channel 8 x + j at place j D / 8 + x) that the
// decoding lanes write without conflicts; it is undone when results are stored.
//
// What bounds it: 128 blocks of 3..9 rows x 4 heads behind 8,192 tokens (8 kv heads of
// 128) 138 us, 9.1e10 operations; traced, which slows them, the plan takes 5.6, the
// work 132.7, the join 12.2. In the prefix part a workgroup's tile took 0.43 us with
// two workgroups a CU before the priorities set below (4 us in all); its products alone
// take 0.25, the rest is decoding (0.1) and the softmax, which a wavefront takes one
// after another with its products and two wavefronts a SIMD hide from each other only
// in part. Starting and ending a part takes 6 us. For 48 and 64 rows of 128
// channels of a request's own tokens (the heavy batch's 9 rows x 4 heads are of the
// former) the work kernel spills 19 and 47 registers, outside of the loops over
// tiles but for six reloads in the loop over pairs of own tiles of 64 rows.
// Against the attention that shares nothing (32 query and 8 kv heads of 128): the
// heavy batch 134 us and 199, with all 9 rows 214 and 261; 8 blocks of up to 6 rows
// behind 2,000 tokens 25 and 21: three launches pay from about 64 requests behind
// 2,000 tokens or 32 blocks behind 8,000 on.
#include <algorithm>
#include <climits>

#include "attend_kernel.h"

namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16;

constexpr int kMaxGroups = SV_MAX_GROUPS;
constexpr int kPlanWaves = 16;
constexpr int kRows = 128;          // rows of a workgroup of the prefix part
// A part has no fewer tiles than this: starting and ending one costs 6 us, of which
// more parts save less (8 requests behind 2,000 tokens: the work 14.9 and the join
// 5.0 us with 8, 16.7 and 6.9 with 4, 16.8 and 4.1 with 16).
constexpr int kLeastTiles = 8;
constexpr int kFewRows = 4096;      // of a call, a workgroup of the join each
constexpr long long kAcross = 1 << 16;  // of the join's workgroups in x; a dimension holds less than 2^32 threads

// What the plan leaves for a group that shares something.
struct Group {
    int first;          // first work item, and slot of partial results
    int tiles;          // whole tiles of the shared prefix
    int blocks, parts;  // row blocks; parts of the prefix
    int rows;           // rows of one head
    int tokens;         // where its list of block tokens starts
    int leader;         // the request whose pages are read
    int pad;
};

// Where the partial results of a request's shared prefix are: its rows (t group +
// head of the group) follow each other from `row` on among its group's; part i of
// row block n of head h lies in slot first + (i blocks + n) heads + h.
struct Prefix {
    int row, first, blocks, parts;
};

struct SharedArgs {
    AttendArgs a;       // of the requests' own tokens
    const int32_t* groups;
    const int32_t* shared_lens;
    int* skip;          // [B]: tiles of the request's shared prefix
    Prefix* prefix;     // [B]
    Group* group;       // [G]
    int* items;         // number of work items
    int* tokens;        // [B (K + 1)]: block tokens b (K + 1) + t, group by group
    float* prefix_o;    // [slot][kRows][D], not normalised
    float2* prefix_ml;  // [slot][kRows]: reference exponent, sum
    int G;
    int target;         // workgroups of the prefix part
    int tail_grid;      // workgroups for the requests' own tokens
};

// Inclusive prefix sum over a wavefront.
__device__ __forceinline__ unsigned long long wave_scan(unsigned long long v, int lane) {
    #pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const unsigned long long u = __shfl_up(v, o, 64);
        if (lane >= o) v += u;
    }
    return v;
}

// One workgroup. Requests are dealt to its wavefronts in sections; sums over them are
// of integers and places come from prefix sums in the requests' order, so nothing
// depends on the order of the atomics.
__global__ __launch_bounds__(64 * kPlanWaves) void shared_plan_kernel(SharedArgs s) {
    const AttendArgs& a = s.a;
    __shared__ int least[kMaxGroups], leader[kMaxGroups], members[kMaxGroups];
    __shared__ int count[kPlanWaves][kMaxGroups];   // block tokens by wavefront, then of those before it
    __shared__ Group found[kMaxGroups];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = ((a.B + kPlanWaves - 1) / kPlanWaves + 63) / 64 * 64;
    const int b0 = min(wave * per, a.B), b1 = min(b0 + per, a.B);
    // A request's group (-1: none) and block.
    auto request = [&](int b, Block& blk) {
        int g = -1;
        blk = Block{0, 0};
        if (b < b1) {
            g = s.groups[b];
            blk = block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, nullptr, false);
        }
        return blk.len > 0 && (unsigned)g < (unsigned)s.G ? g : -1;
    };
    Block blk;
    int g = request(b0 + lane, blk);            // the only one up to 1,024 requests
    int shared = tid < s.G ? s.shared_lens[tid] : 0;
    for (int i = tid; i < s.G; i += 64 * kPlanWaves) {
        least[i] = leader[i] = INT_MAX;
        members[i] = 0;
    }
    for (int i = lane; i < s.G; i += 64) count[wave][i] = 0;
    __syncthreads();
    for (int i = b0; i < b1; i += 64) {
        if (i > b0) g = request(i + lane, blk);
        if (g >= 0) {
            atomicMin(&least[g], blk.ctx);
            atomicMin(&leader[g], i + lane);
            atomicAdd(&members[g], 1);
            atomicAdd(&count[wave][g], blk.len);
        }
    }
    __syncthreads();
    if (tid < s.G) {
        Group m{};
        int n = 0;
        #pragma unroll
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = count[w][tid];
            count[w][tid] = n;
            n += c;
        }
        m.tiles = members[tid] >= 2 ? min(max(shared, 0), least[tid]) / kTile : 0;
        if (m.tiles > 0) {
            m.rows = n * a.group;
            m.blocks = (m.rows + kRows - 1) / kRows;
            m.tokens = n;
            m.leader = leader[tid];
        }
        found[tid] = m;
    }
    __syncthreads();
    if (wave == 0) {
        // The length of a part: all units' tiles over the workgroups that run at once,
        // rounded for each group, so that a part may be up to 1.5 times as long, or the
        // items a few more than the workgroups, some of which then take two (128 blocks
        // of 9 rows x 4 heads: 576 items on 512).
        const int heads = a.pages.heads, each = (s.G + 63) / 64, g0 = lane * each, g1 = min(g0 + each, s.G);
        unsigned long long work = 0, units = 0;
        for (int i = g0; i < g1; ++i) work += (unsigned long long)found[i].blocks * heads * found[i].tiles;
        work = wave_scan(work, lane);
        work = __shfl(work, 63, 64);
        const unsigned long long share = max((work + s.target - 1) / s.target, (unsigned long long)kLeastTiles);
        unsigned long long tokens = 0;
        for (int i = g0; i < g1; ++i) {
            const unsigned long long t = found[i].tiles;
            const int parts = t > 0 ? (int)min(max((t + share / 2) / share, 1ull), t) : 0;
            found[i].parts = parts;
            units += (unsigned long long)found[i].blocks * heads * parts;
            tokens += found[i].tokens;
        }
        const unsigned long long all = wave_scan(units, lane);
        int at = (int)(all - units), token = (int)(wave_scan(tokens, lane) - tokens);
        for (int i = g0; i < g1; ++i) {
            Group m = found[i];
            const int n = m.tokens;
            m.first = at;
            m.tokens = token;
            at += m.blocks * heads * m.parts;
            token += n;
            found[i] = m;
            s.group[i] = m;
        }
        if (lane == 63) *s.items = (int)all;
    }
    __syncthreads();
    for (int i = b0; i < b1; i += 64) {
        if (i > b0 || b1 - b0 > 64) g = request(i + lane, blk);
        if (g >= 0 && found[g].tiles == 0) g = -1;
        // Block tokens of earlier requests of the same group in this wavefront, group by group.
        int at = 0;
        unsigned long long left = __ballot(g >= 0);
        while (left != 0) {
            const int one = __builtin_amdgcn_readlane(g, __builtin_ctzll(left));
            const unsigned long long same = __ballot(g == one), before = same & ((1ull << lane) - 1);
            int sum = 0;
            #pragma unroll
            for (int bit = 0; bit < 6; ++bit) sum += __popcll(before & __ballot(blk.len >> bit & 1)) << bit;
            if (g == one) at = count[wave][g] + sum;
            left &= ~same;
        }
        if (i + lane < b1) {
            Prefix p{};
            int skip = 0;
            if (g >= 0) {
                atomicAdd(&count[wave][g], blk.len);
                const Group& m = found[g];
                skip = m.tiles;
                p = Prefix{at * a.group, m.first, m.blocks, m.parts};
                for (int t = 0; t < blk.len; ++t) s.tokens[m.tokens + at + t] = (i + lane) * (a.K + 1) + t;
            }
            s.prefix[i + lane] = p;
            s.skip[i + lane] = skip;
        }
    }
}

// An iteration's tiles (64 tokens of 128 channels), decoded by the whole workgroup:
// D threads a tile, each 16 bytes of its keys' and 16 of its values' codes.
struct Raw {
    uint4 keys, values;
    unsigned key_scales, value_scales;
};

template <int D>
struct Stage {
    using L = Tile<D>;
    static constexpr int kTiles = 256 / D;                      // tiles of an iteration
    static constexpr int kKeys = 64 * D, kBytes = 128 * D;      // bytes in LDS of a tile's keys, of both
    static constexpr int kStage = kTiles * kBytes;
    int tile;                       // which of the iteration's tiles
    unsigned from;                  // where in the tile the keys' codes are
    unsigned key_scale, key_shift, value_scale;
    unsigned key_to, value_to;      // where its first channels go in a stage

    __device__ __forceinline__ explicit Stage(int tid) {
        const int v = tid % D, lanes = D == 64 ? 8 : 16;
        tile = D == 64 ? scalar(tid / 64) : D == 128 ? scalar(tid / 128) : 0;
        from = 16 * v;
        const int in = v % lanes, quad = v / lanes % 4, half = v / (4 * lanes) % 2, plane = v / (8 * lanes);
        if constexpr (D == 64) {    // [half][unit of 16 channels][2 tokens]
            key_scale = L::kKScales + quad / 2 * 32 + 4 * in;
            key_shift = 8 * half;
            key_to = (2 * quad * kTile + 16 * half + 2 * in) * 16;
        } else {                    // [half][unit of 32 channels][token]
            const int unit = v / 16 % (D / 32), h = v / (D / 2);
            key_scale = L::kKScales + unit * 32 + 2 * (in & ~1);
            key_shift = 16 * (in & 1) + 8 * h;
            key_to = (4 * unit * kTile + 16 * h + in) * 16;
        }
        // [plane][half][quad][8 channels]
        value_scale = L::kVScales + (plane * 4 + in / 4) * 32 + 8 * quad + 4 * half;
        value_to = kKeys + ((2 * half + (quad & 1)) * D + plane * 16 + in) * 16 + (quad >> 1) * 8;
        key_to += tile * kBytes;
        value_to += tile * kBytes;
    }

    __device__ __forceinline__ void load(const uint8_t* at, Raw& r) const {
        r.keys = *reinterpret_cast<const uint4*>(at + from);
        r.values = *reinterpret_cast<const uint4*>(at + from + 16 * D);
        r.key_scales = *reinterpret_cast<const unsigned*>(at + key_scale);
        r.value_scales = *reinterpret_cast<const unsigned*>(at + value_scale);
    }

    __device__ __forceinline__ void decode(const Raw& r, unsigned char* stage) const {
        const unsigned kw[4] = {r.keys.x, r.keys.y, r.keys.z, r.keys.w}, ks = r.key_scales >> key_shift;
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float s = scale_of((D == 64 ? ks >> (16 * (i / 2)) : ks) & 255u);
            const u32x4 e = {decode2<0>(kw[i], s), decode2<1>(kw[i], s), decode2<2>(kw[i], s), decode2<3>(kw[i], s)};
            // 8 channels on, or (64 channels, the second token's) one token.
            *reinterpret_cast<u32x4*>(stage + key_to + (D == 64 ? i % 2 * kTile + i / 2 : i * kTile) * 16) = e;
        }
        const unsigned vw[4] = {r.values.x, r.values.y, r.values.z, r.values.w};
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            unsigned e[4];
            #pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float s = scale_of(r.value_scales >> (8 * n) & 255u);
                unsigned c = vw[n];      // 8 channels of token n
                if constexpr (D == 64) c = __builtin_amdgcn_perm(vw[2 + n / 2], vw[n / 2], n & 1 ? 0x07060302u : 0x05040100u);
                e[n] = j == 0 ? decode2<0>(c, s) : j == 1 ? decode2<1>(c, s) : j == 2 ? decode2<2>(c, s) : decode2<3>(c, s);
            }
            const uint2 even = make_uint2(__builtin_amdgcn_perm(e[1], e[0], 0x05040100u),
                                          __builtin_amdgcn_perm(e[3], e[2], 0x05040100u));
            const uint2 odd = make_uint2(__builtin_amdgcn_perm(e[1], e[0], 0x07060302u),
                                         __builtin_amdgcn_perm(e[3], e[2], 0x07060302u));
            *reinterpret_cast<uint2*>(stage + value_to + 2 * j * (D / 8) * 16) = even;
            *reinterpret_cast<uint2*>(stage + value_to + (2 * j + 1) * (D / 8) * 16) = odd;
        }
    }
};

__device__ __forceinline__ float pair_max(float v) {
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Work items first, first + step, ... of the prefix part; lds: two stages.
template <int D>
__device__ __forceinline__ void prefix_body(const SharedArgs& s, unsigned char* lds, int first, int step) {
    using S = Stage<D>;
    const AttendArgs& a = s.a;
    constexpr int kT = S::kTiles, kSteps = D / 16, kBlocks = D / 32;
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6);
    const int col = lane & 31, hi = lane >> 5;
    const S mine(tid);
    const int items = *s.items;
    for (int item = first; item < items; item += step) {
        // The item's group: the last that starts at or before it and has any.
        int g = 0;
        for (int g0 = 0; g0 < s.G; g0 += 64) {
            const int i = g0 + lane;
            const bool here = i < s.G && s.group[i].first <= item && s.group[i].parts > 0;
            const unsigned long long who = __ballot(here);
            if (who != 0) g = g0 + 63 - __builtin_clzll(who);
        }
        const Group grp = s.group[g];
        const int heads = a.pages.heads;
        int at = item - grp.first;
        const int h = scalar(at % heads);
        at /= heads;
        const int block = scalar(at % grp.blocks), part = scalar(at / grp.blocks);
        const int t0 = scalar((int)((long long)grp.tiles * part / grp.parts));
        const int t1 = scalar((int)((long long)grp.tiles * (part + 1) / grp.parts));
        const int leader = scalar(grp.leader);

        // The tile that the wavefront asks for next, and its page. The page comes by
        // a scalar load, whose wait is the barrier's: a vector load here would have
        // to wait for the tiles in flight.
        typedef const __attribute__((address_space(4))) int32_t* Table;
        const Table table = (Table)(a.pages.table + (size_t)leader * a.pages.max_pages);
        const unsigned page_bytes = (unsigned)(heads << (a.pages.shift - 5)) * Tile<D>::kBytes;
        const unsigned head_bytes = (unsigned)(h << (a.pages.shift - 5)) * Tile<D>::kBytes;
        const int in_page = (1 << (a.pages.shift - 5)) - 1;
        bool bad = false;
        int asked = min(t0 + mine.tile, t1 - 1), page = table[asked >> (a.pages.shift - 5)];
        auto fetch = [&](Raw& r) {
            const bool good = (unsigned)page < (unsigned)a.pages.num_pages;
            bad |= !good;
            // The first tiles of the cache stand in for those of a bad page (the
            // group is flagged and its outputs are undefined).
            const unsigned from_page = good ? (unsigned)page : 0u;
            const unsigned long long from = (unsigned long long)from_page * page_bytes + head_bytes +
                                            (unsigned)(asked & in_page) * Tile<D>::kBytes;
            mine.load(a.cache + from, r);
            asked = min(asked + kT, t1 - 1);        // past the end: the last tile
            page = table[asked >> (a.pages.shift - 5)];
        };
        Raw raw;
        fetch(raw);

        // The wavefront's 32 rows as right operands: lane holds row col, channels 16 j + 8 hi ...
        const int row0 = block * kRows + 32 * wave;
        u32x4 q[kSteps];
        {
            const bool some = row0 + col < grp.rows;
            const uint16_t* src = a.q;
            if (some) {
                const int row = row0 + col, token = s.tokens[grp.tokens + row / a.group];
                src += token * a.q_stride + (h * a.group + row % a.group) * D + 8 * hi;
            }
            #pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                q[j] = some ? *reinterpret_cast<const u32x4*>(src + 16 * j) : u32x4{0, 0, 0, 0};
                if (a.negate) q[j] ^= u32x4{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
            }
        }
        f32x16 o[kBlocks];
        #pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            #pragma unroll
            for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
        }
        float ref = kNegInf, sum = 0.0f;

        // An iteration's tiles are decoded while the ones before are worked on, and
        // asked for an iteration before that.
        svdma::ring_barrier();          // the last item's reads are done
        mine.decode(raw, lds);
        fetch(raw);
        int stage = 0;
        for (int t = t0; t < t1; t += kT) {
            svdma::ring_barrier();
            __builtin_amdgcn_s_setprio(0);
            const unsigned char* const now = lds + stage * S::kStage;
            stage ^= 1;
            f32x16 z[kT];
            #pragma unroll
            for (int u = 0; u < kT; ++u) {
                #pragma unroll
                for (int i = 0; i < 16; ++i) z[u][i] = 0.0f;
            }
            #pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                #pragma unroll
                for (int u = 0; u < kT; ++u) {
                    const bf16x8 k = *reinterpret_cast<const bf16x8*>(now + u * S::kBytes + ((2 * j + hi) * kTile + col) * 16);
                    z[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, __builtin_bit_cast(bf16x8, q[j]), z[u], 0, 0, 0);
                }
            }
            mine.decode(raw, lds + stage * S::kStage);
            fetch(raw);
            #pragma unroll
            for (int u = 1; u < kT; ++u) {
                if (t + u >= t1) {
                    #pragma unroll
                    for (int i = 0; i < 16; ++i) z[u][i] = kNegInf;
                }
            }
            const bool fresh = ref == kNegInf;
            const float base = fresh ? 0.0f : ref;
            float top = kNegInf;
            #pragma unroll
            for (int u = 0; u < kT; ++u) {
                #pragma unroll
                for (int i = 0; i < 16; i += 2) top = fmaxf(fmaxf(top, z[u][i]), z[u][i + 1]);
            }
            top = __builtin_fmaf(top, a.c, -base);
            if (__ballot(top > (fresh ? kNegInf : 8.0f)) != 0) {
                top = pair_max(top);
                const float next = fresh ? top : fmaxf(base, base + top);
                const float keep = fresh ? 0.0f : exp2_fast(base - next);
                ref = next;
                sum *= keep;
                #pragma unroll
                for (int j = 0; j < kBlocks; ++j) o[j] *= keep;
            }
            const float off = ref == kNegInf ? 0.0f : ref;
            // Of two wavefronts on a SIMD the one past its scores goes first, so that they
            // do not do the same at the same time (128 requests behind 8,192 tokens: the
            // work kernel 132.7 us with it, 136.8 without).
            __builtin_amdgcn_s_setprio(2);
            #pragma unroll
            for (int u = 0; u < kT; ++u) {
                float e[16];
                #pragma unroll
                for (int i = 0; i < 16; ++i) e[i] = exp2_fast(__builtin_fmaf(z[u][i], a.c, -off));
                float add = 0.0f;
                #pragma unroll
                for (int i = 0; i < 16; i += 4) add += (e[i] + e[i + 1]) + (e[i + 2] + e[i + 3]);
                sum += add;
                #pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float* f = e + 8 * half;
                    const u32x4 w = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                     pack_bf16(f[6], f[7])};
                    #pragma unroll
                    for (int j = 0; j < kBlocks; ++j) {
                        const bf16x8 v = *reinterpret_cast<const bf16x8*>(now + u * S::kBytes + S::kKeys + ((2 * half + hi) * D + 32 * j + col) * 16);
                        o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, __builtin_bit_cast(bf16x8, w), o[j], 0, 0, 0);
                    }
                }
            }
        }
        __builtin_amdgcn_s_setprio(0);
        if (bad) flag(a.status, SV_FLAG_BAD_PAGE);
        // Results row by row: 64 channels at a time through the wavefront's part of
        // the stage, where 4 channels of row n lie n places on (mod 16).
        svdma::ring_barrier();
        f32x4* const turn = reinterpret_cast<f32x4*>(lds) + wave * 512;
        const float all = pair_sum(sum);
        const long long place0 = (long long)item * kRows + 32 * wave;
        if (hi == 0 && row0 + col < grp.rows) s.prefix_ml[place0 + col] = make_float2(ref, all);
        #pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            #pragma unroll
            for (int j = 0; j < kBlocks; ++j) {
                #pragma unroll
                for (int i = 0; i < 16; ++i) {
                    // Place 32 j + 8 (i / 4) + 4 hi + i % 4 holds channel 8 (place % (D / 8)) + place / (D / 8).
                    const int low = 32 * j + 8 * (i / 4) + i % 4;       // place of hi = 0
                    if (low % (D / 8) / 8 != c) continue;
                    const int ch = low % (D / 8) % 8 * 8 + low / (D / 8) + 32 * hi;    // of the 64
                    reinterpret_cast<float*>(turn + col * 16 + ((ch / 4 + col) & 15))[ch % 4] = o[j][i];
                }
            }
            #pragma unroll
            for (int n = 0; n < 8; ++n) {
                const int row = 4 * n + (lane >> 4);
                const f32x4 v = turn[row * 16 + ((lane + row) & 15)];
                if (row0 + row < grp.rows) {
                    *reinterpret_cast<f32x4*>(s.prefix_o + (place0 + row) * D + 64 * c + 4 * (lane & 15)) = v;
                }
            }
        }
    }
}

// Wavefronts of a SIMD at once: 256 channels take most of its registers.
template <int D>
constexpr int shared_occupancy() { return D == 256 ? 1 : 2; }

template <int D, int kMT>
__global__ __launch_bounds__(256, shared_occupancy<D>()) void shared_work_kernel(SharedArgs s) {
    typedef Lds<D, kMT, kFew> Own;
    constexpr size_t kStages = 2 * Stage<D>::kStage, kBytes = kStages > sizeof(Own) ? kStages : sizeof(Own);
    __shared__ __attribute__((aligned(16))) unsigned char lds[kBytes];
    const int g = blockIdx.x;
    if (g < s.target) prefix_body<D>(s, lds, g, s.target);
    else attend_body<D, kMT, kFew, kTail>(s.a, *reinterpret_cast<Own*>(lds), g - s.target, s.tail_grid);
}

// A workgroup joins 1024 / D rows of the outputs, D / 4 lanes and 4 channels a lane
// each, or (kSplit) one row, whose parts are dealt to its 1024 / D sets of lanes: few
// rows may have many parts each. The prefix's parts, then the request's own;
// kDeep of them in flight.
template <int D, bool kSplit>
__global__ __launch_bounds__(256) void shared_join_kernel(SharedArgs s, int unit_rows) {
    const AttendArgs& a = s.a;
    constexpr int kLanes = D / 4, kSets = 256 / kLanes, kDeep = 4, kBy = kSplit ? kSets : 1;
    __shared__ Joined sh[kSplit ? 256 : 1];
    const int set = threadIdx.x / kLanes, ch = threadIdx.x % kLanes * 4;
    const long long row = kSplit ? blockIdx.x : ((long long)blockIdx.y * gridDim.x + blockIdx.x) * kSets + set;
    if (row >= (long long)a.B * (a.K + 1) * a.Hq) return;
    const int head = (int)(row % a.Hq), b = (int)(row / a.Hq / (a.K + 1)), t = (int)(row / a.Hq % (a.K + 1));
    const Block blk = block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, nullptr, false);
    if (t >= blk.len) return;
    const int h = head / a.group, r = t * a.group + (head - h * a.group);
    const Prefix p = s.prefix[b];
    const int2 unit = a.units[(b * a.pages.heads + h) * a.row_blocks + r / unit_rows];
    const int at = p.row + r, n = p.parts + unit.y;
    Joined j{kNegInf, 0.0f, {0, 0, 0, 0}};
    for (int i = kSplit ? set : 0; i < n; i += kDeep * kBy) {
        float2 m[kDeep];
        f32x4 v[kDeep];
        #pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int x = min(i + k * kBy, n - 1);
            const bool shared = x < p.parts;
            const long long place =
                shared ? (p.first + ((long long)x * p.blocks + at / kRows) * a.pages.heads + h) * kRows + at % kRows
                       : (long long)slot_of(unit.x, x - p.parts) * unit_rows + r % unit_rows;
            m[k] = (shared ? s.prefix_ml : a.part_ml)[place];
            v[k] = *reinterpret_cast<const f32x4*>((shared ? s.prefix_o : a.part_o) + place * D + ch);
        }
        #pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            if (i + k * kBy < n) j.add(m[k].x, m[k].y, v[k]);
        }
    }
    if constexpr (kSplit) {
        sh[threadIdx.x] = j;
        __syncthreads();
        if (set > 0) return;
        #pragma unroll
        for (int k = 1; k < kSets; ++k) {
            const Joined& other = sh[k * kLanes + threadIdx.x];
            j.add(other.ref, other.sum, other.acc);
        }
    }
    const float inv = 1.0f / j.sum;
    const unsigned w[2] = {pack_bf16(j.acc[0] * inv, j.acc[1] * inv), pack_bf16(j.acc[2] * inv, j.acc[3] * inv)};
    __builtin_memcpy(__builtin_assume_aligned(a.out + row * D + ch, 8), w, 8);
}

// What the host fixes of a call.
struct SharedPlan {
    Plan tail;
    int target;             // workgroups of the prefix part
    size_t parts;           // rows of the tails' partial results
    size_t at_skip, at_prefix, at_group, at_tokens, at_ml, at_o, at_units, at_part_ml, at_part_o, bytes;
};

SharedPlan shared_plan_of(int B, int K, int G, int Hq, int kv_heads, int D, int page_size, int max_pages) {
    SharedPlan p;
    p.target = 256 * (D == 256 ? shared_occupancy<256>() : shared_occupancy<128>());
    p.tail = plan_of(B, K, Hq, kv_heads, D, page_size, max_pages, 0, 0, p.target);
    // Items: a group has no more than its share of the target and one a unit.
    const size_t rows = (size_t)B * (K + 1) * (Hq / kv_heads);
    const size_t items = p.target + kv_heads * (rows / kRows + std::min(G, std::max(B / 2, 1)));
    const size_t units = (size_t)B * kv_heads * p.tail.row_blocks;
    p.parts = (p.tail.slots + units) * 16 * p.tail.mt;
    size_t at = 256;        // the number of items
    auto take = [&](size_t n) {
        const size_t was = at;
        at += round256(n);
        return was;
    };
    p.at_skip = take((size_t)B * sizeof(int));
    p.at_prefix = take((size_t)B * sizeof(Prefix));
    p.at_group = take((size_t)G * sizeof(Group));
    p.at_tokens = take((size_t)B * (K + 1) * sizeof(int));
    p.at_ml = take(items * kRows * sizeof(float2));
    p.at_o = take(items * kRows * D * sizeof(float));
    p.at_units = take(units * sizeof(int2));
    p.at_part_ml = take(p.parts * sizeof(float2));
    p.at_part_o = take(p.parts * D * sizeof(float));
    p.bytes = at;
    return p;
}

template <int D>
void launch_shared(const SharedArgs& s, const SharedPlan& p, hipStream_t stm) {
    const dim3 grid((unsigned)(p.target + p.tail.grid));
    switch (p.tail.mt) {
        case 1: hipLaunchKernelGGL((shared_work_kernel<D, 1>), grid, dim3(256), 0, stm, s); break;
        case 2: hipLaunchKernelGGL((shared_work_kernel<D, 2>), grid, dim3(256), 0, stm, s); break;
        case 3: hipLaunchKernelGGL((shared_work_kernel<D, (D == 256 ? 2 : 3)>), grid, dim3(256), 0, stm, s); break;
        default: hipLaunchKernelGGL((shared_work_kernel<D, (D == 256 ? 2 : 4)>), grid, dim3(256), 0, stm, s); break;
    }
    // The fewer rows, the more parts each may have (at most the prefix part's workgroups).
    const long long rows = (long long)s.a.B * (s.a.K + 1) * s.a.Hq;
    if (rows <= kFewRows) {
        hipLaunchKernelGGL((shared_join_kernel<D, true>), dim3((unsigned)rows), dim3(256), 0, stm, s, 16 * p.tail.mt);
    } else {
        const long long joins = (rows * D + 1023) / 1024;
        const dim3 across((unsigned)std::min(joins, kAcross), (unsigned)((joins + kAcross - 1) / kAcross));
        hipLaunchKernelGGL((shared_join_kernel<D, false>), across, dim3(256), 0, stm, s, 16 * p.tail.mt);
    }
}

}  // namespace

extern "C" size_t spec_verify_attention_shared_workspace_bytes(int B, int K, int G, int q_heads,
                                                               int kv_heads, int head_dim,
                                                               int page_size, int max_pages) {
    if (B < 1 || G < 0 || G > kMaxGroups || !shape_ok(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, 0)) {
        return 0;
    }
    if (G == 0) return workspace_of(plan_of(B, K, q_heads, kv_heads, head_dim, page_size, max_pages, 0), head_dim);
    return shared_plan_of(B, K, G, q_heads, kv_heads, head_dim, page_size, max_pages).bytes;
}

extern "C" int spec_verify_attention_shared(const void* queries, int64_t query_stride, const void* cache,
                                            const int32_t* page_table, const int32_t* ctx_lens,
                                            const int32_t* budgets, const int32_t* groups,
                                            const int32_t* shared_lens, int B, int K, int G,
                                            int q_heads, int kv_heads, int head_dim, int page_size,
                                            int max_pages, int num_pages, float scale, void* out,
                                            int32_t* out_status, void* workspace,
                                            size_t workspace_bytes, void* stream) {
    if (G < 0 || G > kMaxGroups) return SV_ERR_ARG;
    if (G == 0) {
        return spec_verify_attention(queries, query_stride, cache, page_table, ctx_lens, budgets, B, K,
                                     q_heads, kv_heads, head_dim, page_size, max_pages, num_pages, scale, 0,
                                     out, out_status, workspace, workspace_bytes, stream);
    }
    const int rc = check(queries, query_stride, cache, page_table, ctx_lens, budgets, B, K, q_heads,
                         kv_heads, head_dim, page_size, max_pages, num_pages, scale, 0, out, out_status,
                         workspace);
    if (rc != SV_OK || B == 0) return rc;
    if (!groups || !shared_lens) return SV_ERR_NULL;
    if (!aligned(groups, 4) || !aligned(shared_lens, 4)) return SV_ERR_ALIGN;
    const SharedPlan p = shared_plan_of(B, K, G, q_heads, kv_heads, head_dim, page_size, max_pages);
    if (workspace_bytes < p.bytes) return SV_ERR_ARG;
    char* ws = static_cast<char*>(workspace);
    SharedArgs s{};
    s.a = args_of(p.tail, queries, query_stride, cache, page_table, ctx_lens, budgets, B, K, q_heads, kv_heads,
                  page_size, max_pages, num_pages, scale, out, out_status, ws + p.at_units);
    s.a.skip = s.skip = reinterpret_cast<int*>(ws + p.at_skip);
    s.a.units = reinterpret_cast<int2*>(ws + p.at_units);
    s.a.whole = p.tail.slots;
    s.a.part_ml = reinterpret_cast<float2*>(ws + p.at_part_ml);
    s.a.part_o = reinterpret_cast<float*>(ws + p.at_part_o);
    s.groups = groups;
    s.shared_lens = shared_lens;
    s.items = reinterpret_cast<int*>(ws);
    s.prefix = reinterpret_cast<Prefix*>(ws + p.at_prefix);
    s.group = reinterpret_cast<Group*>(ws + p.at_group);
    s.tokens = reinterpret_cast<int*>(ws + p.at_tokens);
    s.prefix_ml = reinterpret_cast<float2*>(ws + p.at_ml);
    s.prefix_o = reinterpret_cast<float*>(ws + p.at_o);
    s.G = G;
    s.target = p.target;
    s.tail_grid = p.tail.grid;
    const hipStream_t stm = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(shared_plan_kernel, dim3(1), dim3(64 * kPlanWaves), 0, stm, s);
    if (head_dim == 64) launch_shared<64>(s, p, stm);
    else if (head_dim == 128) launch_shared<128>(s, p, stm);
    else launch_shared<256>(s, p, stm);
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
