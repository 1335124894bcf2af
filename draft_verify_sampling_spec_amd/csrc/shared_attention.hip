// shared_attention.hip -- attention of drafted blocks for requests that share a
// long prefix, for MI355X (gfx950).
//
// The mathematics: a softmax over positions [0, p] is joined from its parts over
// [0, s) and [s, p]. The requests of a group hold the same tokens up to s, so the
// part in front of s is a product of all their rows with one set of keys and
// values, which no row masks: it is computed once a group, from the pages of the
// group's first request. Every request's own tokens go through the kernels of
// attend_kernel.h, which join the parts where a row's outputs are written.
//
// Three steps:
//  - plan (one workgroup): for every group the tokens that are shared and whose
//    tiles are whole (up to the shortest context), the list of its rows, and into
//    how many parts of the prefix its work is cut;
//  - prefix: a workgroup takes 4 kRows rows of one head and a part of the prefix;
//  - tails: attention from the first own tile on, and the join.
//
// Prefix kernel. With many rows a tile's keys and values serve many products, so
// the tile is decoded once a workgroup into LDS, as the operands of 32x32x16
// matrix instructions: keys [8 channels' chunk][token][8], values transposed,
// [8 tokens' chunk][channel][8], every read and write of a wavefront a run without bank
// conflicts. Scores are formed transposed, K Q^T: a lane holds one row and
// 16 of the tile's 32 tokens, in the order in which the value product contracts
// them, so probabilities go from one product to the next in registers. The
// values' channels lie in an order (channel 8 x + j at place j D / 8 + x) that the
// decoding lanes write without conflicts; it is undone when results are stored.
// The next tiles' bytes are asked for in registers kAhead tiles ahead.
#include <climits>

#include "attend_kernel.h"

namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16;

constexpr int kMaxGroups = SV_MAX_GROUPS;
constexpr int kPlanWaves = 16;
constexpr int kLeastTiles = 4;      // of a part

// What the plan leaves for a group.
struct Group {
    int first;          // first work item (and slot of partial results)
    int tiles;          // whole tiles of the shared prefix
    int blocks, parts;  // row blocks; parts of the prefix
    int rows;           // rows of one head
    int tokens;         // where its list of block tokens starts
    int leader;         // the request whose pages are read
    int pad;
};

struct SharedArgs {
    AttendArgs a;
    const int32_t* groups;
    const int32_t* shared_lens;
    Prefix* prefix;     // [B]
    Group* group;       // [G]
    int* items;         // number of work items
    int* tokens;        // [B (K + 1)]: block tokens b (K + 1) + t, group by group
    float* prefix_o;
    float2* prefix_ml;
    int G, target;
};

__device__ __forceinline__ unsigned long long wave_scan(unsigned long long v, int lane) {
    #pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const unsigned long long u = __shfl_up(v, o, 64);
        if (lane >= o) v += u;
    }
    return v;
}

// One workgroup. Sums over requests are of integers, places come from prefix
// sums in the requests' order: nothing depends on the order of the atomics.
__global__ __launch_bounds__(64 * kPlanWaves) void shared_plan_kernel(SharedArgs s) {
    const AttendArgs& a = s.a;
    __shared__ int least[kMaxGroups], leader[kMaxGroups], members[kMaxGroups];
    __shared__ int count[kPlanWaves][kMaxGroups];   // block tokens by wavefront, then of those before it
    __shared__ int parts[kMaxGroups], first[kMaxGroups], start[kMaxGroups];
    __shared__ unsigned long long sums[kPlanWaves][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int g = tid; g < s.G; g += 64 * kPlanWaves) {
        least[g] = leader[g] = INT_MAX;
        members[g] = 0;
    }
    for (int i = tid; i < kPlanWaves * s.G; i += 64 * kPlanWaves) count[i / s.G][i % s.G] = 0;
    __syncthreads();
    // A wavefront's requests.
    const int per = ((a.B + kPlanWaves - 1) / kPlanWaves + 63) / 64 * 64;
    const int b0 = min(wave * per, a.B), b1 = min(b0 + per, a.B);
    for (int b = b0 + lane; b < b1; b += 64) {
        const Block blk = block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, nullptr, false);
        const int g = s.groups[b];
        if (blk.len > 0 && (unsigned)g < (unsigned)s.G) {
            atomicMin(&least[g], blk.ctx);
            atomicMin(&leader[g], b);
            atomicAdd(&members[g], 1);
            atomicAdd(&count[wave][g], blk.len);
        }
    }
    __syncthreads();
    // Groups: at most one a thread.
    const int g = tid, rows_of_block = 1 << a.prefix_shift;
    Group mine{};
    int n = 0;
    if (g < s.G) {
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = count[w][g];
            count[w][g] = n;
            n += c;
        }
        mine.tiles = members[g] >= 2 ? min(max(s.shared_lens[g], 0), least[g]) / kTile : 0;
        mine.rows = n * a.group;
        mine.blocks = (mine.rows + rows_of_block - 1) >> a.prefix_shift;
        mine.leader = leader[g];
    }
    // Tiles of all units over the workgroups that run at once: the parts' length.
    auto total = [&](unsigned long long v, int k) {
        v = wave_scan(v, lane);
        if (lane == 63) sums[wave][k] = v;
        __syncthreads();
        unsigned long long all = 0, before = 0;
        for (int w = 0; w < kPlanWaves; ++w) {
            if (w < wave) before += sums[w][k];
            all += sums[w][k];
        }
        __syncthreads();
        struct { unsigned long long upto, all; } r{before + v, all};
        return r;
    };
    const unsigned long long units = (unsigned long long)mine.blocks * a.pages.heads;
    const unsigned long long work = total(units * mine.tiles, 0).all;
    const unsigned long long share = max((work + s.target - 1) / s.target, (unsigned long long)kLeastTiles);
    mine.parts = mine.tiles > 0 ? (int)min(max((mine.tiles + share / 2) / share, 1ull), (unsigned long long)mine.tiles) : 0;
    const auto items = total(units * mine.parts, 0);
    const auto tokens = total(mine.tiles > 0 ? n : 0, 1);
    if (g < s.G) {
        mine.first = (int)(items.upto - units * mine.parts);
        mine.tokens = (int)tokens.upto - (mine.tiles > 0 ? n : 0);
        parts[g] = mine.parts;
        first[g] = mine.first;
        start[g] = mine.tokens;
        s.group[g] = mine;
        least[g] = mine.tiles;
        members[g] = mine.blocks;
    }
    if (tid == 0) *s.items = (int)items.all;
    __syncthreads();
    for (int i0 = b0; i0 < b1; i0 += 64) {
        const int b = i0 + lane;
        Block blk{0, 0};
        int g = -1;
        if (b < b1) {
            blk = block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, nullptr, false);
            g = s.groups[b];
            if (blk.len == 0 || (unsigned)g >= (unsigned)s.G || least[g] == 0) g = -1;
        }
        int at = g >= 0 ? count[wave][g] : 0;
        #pragma unroll
        for (int j = 0; j < 64; ++j) {
            const int other = __builtin_amdgcn_readlane(g, j), len = __builtin_amdgcn_readlane(blk.len, j);
            if (j < lane && other == g) at += len;
        }
        Prefix p{};
        if (g >= 0) {
            atomicAdd(&count[wave][g], blk.len);
            p.tiles = least[g];
            p.row = at * a.group;
            p.first = first[g];
            p.blocks = members[g];
            p.parts = parts[g];
            for (int t = 0; t < blk.len; ++t) s.tokens[start[g] + at + t] = b * (a.K + 1) + t;
        }
        if (b < b1) s.prefix[b] = p;
    }
}

// 16 bytes of a tile's codes and their scales, as one thread decodes them. Keys
// come first: pieces [0, D) are theirs, [D, 2 D) the values'.
struct Piece {
    uint4 codes;
    unsigned scales;
};

template <int D>
struct Stage {
    using L = Tile<D>;
    static constexpr int kTiles = D == 64 ? 2 : 1;              // tiles of an iteration
    static constexpr int kPieces = 2 * D * kTiles / 256;        // of a thread
    static constexpr int kKeys = 64 * D, kBytes = 128 * D;      // bytes in LDS of a tile's keys, of both

    static __device__ __forceinline__ Piece load(const uint8_t* tile, int q) {
        Piece p;
        p.codes = *reinterpret_cast<const uint4*>(tile + 16 * q);
        if (q < D) {
            if constexpr (D == 64) {    // [half][unit of 16 channels][2 tokens]
                const int half = q / 32, unit = q / 8 % 4, m = q % 8;
                p.scales = *reinterpret_cast<const unsigned*>(tile + L::kKScales + unit / 2 * 32 + 4 * m) >> (8 * half);
            } else {                    // [half][unit of 32 channels][token]
                const int half = q / (D / 2), unit = q / 16 % (D / 32), tok = q % 16;
                p.scales = tile[L::kKScales + unit * 32 + 2 * tok + half];
            }
        } else {
            const int v = q - D, lanes = D == 64 ? 8 : 16;
            const int x = v % lanes, quad = v / lanes % 4, half = v / (4 * lanes) % 2, plane = v / (8 * lanes);
            const int group = plane * 4 + x / 4;
            p.scales = *reinterpret_cast<const unsigned*>(tile + L::kVScales + group * 32 + 8 * quad + 4 * half);
        }
        return p;
    }

    static __device__ __forceinline__ void decode(const Piece& p, int q, unsigned char* lds) {
        const unsigned w[4] = {p.codes.x, p.codes.y, p.codes.z, p.codes.w};
        if (q < D) {
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                int tok, chunk;
                float s;
                if constexpr (D == 64) {
                    const int half = q / 32, unit = q / 8 % 4, m = q % 8;
                    tok = 16 * half + 2 * m + i / 2;
                    chunk = 2 * unit + i % 2;
                    s = scale_of(p.scales >> (16 * (i / 2)) & 255u);
                } else {
                    const int half = q / (D / 2), unit = q / 16 % (D / 32);
                    tok = 16 * half + q % 16;
                    chunk = 4 * unit + i;
                    s = scale_of(p.scales);
                }
                const u32x4 e = {decode2<0>(w[i], s), decode2<1>(w[i], s), decode2<2>(w[i], s), decode2<3>(w[i], s)};
                *reinterpret_cast<u32x4*>(lds + (chunk * kTile + tok) * 16) = e;
            }
        } else {
            const int v = q - D, lanes = D == 64 ? 8 : 16;
            const int x = v % lanes, quad = v / lanes % 4, half = v / (4 * lanes) % 2, plane = v / (8 * lanes);
            unsigned c[4];      // 8 channels of each token
            #pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (D == 64) c[r] = __builtin_amdgcn_perm(w[2 + r / 2], w[r / 2], r & 1 ? 0x07060302u : 0x05040100u);
                else c[r] = w[r];
            }
            float s[4];
            #pragma unroll
            for (int r = 0; r < 4; ++r) s[r] = scale_of(p.scales >> (8 * r) & 255u);
            unsigned char* to = lds + kKeys + ((2 * half + (quad & 1)) * D + plane * 16 + x) * 16 + (quad >> 1) * 8;
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                unsigned e[4];
                #pragma unroll
                for (int r = 0; r < 4; ++r) {
                    e[r] = j == 0   ? decode2<0>(c[r], s[r])
                           : j == 1 ? decode2<1>(c[r], s[r])
                           : j == 2 ? decode2<2>(c[r], s[r])
                                    : decode2<3>(c[r], s[r]);
                }
                const uint2 even = make_uint2(__builtin_amdgcn_perm(e[1], e[0], 0x05040100u),
                                              __builtin_amdgcn_perm(e[3], e[2], 0x05040100u));
                const uint2 odd = make_uint2(__builtin_amdgcn_perm(e[1], e[0], 0x07060302u),
                                             __builtin_amdgcn_perm(e[3], e[2], 0x07060302u));
                *reinterpret_cast<uint2*>(to + (2 * j) * (D / 8) * 16) = even;
                *reinterpret_cast<uint2*>(to + (2 * j + 1) * (D / 8) * 16) = odd;
            }
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

template <int D>
__global__ __launch_bounds__(256, 2) void shared_prefix_kernel(SharedArgs s) {
    using S = Stage<D>;
    const AttendArgs& a = s.a;
    constexpr int kSteps = D / 16, kBlocks = D / 32, kAhead = 2;
    __shared__ __attribute__((aligned(16))) unsigned char lds[2][S::kTiles * S::kBytes];
    const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6);
    const int col = lane & 31, hi = lane >> 5;
    const int items = *s.items;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
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

        // The wavefront's 32 rows as right operands: lane holds row col, channels 16 j + 8 hi ...
        const int row = (block << a.prefix_shift) + 32 * wave + col;
        u32x4 q[kSteps];
        const bool some = row < grp.rows;
        const uint16_t* src = a.q;
        if (some) {
            const int token = s.tokens[grp.tokens + row / a.group];
            src += token * a.q_stride + (h * a.group + row % a.group) * D + 8 * hi;
        }
        #pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            q[j] = some ? *reinterpret_cast<const u32x4*>(src + 16 * j) : u32x4{0, 0, 0, 0};
            if (a.negate) q[j] ^= u32x4{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
        }

        f32x16 o[kBlocks];
        #pragma unroll
        for (int j = 0; j < kBlocks; ++j) {
            #pragma unroll
            for (int i = 0; i < 16; ++i) o[j][i] = 0.0f;
        }
        float ref = kNegInf, sum = 0.0f;

        // Page numbers of 64 tiles, one a lane.
        int pages = 0, paged = -64;
        bool bad = false;
        auto fetch = [&](int t, Piece (&p)[S::kPieces]) {
            #pragma unroll
            for (int k = 0; k < S::kPieces; ++k) {
                // Past the part's end the last tile stands in.
                const int piece = tid + 256 * k;
                const int tile = min(t + (S::kTiles > 1 ? k * 256 / (2 * D) + tid / (2 * D) : 0), t1 - 1);
                const int q = piece % (2 * D);
                long long from;
                if constexpr (S::kTiles > 1) {
                    from = a.pages.tile(leader, h, tile * kTile, Tile<D>::kBytes);
                } else {
                    if (tile - paged >= 64) {
                        paged = tile;
                        pages = a.pages.page(leader, min(tile + lane, t1 - 1) * kTile);
                    }
                    from = a.pages.tile_in(__builtin_amdgcn_readlane(pages, tile - paged), h, tile * kTile,
                                           Tile<D>::kBytes);
                }
                if (from < 0) {
                    bad = true;
                    from = 0;
                }
                p[k] = S::load(a.cache + from, q);
            }
        };
        auto stage = [&](const Piece (&p)[S::kPieces], int buf) {
            #pragma unroll
            for (int k = 0; k < S::kPieces; ++k) {
                const int piece = tid + 256 * k;
                S::decode(p[k], piece % (2 * D), lds[buf] + piece / (2 * D) * S::kBytes);
            }
        };
        Piece ahead[kAhead][S::kPieces];
        #pragma unroll
        for (int k = 0; k < kAhead; ++k) fetch(t0 + k * S::kTiles, ahead[k]);
        svdma::ring_barrier();          // the last item's reads are done
        stage(ahead[0], 0);
        int buf = 0;
        for (int t = t0; t < t1; t += S::kTiles) {
            svdma::ring_barrier();
            #pragma unroll
            for (int k = 0; k + 1 < kAhead; ++k) {
                #pragma unroll
                for (int i = 0; i < S::kPieces; ++i) ahead[k][i] = ahead[k + 1][i];
            }
            fetch(t + kAhead * S::kTiles, ahead[kAhead - 1]);
            if (t + S::kTiles < t1) stage(ahead[0], buf ^ 1);
            #pragma unroll
            for (int u = 0; u < S::kTiles; ++u) {
                if (S::kTiles > 1 && t + u >= t1) break;
                const unsigned char* keys = lds[buf] + u * S::kBytes;
                const unsigned char* values = keys + S::kKeys;
                f32x16 z;
                #pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = 0.0f;
                #pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                    const bf16x8 k = *reinterpret_cast<const bf16x8*>(keys + ((2 * j + hi) * kTile + col) * 16);
                    z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, __builtin_bit_cast(bf16x8, q[j]), z, 0, 0, 0);
                }
                const bool fresh = ref == kNegInf;
                float base = fresh ? 0.0f : ref;
                float e[16];
                #pragma unroll
                for (int i = 0; i < 16; ++i) e[i] = __builtin_fmaf(z[i], a.c, -base);
                float top = e[0];
                #pragma unroll
                for (int i = 1; i < 16; ++i) top = fmaxf(top, e[i]);
                if (__ballot(top > (fresh ? kNegInf : 8.0f)) != 0) {
                    top = pair_max(top);
                    const float next = fresh ? top : fmaxf(base, base + top);
                    const float keep = fresh ? 0.0f : exp2_fast(base - next);
                    const float off = next == kNegInf ? 0.0f : next;
                    ref = next;
                    sum *= keep;
                    #pragma unroll
                    for (int j = 0; j < kBlocks; ++j) o[j] *= keep;
                    #pragma unroll
                    for (int i = 0; i < 16; ++i) e[i] = __builtin_fmaf(z[i], a.c, -off);
                }
                #pragma unroll
                for (int i = 0; i < 16; ++i) e[i] = exp2_fast(e[i]);
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
                        const bf16x8 v = *reinterpret_cast<const bf16x8*>(values + ((2 * half + hi) * D + 32 * j + col) * 16);
                        o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, __builtin_bit_cast(bf16x8, w), o[j], 0, 0, 0);
                    }
                }
            }
            buf ^= 1;
        }
        if (bad) flag(a.status, SV_FLAG_BAD_PAGE);
        sum = pair_sum(sum);
        const long long slot = ((long long)item << a.prefix_shift) + 32 * wave + col;
        if (some) {
            if (hi == 0) s.prefix_ml[slot] = make_float2(ref, sum);
            float* to = s.prefix_o + slot * D;
            #pragma unroll
            for (int j = 0; j < kBlocks; ++j) {
                #pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int place = 32 * j + 8 * (i / 4) + 4 * hi + i % 4;
                    to[place % (D / 8) * 8 + place / (D / 8)] = o[j][i];
                }
            }
        }
    }
}

// What the host fixes of a call.
struct SharedPlan {
    Plan tail;
    int shift;              // log2 of a row block's rows
    int target;             // workgroups of the prefix kernel
    size_t slots;           // work items, at most
    size_t at_prefix, at_group, at_tokens, at_ml, at_o, at_tail, bytes;
};

SharedPlan shared_plan_of(int B, int K, int G, int Hq, int kv_heads, int D, int page_size, int max_pages) {
    SharedPlan p;
    p.tail = plan_of(B, K, Hq, kv_heads, D, page_size, max_pages, 0);
    p.shift = 7;
    p.target = 512;
    // Items: a group has no more than its share of the target and one a unit.
    const size_t rows = (size_t)B * (K + 1) * (Hq / kv_heads);
    const size_t units = kv_heads * ((rows >> p.shift) + std::min(G, std::max(B / 2, 1)));
    p.slots = p.target + units;
    size_t at = 256;        // the number of items
    auto take = [&](size_t n) {
        const size_t was = at;
        at += round256(n);
        return was;
    };
    p.at_prefix = take((size_t)B * sizeof(Prefix));
    p.at_group = take((size_t)G * sizeof(Group));
    p.at_tokens = take((size_t)B * (K + 1) * sizeof(int));
    p.at_ml = take((p.slots << p.shift) * sizeof(float2));
    p.at_o = take((p.slots << p.shift) * D * sizeof(float));
    p.at_tail = take(workspace_of(p.tail, D));
    p.bytes = at;
    return p;
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
                  page_size, max_pages, num_pages, scale, out, out_status, ws + p.at_tail);
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
    s.a.prefix = s.prefix;
    s.a.prefix_ml = s.prefix_ml;
    s.a.prefix_o = s.prefix_o;
    s.a.prefix_shift = p.shift;
    const hipStream_t stm = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(shared_plan_kernel, dim3(1), dim3(64 * kPlanWaves), 0, stm, s);
    const dim3 grid((unsigned)p.target);
    switch (head_dim) {
        case 64: hipLaunchKernelGGL((shared_prefix_kernel<64>), grid, dim3(256), 0, stm, s); break;
        case 128: hipLaunchKernelGGL((shared_prefix_kernel<128>), grid, dim3(256), 0, stm, s); break;
        default: hipLaunchKernelGGL((shared_prefix_kernel<256>), grid, dim3(256), 0, stm, s); break;
    }
    return launch_attend<kTail>(s.a, p.tail, head_dim, stm);
}
