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
#include <cmath>

#include "cache_tile.h"

namespace {

using namespace svcache;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) unsigned u32x4;

constexpr int kWaves = 4;
constexpr float kNegInf = -INFINITY;

struct AttendArgs {
    const uint16_t* q;
    long long q_stride;
    const uint8_t* cache;
    const int32_t* ctx_lens;
    const int32_t* budgets;
    uint16_t* out;
    int32_t* status;
    float* part_o;      // [unit][split][16 kMT rows][D], not normalised
    float2* part_ml;    // [unit][split][16 kMT rows]: maximum, sum
    Pages pages;
    int K, Hq, group;
    int row_blocks;     // blocks of 16 kMT rows of a request's (K + 1) group rows
    int chunk;          // tiles of one split
    int splits;         // splits launched per unit
    int window;
    float c;            // scale * log2(e)
};

// The tiles a request's block reads: [first, end).
struct Span {
    int first, end;
};
__device__ __forceinline__ Span span_of(const Block& blk, int window) {
    const int lo = window > 0 ? max(0, blk.ctx - window + 1) : 0;
    return Span{lo / kTile, (blk.ctx + blk.len + kTile - 1) / kTile};
}

__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
    bf16x2 v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(unsigned, v);
}

// Maximum / sum over the four lanes that hold the same row.
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

template <int D, int kMT>
struct Lds {
    static constexpr int kPieces = kMT * Tile<D>::kPlanes * (D == 64 ? 4 : 8) / 4;  // float4 per lane and round
    f32x4 o[kWaves][kPieces][64];
    float m[kWaves][kMT][16];
    float l[kWaves][kMT][16];
};

template <int D, int kMT>
__global__ __launch_bounds__(256) void attend_kernel(AttendArgs a) {
    using L = Tile<D>;
    constexpr int kPlanes = L::kPlanes;
    constexpr int kKeySteps = D / 32;                  // products of 32 channels
    constexpr int kUnitSteps = D == 64 ? 2 : 4;        // of which in one key unit
    constexpr int kChans = D == 64 ? 4 : 8;            // channels of a value piece
    __shared__ Lds<D, kMT> sh;
    const int lane = threadIdx.x & 63, x = lane & 15, quad = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int id = blockIdx.x;
    const int split = id % a.splits;
    id /= a.splits;
    const int unit = id;
    const int rb = id % a.row_blocks;
    id /= a.row_blocks;
    const int h = id % a.pages.heads, b = id / a.pages.heads;

    const Block blk = block_of(a.ctx_lens, a.budgets, b, a.K + 1, a.pages, a.status,
                               split == 0 && rb == 0 && h == 0 && threadIdx.x == 0);
    const int rows = blk.len * a.group;
    if (rb * 16 * kMT >= rows) return;
    const Span span = span_of(blk, a.window);
    const int t0 = span.first + split * a.chunk, t1 = min(t0 + a.chunk, span.end);
    if (t0 >= t1) return;

    // This lane's rows and their queries.
    int pos[kMT];                 // the row's position; rows past the block see nothing
    bf16x8 q[kMT][kKeySteps];
    #pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
        const int r = (rb * kMT + mt) * 16 + x;
        const int t = r / a.group;
        const bool live = r < rows;
        pos[mt] = live ? blk.ctx + t : -1;
        const uint16_t* src = a.q + ((long long)b * (a.K + 1) + t) * a.q_stride +
                              (h * a.group + (r - t * a.group)) * D;
        #pragma unroll
        for (int s = 0; s < kKeySteps; ++s) {
            // Unit of plane s / kUnitSteps and this quad, 8 channels of step s.
            const int ch = (s / kUnitSteps * 4 + quad) * (8 * kUnitSteps) + 8 * (s % kUnitSteps);
            u32x4 w = {0, 0, 0, 0};
            if (live) w = *reinterpret_cast<const u32x4*>(src + ch);
            q[mt][s] = __builtin_bit_cast(bf16x8, w);
        }
    }

    f32x4 o[kMT][kPlanes][kChans];
    float m[kMT], l[kMT];
    #pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
        m[mt] = kNegInf;
        l[mt] = 0.0f;
        #pragma unroll
        for (int p = 0; p < kPlanes; ++p) {
            #pragma unroll
            for (int j = 0; j < kChans; ++j) o[mt][p][j] = f32x4{0, 0, 0, 0};
        }
    }

    // Tokens that every row of the block sees: [all_lo, all_hi).
    const int last = blk.ctx + blk.len - 1;
    const int all_hi = blk.ctx + 1;
    const int all_lo = a.window > 0 ? max(0, last - a.window + 1) : 0;

    for (int tile_at = t0 + wave; tile_at < t1; tile_at += kWaves) {
        const int tok0 = tile_at * kTile;
        const long long at = a.pages.tile(b, h, tok0, L::kBytes);
        if (at < 0) {
            if (lane == 0) flag(a.status, SV_FLAG_BAD_PAGE);
            continue;
        }
        const uint8_t* tile = a.cache + at;
        const bool masked = tok0 < all_lo || tok0 + kTile > all_hi;

        // Scores of 2 x 16 tokens (lane: tokens 16 half + 4 quad + r).
        f32x4 z[kMT][2];
        #pragma unroll
        for (int half = 0; half < 2; ++half) {
            #pragma unroll
            for (int mt = 0; mt < kMT; ++mt) z[mt][half] = f32x4{0, 0, 0, 0};
            #pragma unroll
            for (int p = 0; p < kPlanes; ++p) {
                const int g = D == 64 ? quad >> 1 : p * 4 + quad;
                const float s = scale_of(tile[L::kKScales + g * 32 + x * 2 + half]);
                unsigned w[kUnitSteps];
                __builtin_memcpy(w, tile + half * (8 * D) + ((p * 4 + quad) * 16 + x) * L::U, L::U);
                #pragma unroll
                for (int j = 0; j < kUnitSteps; ++j) {
                    const u32x4 kw = {decode2<0>(w[j], s), decode2<1>(w[j], s),
                                      decode2<2>(w[j], s), decode2<3>(w[j], s)};
                    const bf16x8 kf = __builtin_bit_cast(bf16x8, kw);
                    #pragma unroll
                    for (int mt = 0; mt < kMT; ++mt) {
                        z[mt][half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            kf, q[mt][p * kUnitSteps + j], z[mt][half], 0, 0, 0);
                    }
                }
            }
        }

        // Probabilities and running statistics.
        bf16x8 pf[kMT];
        #pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
            float s[8];
            #pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = z[mt][i >> 2][i & 3] * a.c;
            if (masked) {
                const int lo = a.window > 0 ? pos[mt] - a.window : -1;
                #pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = tok0 + 16 * (i >> 2) + 4 * quad + (i & 3);
                    if (j > pos[mt] || j <= lo) s[i] = kNegInf;
                }
            }
            float top = s[0];
            #pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i]);
            top = fmaxf(quad_max(top), m[mt]);
            // A row that has seen nothing yet keeps -inf; its terms are 0.
            const float ref = top == kNegInf ? 0.0f : top;
            const float keep = exp2f(m[mt] - ref);
            m[mt] = top;
            float sum = 0.0f;
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[i] = exp2f(s[i] - ref);
                sum += s[i];
            }
            l[mt] = l[mt] * keep + sum;
            #pragma unroll
            for (int p = 0; p < kPlanes; ++p) {
                #pragma unroll
                for (int j = 0; j < kChans; ++j) o[mt][p][j] *= keep;
            }
            const u32x4 pw = {pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]),
                              pack_bf16(s[6], s[7])};
            pf[mt] = __builtin_bit_cast(bf16x8, pw);
        }

        // Values: 8 tokens (4 quad + r of both halves) x kChans channels.
        #pragma unroll
        for (int p = 0; p < kPlanes; ++p) {
            const int g = D == 64 ? x >> 3 : p * 4 + (x >> 2);
            unsigned sc[2];
            __builtin_memcpy(sc, tile + L::kVScales + (g * 4 + quad) * 8, 8);
            unsigned w[8];
            #pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint8_t* src =
                    tile + L::kVCodes + (((p * 2 + half) * 4 + quad) * 16 + x) * (4 * L::C);
                if constexpr (D == 64) {
                    unsigned u[2];
                    __builtin_memcpy(u, src, 8);
                    w[4 * half] = u[0] & 0xffffu;
                    w[4 * half + 1] = u[0] >> 16;
                    w[4 * half + 2] = u[1] & 0xffffu;
                    w[4 * half + 3] = u[1] >> 16;
                } else {
                    __builtin_memcpy(&w[4 * half], src, 16);
                }
            }
            float vs[8];
            bool poison = false;
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
                unsigned byte = (sc[i >> 2] >> (8 * (i & 3))) & 255u;
                if (masked) {
                    // What some row does not see must not reach it as 0 * NaN:
                    // tokens past the block hold anything and are cleared;
                    // NaN groups of tokens that other rows see are cleared
                    // here and put into those rows below.
                    const int j = tok0 + 16 * (i >> 2) + 4 * quad + (i & 3);
                    const bool nan = byte == 255u;
                    poison |= nan && j <= last;
                    if (nan || j > last) {
                        byte = 127u;
                        w[i] = 0;
                    }
                }
                vs[i] = scale_of(byte);
            }
            #pragma unroll
            for (int cb = 0; cb < kChans / 2; ++cb) {
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
                for (int mt = 0; mt < kMT; ++mt) {
                    o[mt][p][2 * cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, even), pf[mt], o[mt][p][2 * cb], 0, 0, 0);
                    o[mt][p][2 * cb + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, odd), pf[mt], o[mt][p][2 * cb + 1], 0, 0, 0);
                }
            }
            if (masked && __ballot(poison) != 0) {
                // The accumulators of this lane hold channels of one group of
                // each plane (pieces 4 quad + r): NaN for the rows that see a
                // NaN token of that group.
                const int og = D == 64 ? quad >> 1 : p * 4 + quad;
                for (int tok = 0; tok < kTile; ++tok) {
                    const int j = tok0 + tok;
                    if (j > last || tile[L::v_scale(tok, og)] != 255u) continue;
                    #pragma unroll
                    for (int mt = 0; mt < kMT; ++mt) {
                        if (j > pos[mt] || (a.window > 0 && j <= pos[mt] - a.window)) continue;
                        #pragma unroll
                        for (int c = 0; c < kChans; ++c) o[mt][p][c] *= NAN;
                    }
                }
            }
        }
    }

    // Join the waves: component r of every accumulator in round r, so that
    // wave r ends with kChans consecutive channels per (row, plane).
    #pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
        const float sum = quad_sum(l[mt]);
        if (quad == 0) {
            sh.m[wave][mt][x] = m[mt];
            sh.l[wave][mt][x] = sum;
        }
    }
    __syncthreads();
    float factor[kMT], total[kMT], top[kMT];
    #pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
        top[mt] = kNegInf;
        #pragma unroll
        for (int w = 0; w < kWaves; ++w) top[mt] = fmaxf(top[mt], sh.m[w][mt][x]);
        const float ref = top[mt] == kNegInf ? 0.0f : top[mt];
        factor[mt] = exp2f(m[mt] - ref);
        total[mt] = 0.0f;
        #pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            total[mt] += sh.l[w][mt][x] * exp2f(sh.m[w][mt][x] - ref);
        }
    }
    f32x4 mine[Lds<D, kMT>::kPieces];
    #pragma unroll
    for (int r = 0; r < 4; ++r) {
        #pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
            #pragma unroll
            for (int p = 0; p < kPlanes; ++p) {
                #pragma unroll
                for (int c = 0; c < kChans; c += 4) {
                    const f32x4 v = {o[mt][p][c][r] * factor[mt], o[mt][p][c + 1][r] * factor[mt],
                                     o[mt][p][c + 2][r] * factor[mt],
                                     o[mt][p][c + 3][r] * factor[mt]};
                    sh.o[wave][((mt * kPlanes + p) * kChans + c) / 4][lane] = v;
                }
            }
        }
        __syncthreads();
        if (wave == r) {
            #pragma unroll
            for (int i = 0; i < Lds<D, kMT>::kPieces; ++i) {
                mine[i] = sh.o[0][i][lane] + sh.o[1][i][lane] + sh.o[2][i][lane] + sh.o[3][i][lane];
            }
        }
        __syncthreads();
    }

    const bool whole = a.splits == 1;
    #pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
        const int r = (rb * kMT + mt) * 16 + x;
        if (r >= rows) continue;
        const int t = r / a.group;
        const long long part = ((long long)unit * a.splits + split) * (16 * kMT) + mt * 16 + x;
        if (!whole && wave == 0 && quad == 0) a.part_ml[part] = make_float2(top[mt], total[mt]);
        const float inv = 1.0f / total[mt];
        #pragma unroll
        for (int p = 0; p < kPlanes; ++p) {
            const int ch = p * 128 + (4 * quad + wave) * kChans;
            const f32x4* v = &mine[(mt * kPlanes + p) * kChans / 4];
            if (whole) {
                uint16_t* dst = a.out + (((long long)b * (a.K + 1) + t) * a.Hq + h * a.group +
                                         (r - t * a.group)) * D + ch;
                unsigned w[kChans / 2];
                #pragma unroll
                for (int c = 0; c < kChans; c += 2) {
                    w[c / 2] = pack_bf16(v[c / 4][c % 4] * inv, v[c / 4][c % 4 + 1] * inv);
                }
                __builtin_memcpy(dst, w, 2 * kChans);
            } else {
                #pragma unroll
                for (int c = 0; c < kChans; c += 4) {
                    *reinterpret_cast<f32x4*>(a.part_o + part * D + ch + c) = v[c / 4];
                }
            }
        }
    }
}

// Joins the splits of one row: one wavefront per row, in the order of the
// splits.
template <int D, int kMT>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int B) {
    const int lane = threadIdx.x & 63;
    const int T = a.K + 1;
    const long long i = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (i >= (long long)B * T * a.Hq) return;
    const int head = (int)(i % a.Hq);
    const int t = (int)(i / a.Hq % T), b = (int)(i / a.Hq / T);
    const Block blk = block_of(a.ctx_lens, a.budgets, b, T, a.pages, nullptr, false);
    if (t >= blk.len) return;
    const Span span = span_of(blk, a.window);
    const int n = (span.end - span.first + a.chunk - 1) / a.chunk;
    const int h = head / a.group, r = t * a.group + head % a.group;
    const int rb = r / (16 * kMT), in = r % (16 * kMT);
    const long long unit = ((long long)b * a.pages.heads + h) * a.row_blocks + rb;
    const long long part = unit * a.splits * (16 * kMT) + in;
    float top = kNegInf;
    for (int s = 0; s < n; ++s) top = fmaxf(top, a.part_ml[part + (long long)s * 16 * kMT].x);
    const float ref = top == kNegInf ? 0.0f : top;
    float sum = 0.0f;
    float acc[D / 64] = {};
    for (int s = 0; s < n; ++s) {
        const long long p = part + (long long)s * 16 * kMT;
        const float2 ml = a.part_ml[p];
        const float f = exp2f(ml.x - ref);
        sum += ml.y * f;
        #pragma unroll
        for (int c = 0; c < D / 64; ++c) acc[c] += a.part_o[p * D + lane * (D / 64) + c] * f;
    }
    const float inv = 1.0f / sum;
    uint16_t* dst = a.out + i * D + lane * (D / 64);
    #pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        dst[c] = __builtin_bit_cast(uint16_t, (__bf16)(acc[c] * inv));
    }
}

// How a call is cut: rows per wavefront, row blocks, splits.
struct Plan {
    int mt, row_blocks, chunk, splits;
    long long units;
};

Plan plan_of(int B, int K, int Hq, int kv_heads, int D, int page_size, int max_pages, int window) {
    Plan p;
    const int rows = (K + 1) * (Hq / kv_heads);
    const int most = D == 256 ? 2 : 4;       // accumulators: kMT D / 4 registers a lane
    p.mt = (rows + 15) / 16 < most ? (rows + 15) / 16 : most;
    p.row_blocks = (rows + 16 * p.mt - 1) / (16 * p.mt);
    p.units = (long long)B * kv_heads * p.row_blocks;
    long long tokens = (long long)max_pages * page_size;
    if (window > 0 && tokens > (long long)window + K + kTile) tokens = (long long)window + K + kTile;
    const int tiles = (int)((tokens + kTile - 1) / kTile) + 1;
    // Enough workgroups for the 256 CUs, no split shorter than 16 tiles.
    long long splits = (1024 + p.units - 1) / p.units;
    const long long longest = (tiles + 15) / 16;
    if (splits > longest) splits = longest;
    p.chunk = (int)((tiles + splits - 1) / splits);
    p.splits = (tiles + p.chunk - 1) / p.chunk;
    return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t parts_of(const Plan& p) { return (size_t)p.units * p.splits * 16 * p.mt; }

bool shape_ok(int B, int K, int Hq, int kv_heads, int D, int page_size, int max_pages, int window) {
    return B >= 0 && B <= SV_MAX_BATCH && K >= 0 && K <= SV_MAX_K && window >= 0 &&
           geometry_ok(kv_heads, D, page_size, max_pages, 1) && Hq >= kv_heads &&
           Hq <= SV_MAX_HEADS && Hq % kv_heads == 0;
}

template <int D, int kMT>
void launch(const AttendArgs& a, const Plan& p, int B, hipStream_t s) {
    hipLaunchKernelGGL((attend_kernel<D, kMT>), dim3((unsigned)(p.units * p.splits)), dim3(256), 0,
                       s, a);
    if (p.splits > 1) {
        const long long rows = (long long)B * (a.K + 1) * a.Hq;
        hipLaunchKernelGGL((attend_join_kernel<D, kMT>), dim3((unsigned)((rows + 3) / 4)),
                           dim3(256), 0, s, a, B);
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
    if (p.splits == 1) return 256;
    return round256(parts_of(p) * head_dim * sizeof(float)) + round256(parts_of(p) * sizeof(float2));
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
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(
        static_cast<char*>(workspace) +
        (p.splits == 1 ? 0 : round256(parts_of(p) * head_dim * sizeof(float))));
    a.pages = make_pages(page_table, kv_heads, page_size, max_pages, num_pages);
    a.K = K;
    a.Hq = q_heads;
    a.group = q_heads / kv_heads;
    a.row_blocks = p.row_blocks;
    a.chunk = p.chunk;
    a.splits = p.splits;
    a.window = window;
    a.c = (float)((double)scale * 1.4426950408889634);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (head_dim * 8 + p.mt) {
        case 64 * 8 + 1: launch<64, 1>(a, p, B, s); break;
        case 64 * 8 + 2: launch<64, 2>(a, p, B, s); break;
        case 64 * 8 + 3: launch<64, 3>(a, p, B, s); break;
        case 64 * 8 + 4: launch<64, 4>(a, p, B, s); break;
        case 128 * 8 + 1: launch<128, 1>(a, p, B, s); break;
        case 128 * 8 + 2: launch<128, 2>(a, p, B, s); break;
        case 128 * 8 + 3: launch<128, 3>(a, p, B, s); break;
        case 128 * 8 + 4: launch<128, 4>(a, p, B, s); break;
        case 256 * 8 + 1: launch<256, 1>(a, p, B, s); break;
        default: launch<256, 2>(a, p, B, s); break;
    }
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
