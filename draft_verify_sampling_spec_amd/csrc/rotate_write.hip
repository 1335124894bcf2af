// rotate_write.hip -- queries and keys normalised per head and rotated to their
// positions, keys and values quantised into the paged 4-bit cache, in one pass
// over a step's projections, for MI355X (gfx950).
//
// The mathematics, per token and head of D channels: y = x w / sqrt(mean(x^2) +
// eps) (or y = x), then each of the rot / 2 pairs (y_i, y_j) is turned by the
// angle a_i = position * inv_freq_i,
//   (y_i cos a - y_j sin a, y_j cos a + y_i sin a) * factor.
// Sums and products are fp32. A position times a frequency loses its fraction
// in fp32 (at 10^6 a step is 2^-4 radians), so the angle is formed in fp64, in
// turns, and its sine and cosine too, once a token, before they are rounded to
// fp32. Queries are rounded to bf16, what the attention reads. Keys are
// rounded to bf16 too before they are quantised, so that the cache holds the
// same bytes as if the rotated keys had been stored and written.
//
// A wavefront takes a token, its weights and its angles' sines and cosines in registers:
// D / 8 lanes share a head's row, 8 channels each, 64 lanes a step of 512 / D rows,
// with kBatch steps' rows asked for together. Sums over a row and its halves'
// exchange go through lane permutations of the VALU, not through LDS.
//
// What bounds it: reads and writes, 4.3 TB/s for prompts (16 of 1,025..2,049 tokens, 32
// query and 8 kv heads of 128, bf16: 122 us; a copy moves 5.1), then the VALU (a
// workgroup per token chunk and head, whose rows changed kind and token from step to
// step, took 212). A step's 48 tokens take 5.4 us.
#include <cmath>

#include "cache_rows.h"

namespace {

using namespace svcache;

struct RotateArgs {
    const void* q;
    const void* k;
    const void* v;
    long long q_stride, k_stride, v_stride;
    const int32_t* slots;
    const int32_t* positions;
    const float* inv_freq;
    const void* q_norm;
    const void* k_norm;
    uint16_t* out;
    uint16_t* out_keys;
    uint8_t* cache;
    int32_t* status;
    long long tokens;
    float eps, factor;
    int Hq, group, heads, shift, num_pages;
    int rot;
    int span;           // kv heads of a workgroup
    bool interleaved, norm_bf16;
};

constexpr int kLeastWaves = 2048;
constexpr int kBatch = 4;           // steps of a wavefront in flight
constexpr unsigned kAcross = 1 << 16;   // workgroups of a grid's x; a dimension holds less than 2^32 threads

// Eight channels as they are stored.
template <typename S>
struct Eight {
    uint4 raw[sizeof(S) / 2];
    __device__ __forceinline__ void load(const S* p) {
        #pragma unroll
        for (int i = 0; i < (int)sizeof(S) / 2; ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const { load8(reinterpret_cast<const S*>(raw), x); }
};

template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, true));
}

// Sum over the kLanes lanes of a row, in all of them.
template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
    v += dpp<0xb1>(v);                          // lane ^ 1
    v += dpp<0x4e>(v);                          // lane ^ 2
    v += dpp<0x141>(v);                         // the other four of eight
    if (kLanes >= 16) v += dpp<0x140>(v);       // the other eight of sixteen
    if (kLanes == 32) {
        auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    return v;
}

// The value half a row of kLanes lanes away.
template <int kLanes>
__device__ __forceinline__ float half_row(float v, int lane) {
    if constexpr (kLanes == 8) return dpp<0x1b>(dpp<0x141>(v));     // 7 - lane, then reversed in fours
    if constexpr (kLanes == 16) return dpp<0x128>(v);
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(lane & 16 ? a[0] : a[1]);
}

template <int D, typename S>
__global__ __launch_bounds__(256, 4) void rotate_write_kernel(RotateArgs a) {
    constexpr int kLanes = D / 8, kSide = 64 / kLanes;      // lanes of a row, rows of a step
    __shared__ float2 turns[4][D / 2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int c = lane % kLanes, side = lane / kLanes;
    const int h0 = blockIdx.y * a.span, heads = min(a.span, a.heads - h0), queries = heads * a.group;
    const int half = a.rot / 2, qs = (queries + kSide - 1) / kSide, ks = (heads + kSide - 1) / kSide;
    float wq[8], wk[8];
    if (a.q_norm) {
        if (a.norm_bf16) load8(static_cast<const uint16_t*>(a.q_norm) + 8 * c, wq);
        else load8(static_cast<const float*>(a.q_norm) + 8 * c, wq);
    }
    if (a.k_norm) {
        if (a.norm_bf16) load8(static_cast<const uint16_t*>(a.k_norm) + 8 * c, wk);
        else load8(static_cast<const float*>(a.k_norm) + 8 * c, wk);
    }
    const long long n = ((long long)blockIdx.z * gridDim.x + blockIdx.x) * 4 + wave;
    if (n >= a.tokens) return;
    const int slot = __builtin_amdgcn_readfirstlane(a.slots[n]);
    if (slot < 0) return;
    if (slot >= (long long)a.num_pages << a.shift) {
        if (lane == 0) flag(a.status, SV_FLAG_BAD_PAGE);
        return;
    }
    // Steps of kSide rows: queries, then keys, then values.
    const S* const q = static_cast<const S*>(a.q) + n * a.q_stride + (long long)h0 * a.group * D;
    const S* const kk = static_cast<const S*>(a.k) + n * a.k_stride + (long long)h0 * D;
    const S* const v = static_cast<const S*>(a.v) + n * a.v_stride + (long long)h0 * D;
    Eight<S> in[kBatch];
    auto ask = [&](int s0) {
        #pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int s = s0 + i;
            const S* const src = s < qs ? q : s < qs + ks ? kk : v;
            const int r = (s < qs ? s : s < qs + ks ? s - qs : s - qs - ks) * kSide + side;
            if (s < qs + 2 * ks && r < (s < qs ? queries : heads)) in[i].load(src + r * D + 8 * c);
        }
    };
    ask(0);
    // The angles, while the first rows are on their way.
    for (int i = lane; i < half; i += 64) {
        // 1 / (2 pi): the angle in turns, of which only the fraction counts.
        double x = (double)a.positions[n] * ((double)a.inv_freq[i] * 0.15915494309189533577);
        x -= rint(x);
        double sn, cs;
        sincospi(2.0 * x, &sn, &cs);
        turns[wave][i] = make_float2((float)cs * a.factor, (float)sn * a.factor);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // read by other lanes of the wavefront only
    // Channel j becomes x_j cs_j + (its pair's other) sn_j.
    float cs[8], sn[8];
    #pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int ch = 8 * c + j;
        const bool second = a.interleaved ? (j & 1) != 0 : ch >= half;
        float2 turn = make_float2(1.0f, 0.0f);
        if (8 * c < a.rot) turn = turns[wave][a.interleaved ? ch / 2 : second ? ch - half : ch];
        cs[j] = turn.x;
        sn[j] = second ? turn.y : -turn.y;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int in_page = slot & ((1 << a.shift) - 1), tok = in_page & (kTile - 1);
    uint8_t* const tile = a.cache + ((((long long)(slot >> a.shift) * a.heads + h0) << (a.shift - 5)) + (in_page >> 5)) * Tile<D>::kBytes;
    const int head_bytes = Tile<D>::kBytes << (a.shift - 5);
    for (int s0 = 0; s0 < qs + 2 * ks; s0 += kBatch) {
        if (s0 > 0) ask(s0);
        #pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int s = s0 + i;
            if (s >= qs + 2 * ks) break;
            const bool query = s < qs, value = s >= qs + ks;
            const int r = (query ? s : value ? s - qs - ks : s - qs) * kSide + side;
            if (r >= (query ? queries : heads)) continue;       // whole rows
            float x[8];
            in[i].get(x);
            if (!value) {
                if (query ? a.q_norm != nullptr : a.k_norm != nullptr) {
                    float sum = 0.0f;
                    #pragma unroll
                    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
                    const float f = __builtin_amdgcn_rsqf(row_sum<kLanes>(sum) * (1.0f / D) + a.eps);
                    #pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = x[j] * f * (query ? wq[j] : wk[j]);
                }
                if (a.rot > 0) {
                    float other[8];
                    if (a.interleaved) {
                        #pragma unroll
                        for (int j = 0; j < 8; ++j) other[j] = x[j ^ 1];
                    } else if (a.rot == D) {
                        #pragma unroll
                        for (int j = 0; j < 8; ++j) other[j] = half_row<kLanes>(x[j], lane);
                    } else {
                        // rot / 16 lanes away; lanes that do not turn take their own.
                        const int away = a.rot / 16;
                        const int from = 8 * c < half ? lane + away : 8 * c < a.rot ? lane - away : lane;
                        #pragma unroll
                        for (int j = 0; j < 8; ++j) other[j] = __shfl(x[j], from);
                    }
                    if (8 * c < a.rot) {        // a product with 0 would spread an infinity
                        #pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = x[j] * cs[j] + other[j] * sn[j];
                    }
                }
                unsigned w[4];
                #pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = pack2(x[2 * j], x[2 * j + 1]);
                uint16_t* out = query ? a.out + (n * a.Hq + h0 * a.group) * (long long)D
                                      : a.out_keys ? a.out_keys + (n * a.heads + h0) * (long long)D : nullptr;
                if (out) *reinterpret_cast<uint4*>(out + r * D + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
                if (query) continue;
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[2 * j] = __uint_as_float(w[j] << 16);
                    x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                }
            }
            uint8_t* const mine = tile + (long long)r * head_bytes;
            unsigned byte;
            const unsigned w = quantise8(x, byte);
            put_codes<D>(mine, value, tok, c, w);
            if ((c & 3) == 0) {
                mine[value ? Tile<D>::v_scale(tok, c >> 2) : Tile<D>::k_scale(tok, c >> 2)] = (uint8_t)byte;
            }
        }
    }
}

template <int D, typename S>
void launch(const RotateArgs& a, hipStream_t s) {
    const unsigned chunks = (unsigned)((a.tokens + 3) / 4);
    const dim3 grid(chunks < kAcross ? chunks : kAcross, (unsigned)((a.heads + a.span - 1) / a.span),
                    (chunks + kAcross - 1) / kAcross);
    hipLaunchKernelGGL((rotate_write_kernel<D, S>), grid, dim3(256), 0, s, a);
}

}  // namespace

extern "C" int spec_verify_cache_write_rotated(
    const void* queries, const void* keys, const void* values, int dtype, int64_t query_stride,
    int64_t key_stride, int64_t value_stride, const int32_t* slots, const int32_t* positions,
    int64_t tokens, const float* inv_freq, int rot, int interleaved, float factor,
    const void* q_norm, const void* k_norm, int norm_dtype, float eps, int q_heads, int kv_heads,
    int head_dim, int page_size, int num_pages, void* cache, void* out_queries, void* out_keys,
    int32_t* out_status, void* stream) {
    if (tokens < 0 || tokens > SV_MAX_STRIDE || !geometry_ok(kv_heads, head_dim, page_size, 1, num_pages) ||
        (long long)num_pages * page_size > 0x7fffffffll || q_heads < kv_heads ||
        q_heads > SV_MAX_HEADS || q_heads % kv_heads != 0 || rot < 0 || rot > head_dim ||
        rot % 16 != 0 || !std::isfinite(factor) || !(eps >= 0.0f) || !std::isfinite(eps)) {
        return SV_ERR_ARG;
    }
    const bool norm = q_norm || k_norm;
    if ((dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16) ||
        (norm && norm_dtype != SV_DTYPE_F32 && norm_dtype != SV_DTYPE_BF16)) {
        return SV_ERR_DTYPE;
    }
    if (tokens == 0) return SV_OK;
    const int64_t lanes = dtype == SV_DTYPE_F32 ? 4 : 8;       // elements of 16 bytes
    const int64_t kv = (int64_t)kv_heads * head_dim;
    if (query_stride < (int64_t)q_heads * head_dim || key_stride < kv || value_stride < kv ||
        query_stride > SV_MAX_STRIDE || key_stride > SV_MAX_STRIDE || value_stride > SV_MAX_STRIDE) {
        return SV_ERR_ARG;
    }
    if (!queries || !keys || !values || !slots || !positions || !cache || !out_queries ||
        (rot > 0 && !inv_freq)) {
        return SV_ERR_NULL;
    }
    if (!aligned(queries, 16) || !aligned(keys, 16) || !aligned(values, 16) || !aligned(cache, 16) ||
        !aligned(out_queries, 16) || !aligned(out_keys, 16) || !aligned(q_norm, 16) ||
        !aligned(k_norm, 16) || query_stride % lanes != 0 || key_stride % lanes != 0 ||
        value_stride % lanes != 0 || !aligned(slots, 4) || !aligned(positions, 4) ||
        !aligned(inv_freq, 4) || !aligned(out_status, 4)) {
        return SV_ERR_ALIGN;
    }
    RotateArgs a{};
    a.q = queries;
    a.k = keys;
    a.v = values;
    a.q_stride = query_stride;
    a.k_stride = key_stride;
    a.v_stride = value_stride;
    a.slots = slots;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.out = static_cast<uint16_t*>(out_queries);
    a.out_keys = static_cast<uint16_t*>(out_keys);
    a.cache = static_cast<uint8_t*>(cache);
    a.status = out_status;
    a.tokens = tokens;
    a.eps = eps;
    a.factor = factor;
    a.Hq = q_heads;
    a.group = q_heads / kv_heads;
    a.heads = kv_heads;
    a.shift = __builtin_ctz((unsigned)page_size);
    a.num_pages = num_pages;
    a.rot = rot;
    // All heads of a token to one wavefront, which then forms its angles once, or
    // fewer where that gives the chip too few wavefronts (prompts of 32,784 tokens: 125
    // us with 8 heads, 143 with 4; a step's 48 tokens: 5.4 with 1 head, 7.2 with 4).
    a.span = kv_heads;
    while (a.span > 1 && tokens * ((kv_heads + a.span - 1) / a.span) < kLeastWaves) a.span = (a.span + 1) / 2;
    a.interleaved = interleaved != 0;
    a.norm_bf16 = norm_dtype == SV_DTYPE_BF16;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        if (dtype == SV_DTYPE_F32) launch<D, float>(a, s);
        else launch<D, uint16_t>(a, s);
    };
    if (head_dim == 64) go(std::integral_constant<int, 64>{});
    else if (head_dim == 128) go(std::integral_constant<int, 128>{});
    else go(std::integral_constant<int, 256>{});
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
