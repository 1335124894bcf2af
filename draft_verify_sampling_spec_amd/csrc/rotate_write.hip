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
// turns, its fraction is exact to 2^-29, and only then sine and cosine are taken
// in fp32. Queries are rounded to bf16, what the attention reads. Keys are
// rounded to bf16 too before they are quantised, so that the cache holds the
// same bytes as if the rotated keys had been stored and written.
//
// A workgroup takes some consecutive tokens of one kv head: its group of query
// heads, its keys and its values. The angles' sines and cosines lie in LDS, one
// set for all of the workgroup's heads. D / 8 lanes share a head's row, 8
// channels each.
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
    int per;            // tokens of a workgroup
    bool interleaved, norm_bf16;
};

constexpr int kMostTokens = 32;

template <int D>
__device__ __forceinline__ void weights8(const void* w, bool bf16, int c, float (&y)[8]) {
    if (bf16) load8(static_cast<const uint16_t*>(w) + 8 * c, y);
    else load8(static_cast<const float*>(w) + 8 * c, y);
}

template <int D, typename S>
__global__ __launch_bounds__(256) void rotate_write_kernel(RotateArgs a) {
    constexpr int kLanes = D / 8;
    __shared__ float2 turn[kMostTokens * (D / 2)];
    const int h = blockIdx.y, half = a.rot / 2;
    const long long n0 = (long long)blockIdx.x * a.per;
    const int count = (int)min((long long)a.per, a.tokens - n0);
    for (int i = threadIdx.x; i < count * half; i += 256) {
        const int t = i / half, j = i - t * half;
        // 1 / (2 pi): the angle in turns, of which only the fraction counts.
        double x = (double)a.positions[n0 + t] * ((double)a.inv_freq[j] * 0.15915494309189533577);
        x -= rint(x);
        float sn, cs;
        sincospif(2.0f * (float)x, &sn, &cs);
        turn[t * (D / 2) + j] = make_float2(cs * a.factor, sn * a.factor);
    }
    __syncthreads();
    const int rows = a.group + 2, c = threadIdx.x % kLanes;
    const long long capacity = (long long)a.num_pages << a.shift;
    // Whole rows at a time: the lanes of a row agree on every branch.
    for (int i = threadIdx.x / kLanes; i < count * rows; i += 256 / kLanes) {
        const int t = i / rows, r = i - t * rows;
        const long long n = n0 + t;
        const int slot = a.slots[n];
        if (slot < 0) continue;
        if (slot >= capacity) {
            if (c == 0) flag(a.status, SV_FLAG_BAD_PAGE);
            continue;
        }
        const bool query = r < a.group, value = r == a.group + 1;
        const S* src = query   ? static_cast<const S*>(a.q) + n * a.q_stride + (long long)(h * a.group + r) * D
                       : value ? static_cast<const S*>(a.v) + n * a.v_stride + (long long)h * D
                               : static_cast<const S*>(a.k) + n * a.k_stride + (long long)h * D;
        float x[8];
        load8(src + 8 * c, x);
        if (!value) {
            const void* norm = query ? a.q_norm : a.k_norm;
            if (norm) {
                float sum = 0.0f;
                #pragma unroll
                for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
                #pragma unroll
                for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor(sum, o);
                const float f = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
                float w[8];
                weights8<D>(norm, a.norm_bf16, c, w);
                #pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] * f * w[j];
            }
            if (a.interleaved) {
                if (8 * c < a.rot) {
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 cs = turn[t * (D / 2) + 4 * c + j];
                        const float p = x[2 * j], q = x[2 * j + 1];
                        x[2 * j] = __builtin_fmaf(p, cs.x, -(q * cs.y));
                        x[2 * j + 1] = __builtin_fmaf(q, cs.x, p * cs.y);
                    }
                }
            } else {
                // The other channel of a pair lies rot / 16 lanes away.
                const int away = a.rot / 16, first = 8 * c < half ? c : c - away;
                const bool turns = 8 * c < a.rot;
                const int lane = threadIdx.x & 63;
                const int from = turns ? (8 * c < half ? lane + away : lane - away) : lane;
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float other = __shfl(x[j], from);
                    if (turns) {
                        const float2 cs = turn[t * (D / 2) + 8 * first + j];
                        x[j] = __builtin_fmaf(x[j], cs.x, 8 * c < half ? -(other * cs.y) : other * cs.y);
                    }
                }
            }
            unsigned w[4];
            #pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack2(x[2 * j], x[2 * j + 1]);
            uint16_t* out = query ? a.out + (n * a.Hq + h * a.group + r) * (long long)D
                                  : a.out_keys ? a.out_keys + (n * a.heads + h) * (long long)D : nullptr;
            if (out) *reinterpret_cast<uint4*>(out + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
            if (query) continue;
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[2 * j] = __uint_as_float(w[j] << 16);
                x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
        const int in = slot & ((1 << a.shift) - 1), tok = in & (kTile - 1);
        uint8_t* tile = a.cache + ((((long long)(slot >> a.shift) * a.heads + h) << (a.shift - 5)) + (in >> 5)) * Tile<D>::kBytes;
        unsigned byte;
        const unsigned w = quantise8(x, byte);
        put_codes<D>(tile, value, tok, c, w);
        if ((c & 3) == 0) {
            tile[value ? Tile<D>::v_scale(tok, c >> 2) : Tile<D>::k_scale(tok, c >> 2)] = (uint8_t)byte;
        }
    }
}

template <int D, typename S>
void launch(RotateArgs a, hipStream_t s) {
    const unsigned chunks = (unsigned)((a.tokens + a.per - 1) / a.per);
    hipLaunchKernelGGL((rotate_write_kernel<D, S>), dim3(chunks, (unsigned)a.heads), dim3(256), 0, s, a);
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
    a.per = 8;
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
