// block_cache.hip -- writing tokens into the paged 4-bit key/value cache and
// reading them back, for MI355X (gfx950).
//
// The mathematics: every token's keys and values of one head are cut into
// groups of 32 channels. A group with largest magnitude a gets the scale
// s = 2^e, e the smallest integer >= -64 with a <= 6 s, and channel x becomes
// the e2m1 code nearest to x / s (ties to even). s is a power of two, so
// x / s and code * s are exact and the code is a function of x alone; a read
// returns code * s, at most s from x (half of e2m1's widest step, 2, times s).
// A token never shares a scale with another one: a rejected drafted token is
// undone by the lengths alone, and the next token overwrites it.
//
// Both kernels move each byte once and are bound by HBM (long prompts) or by
// the launch (a verify block). Kernel times, heads of 128 channels, 8 of them: 16
// prompts of 1,025..2,049 fp32 tokens written in 60 us (4.0 TB/s) and read back
// in 44 (5.4); 8 contexts of 8,192..16,384 tokens read as bf16 in 99 (4.5); 8
// blocks of 6 tokens written in 3.4 and read in 3.1.
#include "cache_tile.h"

namespace {

using namespace svcache;

// Eight consecutive channels as fp32.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// The group scale byte and the four code bytes of this thread's 8 channels;
// the 4 lanes of a group are adjacent.
__device__ __forceinline__ unsigned quantise8(const float (&x)[8], unsigned& byte) {
    unsigned amax = 0;
    #pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
    amax = max(amax, (unsigned)__shfl_xor((int)amax, 1));
    amax = max(amax, (unsigned)__shfl_xor((int)amax, 2));
    byte = cache_scale_byte(amax);
    if (byte == 255u) return 0;
    const float s = scale_of(byte);
    unsigned w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
    return w;
}

template <int D>
__device__ __forceinline__ void put_codes(uint8_t* tile, bool value, int tok, int c, unsigned w) {
    using L = Tile<D>;
    if (!value) {
        *reinterpret_cast<unsigned*>(tile + L::k_codes(tok, c)) = w;
    } else if (D >= 128) {
        *reinterpret_cast<unsigned*>(tile + L::v_codes(tok, c)) = w;
    } else {
        *reinterpret_cast<uint16_t*>(tile + L::v_codes(tok, c)) = (uint16_t)w;
        *reinterpret_cast<uint16_t*>(tile + L::v_codes(tok, c) + 4 * L::C) = (uint16_t)(w >> 16);
    }
}

template <int D>
__device__ __forceinline__ unsigned get_codes(const uint8_t* tile, bool value, int tok, int c) {
    using L = Tile<D>;
    if (!value) return *reinterpret_cast<const unsigned*>(tile + L::k_codes(tok, c));
    if (D >= 128) return *reinterpret_cast<const unsigned*>(tile + L::v_codes(tok, c));
    return *reinterpret_cast<const uint16_t*>(tile + L::v_codes(tok, c)) |
           ((unsigned)*reinterpret_cast<const uint16_t*>(tile + L::v_codes(tok, c) + 4 * L::C)
            << 16);
}

// Which token and 8 channels task i of a workgroup is: a workgroup takes the
// tokens of one cache tile and head, 8 channels at a time, so that the tile's
// lines are its own: a wavefront's 4-byte pieces of them are runs of 64 bytes
// (keys) or 256 bytes (values), its 16-byte pieces of the tensors whole rows.
// (Tokens across all heads in a workgroup measured 169 against 110 us for a read
// of eight contexts of 8,192..16,384 tokens.)
template <int D>
struct Task {
    static constexpr int kPer = D / 8, kSide = kTile * kPer, kAll = 2 * kSide;
    int c, tok;
    bool value;
    __device__ __forceinline__ explicit Task(int i)
        : c(i % kPer), tok(i % kSide / kPer), value(i >= kSide) {}
};

// blockIdx.y: request; x: (tile of the block's tokens, head).
template <int D, typename S>
__global__ __launch_bounds__(256) void cache_write_kernel(
    const S* __restrict__ keys, const S* __restrict__ values, long long key_stride,
    long long value_stride, const int32_t* __restrict__ ctx_lens,
    const int32_t* __restrict__ budgets, int T, Pages pages, uint8_t* __restrict__ cache,
    int32_t* __restrict__ status) {
    const int b = blockIdx.y, h = blockIdx.x % pages.heads;
    const Block blk = block_of(ctx_lens, budgets, b, T, pages, status,
                               blockIdx.x == 0 && threadIdx.x == 0);
    if (blk.len == 0) return;
    const int pos0 = (blk.ctx / kTile + (int)(blockIdx.x / pages.heads)) * kTile;
    if (pos0 >= blk.ctx + blk.len) return;
    const long long at = pages.tile(b, h, pos0, Tile<D>::kBytes);
    if (at < 0) {
        if (threadIdx.x == 0) flag(status, SV_FLAG_BAD_PAGE);
        return;
    }
    uint8_t* tile = cache + at;
    #pragma unroll
    for (int i = threadIdx.x; i < Task<D>::kAll; i += 256) {
        const Task<D> task(i);
        const int t = pos0 + task.tok - blk.ctx;            // the 4 lanes of a group agree
        if (t < 0 || t >= blk.len) continue;
        const S* src = task.value ? values + ((long long)b * T + t) * value_stride
                                  : keys + ((long long)b * T + t) * key_stride;
        float x[8];
        load8(src + h * D + 8 * task.c, x);
        unsigned byte;
        const unsigned w = quantise8(x, byte);
        put_codes<D>(tile, task.value, task.tok, task.c, w);
        if ((task.c & 3) == 0) {
            tile[task.value ? Tile<D>::v_scale(task.tok, task.c >> 2)
                            : Tile<D>::k_scale(task.tok, task.c >> 2)] = (uint8_t)byte;
        }
    }
}

__device__ __forceinline__ void store8(float* p, const unsigned (&v)[4]) {
    float4 a, b;
    a.x = __uint_as_float(v[0] << 16); a.y = __uint_as_float(v[0] & 0xffff0000u);
    a.z = __uint_as_float(v[1] << 16); a.w = __uint_as_float(v[1] & 0xffff0000u);
    b.x = __uint_as_float(v[2] << 16); b.y = __uint_as_float(v[2] & 0xffff0000u);
    b.z = __uint_as_float(v[3] << 16); b.w = __uint_as_float(v[3] & 0xffff0000u);
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
}
__device__ __forceinline__ void store8(uint16_t* p, const unsigned (&v)[4]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
}

// Every value is exact in bf16.
template <int D, typename S>
__global__ __launch_bounds__(256) void cache_read_kernel(
    const uint8_t* __restrict__ cache, const int32_t* __restrict__ starts,
    const int32_t* __restrict__ lens, int T, Pages pages, S* __restrict__ out_keys,
    S* __restrict__ out_values, int32_t* __restrict__ status) {
    const int b = blockIdx.y, h = blockIdx.x % pages.heads;
    const int start = starts ? starts[b] : 0;
    const int n = lens[b];
    if (start < 0 || n <= 0) return;
    if (n > T || (long long)start + n > ((long long)pages.max_pages << pages.shift)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag(status, SV_FLAG_BAD_LENGTH);
        return;
    }
    const int pos0 = (start / kTile + (int)(blockIdx.x / pages.heads)) * kTile;
    if (pos0 >= start + n) return;
    const long long at = pages.tile(b, h, pos0, Tile<D>::kBytes);
    if (at < 0) {
        if (threadIdx.x == 0) flag(status, SV_FLAG_BAD_PAGE);
        return;
    }
    const uint8_t* tile = cache + at;
    #pragma unroll
    for (int i = threadIdx.x; i < Task<D>::kAll; i += 256) {
        const Task<D> task(i);
        const int t = pos0 + task.tok - start;
        if (t < 0 || t >= n) continue;
        const unsigned w = get_codes<D>(tile, task.value, task.tok, task.c);
        const float s = scale_of(tile[task.value ? Tile<D>::v_scale(task.tok, task.c >> 2)
                                                 : Tile<D>::k_scale(task.tok, task.c >> 2)]);
        const unsigned v[4] = {decode2<0>(w, s), decode2<1>(w, s), decode2<2>(w, s), decode2<3>(w, s)};
        S* out = task.value ? out_values : out_keys;
        store8(out + (((long long)b * T + t) * pages.heads + h) * D + 8 * task.c, v);
    }
}

// Tiles that T tokens from any position touch, times heads.
unsigned blocks_for(int T, int heads) { return (unsigned)((T + 2ll * kTile - 2) / kTile * heads); }

template <int D, typename S>
void launch_write(const void* keys, const void* values, int64_t ks, int64_t vs,
                  const int32_t* ctx, const int32_t* budgets, int B, int T, const Pages& pages,
                  void* cache, int32_t* status, hipStream_t s) {
    hipLaunchKernelGGL((cache_write_kernel<D, S>),
                       dim3(blocks_for(T, pages.heads), (unsigned)B), dim3(256), 0, s,
                       static_cast<const S*>(keys), static_cast<const S*>(values), ks, vs, ctx,
                       budgets, T, pages, static_cast<uint8_t*>(cache), status);
}

template <int D, typename S>
void launch_read(const void* cache, const int32_t* starts, const int32_t* lens, int B, int T,
                 const Pages& pages, void* ok, void* ov, int32_t* status, hipStream_t s) {
    hipLaunchKernelGGL((cache_read_kernel<D, S>),
                       dim3(blocks_for(T, pages.heads), (unsigned)B), dim3(256), 0, s,
                       static_cast<const uint8_t*>(cache), starts, lens, T, pages,
                       static_cast<S*>(ok), static_cast<S*>(ov), status);
}

}  // namespace

extern "C" size_t spec_verify_cache_bytes(int num_pages, int kv_heads, int head_dim,
                                          int page_size) {
    if (!geometry_ok(kv_heads, head_dim, page_size, 1, num_pages)) return 0;
    return (size_t)num_pages * kv_heads * (page_size / kTile) * (34 * head_dim);
}

extern "C" int spec_verify_cache_write(const void* keys, const void* values, int dtype,
                                       int64_t key_stride, int64_t value_stride,
                                       const int32_t* page_table, const int32_t* ctx_lens,
                                       const int32_t* budgets, int B, int T, int kv_heads,
                                       int head_dim, int page_size, int max_pages, int num_pages,
                                       void* cache, int32_t* out_status, void* stream) {
    const int64_t row = (int64_t)kv_heads * head_dim;
    if (B < 0 || B > SV_MAX_BATCH || T < 0 || T > SV_MAX_CONTEXT ||
        !geometry_ok(kv_heads, head_dim, page_size, max_pages, num_pages)) {
        return SV_ERR_ARG;
    }
    if (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16) return SV_ERR_DTYPE;
    if (B == 0 || T == 0) return SV_OK;
    const int lanes = dtype == SV_DTYPE_F32 ? 4 : 8;       // elements of 16 bytes
    if ((long long)T * row > (1ll << 33) || key_stride < row || value_stride < row || key_stride > SV_MAX_STRIDE ||
        value_stride > SV_MAX_STRIDE) {
        return SV_ERR_ARG;
    }
    if (!keys || !values || !page_table || !ctx_lens || !cache) return SV_ERR_NULL;
    if (!aligned(keys, 16) || !aligned(values, 16) || !aligned(cache, 16) ||
        key_stride % lanes != 0 || value_stride % lanes != 0 || !aligned(page_table, 4) ||
        !aligned(ctx_lens, 4) || !aligned(budgets, 4) || !aligned(out_status, 4)) {
        return SV_ERR_ALIGN;
    }
    const Pages pages = make_pages(page_table, kv_heads, page_size, max_pages, num_pages);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        if (dtype == SV_DTYPE_F32) {
            launch_write<D, float>(keys, values, key_stride, value_stride, ctx_lens, budgets, B, T,
                                   pages, cache, out_status, s);
        } else {
            launch_write<D, uint16_t>(keys, values, key_stride, value_stride, ctx_lens, budgets, B,
                                      T, pages, cache, out_status, s);
        }
    };
    if (head_dim == 64) go(std::integral_constant<int, 64>{});
    else if (head_dim == 128) go(std::integral_constant<int, 128>{});
    else go(std::integral_constant<int, 256>{});
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

extern "C" int spec_verify_cache_read(const void* cache, const int32_t* page_table,
                                      const int32_t* starts, const int32_t* lens, int B, int T,
                                      int kv_heads, int head_dim, int page_size, int max_pages,
                                      int num_pages, int dtype, void* out_keys, void* out_values,
                                      int32_t* out_status, void* stream) {
    if (B < 0 || B > SV_MAX_BATCH || T < 0 || T > SV_MAX_CONTEXT ||
        !geometry_ok(kv_heads, head_dim, page_size, max_pages, num_pages)) {
        return SV_ERR_ARG;
    }
    if (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16) return SV_ERR_DTYPE;
    if (B == 0 || T == 0) return SV_OK;
    if ((long long)T * kv_heads * head_dim > (1ll << 33)) return SV_ERR_ARG;
    if (!cache || !page_table || !lens || !out_keys || !out_values) return SV_ERR_NULL;
    if (!aligned(cache, 16) || !aligned(out_keys, 16) || !aligned(out_values, 16) ||
        !aligned(page_table, 4) || !aligned(starts, 4) || !aligned(lens, 4) ||
        !aligned(out_status, 4)) {
        return SV_ERR_ALIGN;
    }
    const Pages pages = make_pages(page_table, kv_heads, page_size, max_pages, num_pages);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        if (dtype == SV_DTYPE_F32) {
            launch_read<D, float>(cache, starts, lens, B, T, pages, out_keys, out_values,
                                  out_status, s);
        } else {
            launch_read<D, uint16_t>(cache, starts, lens, B, T, pages, out_keys, out_values,
                                     out_status, s);
        }
    };
    if (head_dim == 64) go(std::integral_constant<int, 64>{});
    else if (head_dim == 128) go(std::integral_constant<int, 128>{});
    else go(std::integral_constant<int, 256>{});
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
