// head_fp8.hip -- the output head in 8-bit floating point, for MI355X
// (gfx950): quantising hidden states and heads, and their product.
//
// The mathematics: a block (1 x 128 of a state, 128 x 128 of a head) with
// largest magnitude a gets the scale s = 2^e, e the smallest integer >= -64
// with a <= 448 s, and x becomes the e4m3 code nearest to x / s (ties to
// even); both x / s and code * s are exact. The logits are
//   z[r, v] = sum_blk s_h[r, blk] s_w[v / 128, blk] sum_i h[r, i] w[v, i].
// A scale that is a power of two costs the product nothing: decoding a code
// to bf16 times its scale is exact.
#include <cmath>

#include "cache_tile.h"

namespace {

using svcache::aligned;
using svcache::scale_byte;
using svcache::scale_of;
using svcache::bf16x2;

constexpr int kBlock = 128;

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) unsigned u32x4;

// e4m3: largest value 448 = 1.75 * 2^8.
__device__ __forceinline__ unsigned head_scale_byte(unsigned amax_bits) {
    return scale_byte<0x600000u, 8>(amax_bits);
}

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

__device__ __forceinline__ unsigned magnitude(const float (&x)[8]) {
    unsigned a = 0;
    #pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(x[i]) & 0x7fffffffu);
    return a;
}

// Eight e4m3 codes of x / 2^(byte - 127); NaN codes for a NaN scale.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], unsigned byte) {
    if (byte == 255u) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    const float inv = __uint_as_float((254u - byte) << 23);
    float y[8];
    #pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(x[i] * inv, -448.0f, 448.0f);
    int a = 0, b = 0;
    a = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], a, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], a, true);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], b, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], b, true);
    return make_uint2((unsigned)a, (unsigned)b);
}

// One scale per row and 128 channels: 16 lanes of 8 channels a block.
template <typename S>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const S* __restrict__ src, int rows,
                                                            int H, int blocks,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long blk = i >> 4;                 // row * blocks + block
    if (blk >= (long long)rows * blocks) return;
    const long long row = blk / blocks;
    const int ch = (int)(blk - row * blocks) * kBlock + (int)(i & 15) * 8;
    float x[8] = {};
    if (ch < H) load8(src + row * H + ch, x);
    unsigned amax = magnitude(x);
    #pragma unroll
    for (int o = 1; o < 16; o <<= 1) amax = max(amax, (unsigned)__shfl_xor((int)amax, o));
    const unsigned byte = head_scale_byte(amax);
    *reinterpret_cast<uint2*>(codes + row * blocks * kBlock + ch) = encode8(x, byte);
    if ((i & 15) == 0) scales[blk] = (uint8_t)byte;
}

// One scale per 128 x 128 block: a workgroup each, 8 values x 8 rows a thread.
template <typename S>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const S* __restrict__ src, int rows,
                                                              int H, int blocks,
                                                              uint8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
    __shared__ unsigned wave_max[4];
    const int rb = blockIdx.x / blocks, cb = blockIdx.x - rb * blocks;
    const int ch = cb * kBlock + (threadIdx.x & 15) * 8;
    const int row0 = rb * kBlock + (threadIdx.x >> 4);
    float x[8][8] = {};
    unsigned amax = 0;
    #pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int row = row0 + 16 * k;
        if (row < rows && ch < H) load8(src + (long long)row * H + ch, x[k]);
    }
    #pragma unroll
    for (int k = 0; k < 8; ++k) amax = max(amax, magnitude(x[k]));
    #pragma unroll
    for (int o = 1; o < 64; o <<= 1) amax = max(amax, (unsigned)__shfl_xor((int)amax, o));
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = max(max(wave_max[0], wave_max[1]), max(wave_max[2], wave_max[3]));
    const unsigned byte = head_scale_byte(amax);
    #pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int row = row0 + 16 * k;
        if (row < rows) {
            *reinterpret_cast<uint2*>(codes + (long long)row * blocks * kBlock + ch) =
                encode8(x[k], byte);
        }
    }
    if (threadIdx.x == 0) scales[blockIdx.x] = (uint8_t)byte;
}

// Eight codes (two dwords) times scale as bf16, exactly.
__device__ __forceinline__ bf16x8 decode8(unsigned a, unsigned b, float s) {
    const u32x4 w = {
        __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false)),
        __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true)),
        __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false)),
        __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true))};
    return __builtin_bit_cast(bf16x8, w);
}

struct LogitArgs {
    const uint8_t* h;
    const uint8_t* hs;
    const uint8_t* w;
    const uint8_t* ws;
    void* out;
    int R, V, blocks;
};

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) {
    *p = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// A wavefront: 16 vocabulary columns x 16 kMT rows, the head's codes straight
// from memory.
template <int kMT, typename O>
__global__ __launch_bounds__(256) void logits_stream_kernel(LogitArgs a) {
    const int lane = threadIdx.x & 63, x = lane & 15, quad = lane >> 4;
    const int v0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 16;
    if (v0 >= a.V) return;
    const int r0 = blockIdx.y * 16 * kMT;
    const long long pitch = (long long)a.blocks * kBlock;
    const int wrow = min(v0 + x, a.V - 1);
    const uint8_t* wp = a.w + wrow * pitch + quad * 16;
    const uint8_t* wsp = a.ws + (long long)(wrow / kBlock) * a.blocks;
    const uint8_t* hp[kMT];
    const uint8_t* hsp[kMT];
    #pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
        const int r = min(r0 + mt * 16 + x, a.R - 1);
        hp[mt] = a.h + r * pitch + quad * 16;
        hsp[mt] = a.hs + (long long)r * a.blocks;
    }
    f32x4 acc[kMT] = {};
    for (int k = 0; k < a.blocks; ++k) {
        const u32x4 w0 = *reinterpret_cast<const u32x4*>(wp + (long long)k * kBlock);
        const u32x4 w1 = *reinterpret_cast<const u32x4*>(wp + (long long)k * kBlock + 64);
        const float s = scale_of(wsp[k]);
        const bf16x8 wf[4] = {decode8(w0[0], w0[1], s), decode8(w0[2], w0[3], s),
                              decode8(w1[0], w1[1], s), decode8(w1[2], w1[3], s)};
        #pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
            const u32x4 h0 = *reinterpret_cast<const u32x4*>(hp[mt] + (long long)k * kBlock);
            const u32x4 h1 = *reinterpret_cast<const u32x4*>(hp[mt] + (long long)k * kBlock + 64);
            const float t = scale_of(hsp[mt][k]);
            acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[0], decode8(h0[0], h0[1], t), acc[mt], 0, 0, 0);
            acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[1], decode8(h0[2], h0[3], t), acc[mt], 0, 0, 0);
            acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[2], decode8(h1[0], h1[1], t), acc[mt], 0, 0, 0);
            acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[3], decode8(h1[2], h1[3], t), acc[mt], 0, 0, 0);
        }
    }
    O* out = static_cast<O*>(a.out);
    #pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
        const int r = r0 + mt * 16 + x;
        if (r >= a.R) continue;
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int v = v0 + 4 * quad + i;
            if (v < a.V) put(out + (long long)r * a.V + v, acc[mt][i]);
        }
    }
}

template <int kMT>
void launch_stream(const LogitArgs& a, int dtype, hipStream_t s) {
    const dim3 grid((unsigned)((a.V + 63) / 64), (unsigned)((a.R + 16 * kMT - 1) / (16 * kMT)));
    if (dtype == SV_DTYPE_F32) {
        hipLaunchKernelGGL((logits_stream_kernel<kMT, float>), grid, dim3(256), 0, s, a);
    } else {
        hipLaunchKernelGGL((logits_stream_kernel<kMT, uint16_t>), grid, dim3(256), 0, s, a);
    }
}

}  // namespace

extern "C" int spec_head_quantize(const void* src, int dtype, int rows, int H, int block_rows,
                                  void* out_codes, void* out_scales, void* stream) {
    if (rows < 0 || rows > SV_MAX_VOCAB || H < 8 || H % 8 != 0 || H > SV_MAX_HIDDEN ||
        (block_rows != 1 && block_rows != kBlock)) {
        return SV_ERR_ARG;
    }
    if (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16) return SV_ERR_DTYPE;
    if (rows == 0) return SV_OK;
    if (!src || !out_codes || !out_scales) return SV_ERR_NULL;
    if (!aligned(src, 16) || !aligned(out_codes, 16)) return SV_ERR_ALIGN;
    const int blocks = (H + kBlock - 1) / kBlock;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t* codes = static_cast<uint8_t*>(out_codes);
    uint8_t* scales = static_cast<uint8_t*>(out_scales);
    const dim3 grid(block_rows == 1
                        ? (unsigned)(((long long)rows * blocks * 16 + 255) / 256)
                        : (unsigned)((rows + kBlock - 1) / kBlock * blocks));
    if (dtype == SV_DTYPE_F32) {
        const float* p = static_cast<const float*>(src);
        if (block_rows == 1) {
            hipLaunchKernelGGL((quantize_rows_kernel<float>), grid, dim3(256), 0, s, p, rows, H,
                               blocks, codes, scales);
        } else {
            hipLaunchKernelGGL((quantize_blocks_kernel<float>), grid, dim3(256), 0, s, p, rows, H,
                               blocks, codes, scales);
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(src);
        if (block_rows == 1) {
            hipLaunchKernelGGL((quantize_rows_kernel<uint16_t>), grid, dim3(256), 0, s, p, rows, H,
                               blocks, codes, scales);
        } else {
            hipLaunchKernelGGL((quantize_blocks_kernel<uint16_t>), grid, dim3(256), 0, s, p, rows,
                               H, blocks, codes, scales);
        }
    }
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

extern "C" int spec_head_logits(const void* h_codes, const void* h_scales, const void* w_codes,
                                const void* w_scales, int R, int H, int V, int dtype, void* out,
                                void* stream) {
    if (R < 0 || R > SV_MAX_VOCAB || H < 1 || H > SV_MAX_HIDDEN || V < 1 || V > SV_MAX_VOCAB) {
        return SV_ERR_ARG;
    }
    if (dtype != SV_DTYPE_F32 && dtype != SV_DTYPE_BF16) return SV_ERR_DTYPE;
    if (R == 0) return SV_OK;
    if (!h_codes || !h_scales || !w_codes || !w_scales || !out) return SV_ERR_NULL;
    if (!aligned(h_codes, 16) || !aligned(w_codes, 16) ||
        !aligned(out, dtype == SV_DTYPE_F32 ? 4 : 2)) {
        return SV_ERR_ALIGN;
    }
    LogitArgs a{static_cast<const uint8_t*>(h_codes), static_cast<const uint8_t*>(h_scales),
                static_cast<const uint8_t*>(w_codes), static_cast<const uint8_t*>(w_scales),
                out, R, V, (H + kBlock - 1) / kBlock};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int tiles = (R + 15) / 16;
    if (tiles == 1) launch_stream<1>(a, dtype, s);
    else if (tiles == 2) launch_stream<2>(a, dtype, s);
    else if (tiles == 3) launch_stream<3>(a, dtype, s);
    else launch_stream<4>(a, dtype, s);
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
