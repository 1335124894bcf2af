// cache_rows.h -- eight channels of one token and head at a time, between fp32 or
// bf16 rows and the tiles of the paged 4-bit cache. Shared by the kernels that
// write and read tokens. Internal.
#pragma once

#include "cache_tile.h"

namespace svcache {

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
    amax = max(amax, (unsigned)__builtin_amdgcn_update_dpp(0, (int)amax, 0xb1, 0xf, 0xf, true));    // lane ^ 1
    amax = max(amax, (unsigned)__builtin_amdgcn_update_dpp(0, (int)amax, 0x4e, 0xf, 0xf, true));    // lane ^ 2
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

// Two values rounded to bf16, the first in the low half.
__device__ __forceinline__ unsigned pack2(float a, float b) {
    bf16x2 v;
    v[0] = (__bf16)a;
    v[1] = (__bf16)b;
    return __builtin_bit_cast(unsigned, v);
}

}  // namespace svcache
