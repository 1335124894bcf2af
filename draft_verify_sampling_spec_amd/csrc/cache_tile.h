// cache_tile.h -- the layout of the paged 4-bit key/value cache and the
// 4-bit number format, shared by the kernels that write, read and attend
// over it. Internal; the layout itself is documented in spec_verify.h.
//
// A page holds page_size tokens (a power of two, at least 32) of every kv
// head: [kv head][page_size / 32] tiles of 34 D bytes, one tile being 32
// consecutive tokens of one head. Inside a tile every part lies in the order
// in which the attention's wavefront loads it, so that each of its loads is
// one contiguous run and needs no transposition:
//   keys' codes    16 D  [half: token / 16][unit: U bytes][token % 16][U]
//   values' codes  16 D  [128 channels][half][quad: token % 16 / 4]
//                        [x: 16 pieces of C bytes][token % 4][C]
//   keys' scales      D  [group: 32 channels][token % 16][half]
//   values' scales    D  [group][quad][half][token % 4]
// with U = min(16, D / 8) and C = min(4, D / 32). A byte holds two codes, the
// even channel's in the low half.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "spec_verify.h"

namespace svcache {

constexpr int kTile = 32;       // tokens of a tile
constexpr int kGroup = 32;      // channels that share a scale
constexpr int kMinScaleByte = 127 - 64;   // the smallest scale, 2^-64

template <int D>
struct Tile {
    static_assert(D == 64 || D == 128 || D == 256, "head sizes of the cache");
    static constexpr int U = D / 8 < 16 ? D / 8 : 16;      // bytes of a key unit
    static constexpr int C = D / 32 < 4 ? D / 32 : 4;      // bytes of a value piece
    static constexpr int kPlanes = D <= 128 ? 1 : D / 128;  // value planes of 16 pieces
    static constexpr int kGroups = D / kGroup;
    static constexpr int kBytes = 34 * D;
    static constexpr int kVCodes = 16 * D, kKScales = 32 * D, kVScales = 33 * D;

    // Byte offsets of token tok (0..31): the 4 bytes (8 channels) at byte
    // 4 c of its D / 2 key codes, and of value channels 8 c .. 8 c + 7 (for
    // D = 64 these are two 2-byte pieces, the second 4 C bytes on).
    __host__ __device__ static constexpr int k_codes(int tok, int c) {
        return (tok >> 4) * (8 * D) + (4 * c / U) * (16 * U) + (tok & 15) * U + (4 * c) % U;
    }
    __host__ __device__ static constexpr int v_codes(int tok, int c) {
        const int piece = 4 * c / C, plane = piece >> 4, x = piece & 15;
        return kVCodes + ((plane * 2 + (tok >> 4)) * 4 + ((tok & 15) >> 2)) * (64 * C) +
               x * (4 * C) + (tok & 3) * C;
    }
    __host__ __device__ static constexpr int k_scale(int tok, int g) {
        return kKScales + g * 32 + (tok & 15) * 2 + (tok >> 4);
    }
    __host__ __device__ static constexpr int v_scale(int tok, int g) {
        return kVScales + g * 32 + ((tok & 15) >> 2) * 8 + (tok >> 4) * 4 + (tok & 3);
    }
};

// The scale byte of a block whose largest magnitude has the bit pattern
// amax_bits (fp32, sign clear): 2^(byte - 127) is the smallest power of two,
// at least 2^-64, with amax <= top * scale, top = (1 + kTopMantissa 2^-23) *
// 2^kTopExponent. A carry out of the mantissa means that amax needs the next
// power. At most the scale whose largest value is still finite in fp32 (what
// is larger saturates). 255 (not a number) when the block holds a NaN or an
// infinity.
template <unsigned kTopMantissa, int kTopExponent>
__device__ __forceinline__ unsigned scale_byte(unsigned amax_bits) {
    if (amax_bits >= 0x7f800000u) return 255u;
    const int e = (int)((amax_bits + (0x7fffffu - kTopMantissa)) >> 23) - kTopExponent;
    return (unsigned)min(max(e, kMinScaleByte), 254 - kTopExponent);
}

// e2m1: largest value 6 = 1.5 * 2^2.
__device__ __forceinline__ unsigned cache_scale_byte(unsigned amax_bits) {
    return scale_byte<0x400000u, 2>(amax_bits);
}

// 2^(byte - 127) as fp32 (255 gives +inf, which the conversions below read
// as a NaN scale).
__device__ __forceinline__ float scale_of(unsigned byte) { return __uint_as_float(byte << 23); }

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;

// Byte kByte of `codes` (two e2m1 values, the low half first) times scale as
// two bf16, exactly (scales of the cache keep every product normal). A NaN
// scale makes both NaN, whatever the codes.
template <int kByte>
__device__ __forceinline__ unsigned decode2(unsigned codes, float scale) {
    return __builtin_bit_cast(unsigned,
                              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, kByte));
}

// Page geometry of a call.
struct Pages {
    const int32_t* table;   // [B, max_pages]
    int max_pages, num_pages;
    int shift;              // log2(page_size)
    int heads;

    // The page that holds position pos (>= 0) of request b, as the table has it.
    __device__ __forceinline__ int page(int b, int pos) const {
        return table[(size_t)b * max_pages + (pos >> shift)];
    }
    // Tile of head h with position pos in that page: byte offset in the cache,
    // or -1 when the page is outside the pool.
    __device__ __forceinline__ long long tile_in(int page, int h, int pos, int tile_bytes) const {
        if ((unsigned)page >= (unsigned)num_pages) return -1;
        const int per = 1 << (shift - 5);
        return (((long long)page * heads + h) * per + ((pos >> 5) & (per - 1))) * tile_bytes;
    }
    __device__ __forceinline__ long long tile(int b, int h, int pos, int tile_bytes) const {
        return tile_in(page(b, pos), h, pos, tile_bytes);
    }
};

__device__ __forceinline__ void flag(int32_t* status, unsigned bits) {
    if (status) atomicOr(reinterpret_cast<unsigned*>(status), bits);
}

// A request's block: its context length (negative: an empty slot) and its
// tokens (budget + 1, the budget clamped into [0, width - 1]; NULL budgets:
// width). len = 0 (and ctx = 0, so that nothing derived from it overflows):
// nothing to do. A block that does not fit the request's page table row is
// flagged and skipped.
struct Block {
    int ctx, len;
};
__device__ __forceinline__ Block block_of(const int32_t* ctx_lens, const int32_t* budgets, int b,
                                          int width, const Pages& pages, int32_t* status,
                                          bool report) {
    const int ctx = ctx_lens[b];
    if (ctx < 0) return Block{0, 0};
    int n = width;
    if (budgets) {
        const int kb = budgets[b];
        n = min(max(kb, 0), width - 1) + 1;
        if (report && n - 1 != kb) flag(status, SV_FLAG_BAD_BUDGET);
    }
    if ((long long)ctx + n > ((long long)pages.max_pages << pages.shift)) {
        if (report) flag(status, SV_FLAG_BAD_LENGTH);
        return Block{0, 0};
    }
    return Block{ctx, n};
}

inline bool aligned(const void* p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// Host checks of the cache geometry every entry point shares.
inline bool geometry_ok(int heads, int D, int page_size, int max_pages, int num_pages) {
    return heads >= 1 && heads <= SV_MAX_HEADS && (D == 64 || D == 128 || D == 256) &&
           page_size >= kTile && page_size <= SV_MAX_PAGE && (page_size & (page_size - 1)) == 0 &&
           max_pages >= 1 && num_pages >= 1 &&
           (long long)max_pages * page_size <= SV_MAX_CONTEXT;
}

inline Pages make_pages(const int32_t* table, int heads, int page_size, int max_pages,
                        int num_pages) {
    return Pages{table, max_pages, num_pages, __builtin_ctz((unsigned)page_size), heads};
}

}  // namespace svcache
