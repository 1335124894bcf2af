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
#include <type_traits>

#include "cache_tile.h"
#include "lds_dma.h"

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

// One scale per row and 128 channels: 16 lanes of 8 channels a block. Bound by
// the launch for a step's states (48 x 2,560: 2.6 us), by HBM for many.
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

// One scale per 128 x 128 block: a workgroup each, 8 values x 8 rows a thread,
// held in registers between the maximum and the codes, so that HBM moves every
// byte once: 151,936 x 2,560 in bf16 take 209 us, 5.6 TB/s.
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

// The product, bound by the head's bytes up to about 64 rows (48 rows of fp32
// logits under 151,936 x 2,560: 93 us, 4.5 TB/s) and by LDS and the matrix cores
// above: workgroups hold tiles of TV vocabulary columns x TR rows, the operands'
// codes streamed through an LDS ring of two blocks of 128 channels by
// buffer-to-LDS loads (with three blocks fewer workgroups fit a CU: one row took
// 78 us against 68, 48 rows 100 against 92). A row's 128 bytes are eight chunks
// of 16; chunk c of row i lies at position c ^ (i & 7), so that eight rows at one
// chunk column use eight positions (the loads choose their global chunk
// accordingly; LDS itself is filled linearly). Rows are half a sweep of the banks
// apart, so even rows meet in one half and odd ones in the other, and a fragment's
// read takes twice the cycles it could: SQ_LDS_BANK_CONFLICT is half of
// SQ_LDS_IDX_ACTIVE, 3.8 and 4.0 cycles an LDS instruction for 48 and 2,560 rows
// under 151,936 x 2,560. (head_stats.hip's c ^ ((i / 2) % 8) has next to none.)
//
// kF8: 8-bit matrix instructions with both scales as their operands, for bf16
// logits. Otherwise the codes are decoded to bf16 (exact, scales included) in
// registers and multiplied in bf16, for fp32 logits: the 8-bit instructions
// keep a sum of products only to about 2^-17 of its terms (relative error
// 1.4e-5 of a row's norm, measured at 128, 2,560 and 10,240 channels): under a
// two-hundredth of a bf16 rounding, but two hundred fp32 ones. 2,560 rows of fp32
// logits under 151,936 x 2,560 take 1,730 us (a large bf16 product's rate: 1,414);
// every wavefront decodes what it reads.
template <int TV_, int TR_, int WV_, int WR_, bool kF8_, typename O_>
struct Cfg {
    static constexpr int TV = TV_, TR = TR_, WV = WV_, WR = WR_;
    static constexpr bool kF8 = kF8_;
    using O = O_;
    static constexpr int kWaves = WV * WR, kThreads = 64 * kWaves;
    static constexpr int MV = TV / WV / 32, MR = TR / WR / 32;    // 32 x 32 tiles of a wave
    static constexpr int kLoads = (TV + TR) / 8 / kWaves;         // buffer loads per wave and stage
    static constexpr int kStageBytes = (TV + TR) * kBlock;
    static constexpr int kRing = 2 * kStageBytes;
    static constexpr int kRowBytes = TV * (int)sizeof(O);
    // Rows that the ring holds of the finished tile.
    static constexpr int kPass = kRing / kRowBytes < TR ? kRing / kRowBytes / 64 * 64 : TR;
    static_assert(TV % (32 * WV) == 0 && TR % (32 * WR) == 0, "whole 32 x 32 tiles");
    static_assert((TV + TR) % (8 * kWaves) == 0 && TV % (8 * kWaves) == 0, "even loads");
    static_assert(128 % (TV / WV) == 0, "one head scale per wave and block");
    static_assert(kPass >= 32 && TR % kPass == 0 && kPass % (TR / WR) == 0, "whole waves per pass");
};

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;

__device__ __forceinline__ uint2 pack4(const float (&v)[4], uint16_t) {
    bf16x2 a, b;
    a[0] = (__bf16)v[0]; a[1] = (__bf16)v[1];
    b[0] = (__bf16)v[2]; b[1] = (__bf16)v[3];
    return make_uint2(__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b));
}
__device__ __forceinline__ f32x4 pack4(const float (&v)[4], float) {
    return f32x4{v[0], v[1], v[2], v[3]};
}

template <typename C>
__global__ __launch_bounds__(C::kThreads) void logits_kernel(LogitArgs a, int v_tiles, int band) {
    using O = typename C::O;
    __shared__ __attribute__((aligned(128))) unsigned char ring[C::kRing];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // Tile order: workgroups go round-robin over the 8 XCDs; each XCD takes
    // every eighth column tile and walks a band of row tiles under it, so
    // that a tile of the head is read from HBM once per band and the band's
    // states stay in that XCD's L2.
    const int r_tiles = (a.R + C::TR - 1) / C::TR;
    const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3;
    const int v_per = (v_tiles + 7) / 8;
    const int b0 = at / (v_per * band) * band;
    const int in_band = min(band, r_tiles - b0);
    const int rest = at - b0 * v_per;
    const int vt = rest / in_band * 8 + xcd, rt = b0 + rest % in_band;
    if (vt >= v_tiles) return;
    const int v0 = vt * C::TV, r0 = rt * C::TR;

    const unsigned pitch = (unsigned)a.blocks * kBlock;
    const __amdgpu_buffer_rsrc_t wsrc =
        svdma::rsrc(a.w + (long long)v0 * pitch, (unsigned)min(C::TV, a.V - v0) * pitch);
    const __amdgpu_buffer_rsrc_t hsrc =
        svdma::rsrc(a.h + (long long)r0 * pitch, (unsigned)min(C::TR, a.R - r0) * pitch);
    // Load i of a wave covers rows 8 (i kWaves + wave) .. + 7 of the stage, the
    // head's rows first. Rows past the operand read as zeros.
    const unsigned lane_off = (lane >> 3) * pitch + (((lane & 7) ^ (lane >> 3)) * 16);
    auto fetch = [&](int k) {
        unsigned char* base = ring + (k & 1) * C::kStageBytes;
        #pragma unroll
        for (int i = 0; i < C::kLoads; ++i) {
            const int row = 8 * (i * C::kWaves + wave);
            const bool head = i * C::kWaves * 8 < C::TV;
            const unsigned off = lane_off + (unsigned)(head ? row : row - C::TV) * pitch + k * kBlock;
            svdma::load16(head ? wsrc : hsrc, off, base + row * kBlock);
        }
    };

    const int wv = wave % C::WV, wr = wave / C::WV;
    const int vrow = wv * 32 * C::MV, rrow = wr * 32 * C::MR;
    const uint8_t* wsp = a.ws + (long long)(min(v0 + vrow, a.V - 1) / kBlock) * a.blocks;
    const uint8_t* hsp[C::MR];
    #pragma unroll
    for (int j = 0; j < C::MR; ++j) {
        hsp[j] = a.hs + (long long)min(r0 + rrow + 32 * j + (lane & 31), a.R - 1) * a.blocks;
    }

    f32x16 acc[C::MV][C::MR] = {};
    unsigned sw = wsp[0], sh[C::MR];
    #pragma unroll
    for (int j = 0; j < C::MR; ++j) sh[j] = hsp[j][0];
    fetch(0);
    const unsigned lds_row = (lane & 31) * kBlock;
    for (int k = 0; k < a.blocks; ++k) {
        svdma::wait_vm<0>();          // stage k has arrived
        svdma::ring_barrier();
        // Everyone has read stage k - 1: its place is free.
        if (k + 1 < a.blocks) fetch(k + 1);
        const unsigned sw_now = sw;
        unsigned sh_now[C::MR];
        #pragma unroll
        for (int j = 0; j < C::MR; ++j) sh_now[j] = sh[j];
        if (k + 1 < a.blocks) {
            sw = wsp[k + 1];
            #pragma unroll
            for (int j = 0; j < C::MR; ++j) sh[j] = hsp[j][k + 1];
        }
        const unsigned char* wbase = ring + (k & 1) * C::kStageBytes + vrow * kBlock + lds_row;
        const unsigned char* hbase =
            ring + (k & 1) * C::kStageBytes + (C::TV + rrow) * kBlock + lds_row;
        #pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int c0 = 4 * half + 2 * (lane >> 5);
            const int p0 = (c0 ^ (lane & 7)) * 16, p1 = ((c0 + 1) ^ (lane & 7)) * 16;
            u32x4 wc[C::MV][2], hc[C::MR][2];
            #pragma unroll
            for (int i = 0; i < C::MV; ++i) {
                wc[i][0] = *reinterpret_cast<const u32x4*>(wbase + i * 32 * kBlock + p0);
                wc[i][1] = *reinterpret_cast<const u32x4*>(wbase + i * 32 * kBlock + p1);
            }
            #pragma unroll
            for (int j = 0; j < C::MR; ++j) {
                hc[j][0] = *reinterpret_cast<const u32x4*>(hbase + j * 32 * kBlock + p0);
                hc[j][1] = *reinterpret_cast<const u32x4*>(hbase + j * 32 * kBlock + p1);
            }
            if constexpr (C::kF8) {
                i32x8 hf[C::MR];
                #pragma unroll
                for (int j = 0; j < C::MR; ++j) {
                    hf[j] = __builtin_bit_cast(i32x8, __builtin_shufflevector(hc[j][0], hc[j][1], 0, 1, 2, 3, 4, 5, 6, 7));
                }
                #pragma unroll
                for (int i = 0; i < C::MV; ++i) {
                    const i32x8 wf = __builtin_bit_cast(i32x8, __builtin_shufflevector(wc[i][0], wc[i][1], 0, 1, 2, 3, 4, 5, 6, 7));
                    #pragma unroll
                    for (int j = 0; j < C::MR; ++j) {
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                            wf, hf[j], acc[i][j], 0, 0, 0, (int)sw_now, 0, (int)sh_now[j]);
                    }
                }
            } else {
                #pragma unroll
                for (int q = 0; q < 4; ++q) {
                    bf16x8 hf[C::MR];
                    #pragma unroll
                    for (int j = 0; j < C::MR; ++j) {
                        hf[j] = decode8(hc[j][q >> 1][2 * (q & 1)], hc[j][q >> 1][2 * (q & 1) + 1],
                                        scale_of(sh_now[j]));
                    }
                    #pragma unroll
                    for (int i = 0; i < C::MV; ++i) {
                        const bf16x8 wf = decode8(wc[i][q >> 1][2 * (q & 1)],
                                                  wc[i][q >> 1][2 * (q & 1) + 1], scale_of(sw_now));
                        #pragma unroll
                        for (int j = 0; j < C::MR; ++j) {
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf, hf[j], acc[i][j], 0, 0, 0);
                        }
                    }
                }
            }
        }
    }

    // The tile goes out through LDS, row by row: 16-byte chunk c of row i at
    // c ^ (i & mask).
    constexpr int kChunks = C::kRowBytes / 16;
    constexpr int kMask = (kChunks < 32 ? kChunks : 32) - 1;
    constexpr int kPer = 16 / (int)sizeof(O);                      // values of a chunk
    const bool wide = (a.V * (int)sizeof(O)) % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
    O* out = static_cast<O*>(a.out);
    #pragma unroll
    for (int pass = 0; pass < C::TR / C::kPass; ++pass) {
        __syncthreads();
        if (rrow / C::kPass == pass) {
            #pragma unroll
            for (int j = 0; j < C::MR; ++j) {
                const int row = rrow % C::kPass + 32 * j + (lane & 31);
                #pragma unroll
                for (int i = 0; i < C::MV; ++i) {
                    #pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float v[4] = {acc[i][j][4 * g], acc[i][j][4 * g + 1],
                                            acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                        const int col = vrow + 32 * i + 8 * g + 4 * (lane >> 5);
                        unsigned char* dst = ring + row * C::kRowBytes +
                                             ((col / kPer) ^ (row & kMask)) * 16 + col % kPer * sizeof(O);
                        const auto w = pack4(v, O{});
                        __builtin_memcpy(__builtin_assume_aligned(dst, sizeof(w)), &w, sizeof(w));
                    }
                }
            }
        }
        __syncthreads();
        const int rows = min(C::kPass, a.R - r0 - pass * C::kPass), cols = min(C::TV, a.V - v0);
        O* dst = out + (long long)(r0 + pass * C::kPass) * a.V + v0;
        if (wide) {
            for (int i = threadIdx.x; i < C::kPass * kChunks; i += C::kThreads) {
                const int row = i / kChunks, c = i % kChunks;
                if (row < rows && c * kPer < cols) {
                    *reinterpret_cast<u32x4*>(dst + (long long)row * a.V + c * kPer) =
                        *reinterpret_cast<const u32x4*>(ring + row * C::kRowBytes + (c ^ (row & kMask)) * 16);
                }
            }
        } else {
            for (int i = threadIdx.x; i < C::kPass * C::TV; i += C::kThreads) {
                const int row = i / C::TV, col = i % C::TV;
                if (row < rows && col < cols) {
                    dst[(long long)row * a.V + col] = *reinterpret_cast<const O*>(
                        ring + row * C::kRowBytes + ((col / kPer) ^ (row & kMask)) * 16 + col % kPer * sizeof(O));
                }
            }
        }
    }
}

template <typename C>
void launch_logits(const LogitArgs& a, hipStream_t s) {
    const int v_tiles = (a.V + C::TV - 1) / C::TV, r_tiles = (a.R + C::TR - 1) / C::TR;
    const int bands = (r_tiles + 7) / 8;
    const int band = (r_tiles + bands - 1) / bands;
    const long long grid = (long long)(v_tiles + 7) / 8 * 8 * r_tiles;
    hipLaunchKernelGGL((logits_kernel<C>), dim3((unsigned)grid), dim3(C::kThreads), 0, s, a, v_tiles,
                       band);
}

// bf16 logits of many rows and columns, 8-bit products: tiles of 256 x 256 by
// four wavefronts, one a SIMD, of 128 x 128 each, so that a fragment read from
// LDS serves four products (with eight wavefronts of 128 x 64 LDS is as busy as
// the matrix cores, conflicts included). The accumulators are 256 registers, and
// the fragments are held twice:
//  - A stage (128 channels) has two phases, one half of its channels each. While
//    a phase's 16 products run, the next phase's fragments are read; in the
//    second the place in LDS that has been read is filled with the stage after
//    the next. Products, reads and loads alternate in the order written here.
//  - One barrier a stage, between its phases: every wave has read the stage
//    whole, and the next one has arrived.
// A workgroup goes through its tiles without a break: the next tile's first
// stages are under way while one ends, and its outputs go straight from the
// registers.
// 2,560 rows x 151,936 columns x 2,560 channels: 945..965 us (logits_kernel's 256
// x 256 tiles: 1,005), 8,192 of each: 403 (450). Products alone take two thirds of
// the loop's time at 1.9 GHz; 140 us are the outputs' 778 MB, which all workgroups
// write at the same time. (Measured with a wait for a stage that took 1 % less but
// counted on how many loads the compiler makes: 930, without the outputs 788, and
// 921 without waiting for a tile's stores before the next one's second stage.)
struct Large {
    static constexpr int T = 256, kWaves = 4, M = 4;        // tile, wavefronts, 32 x 32 tiles of a wave
    static constexpr int kLoads = 2 * T / 8 / kWaves, kStageBytes = 2 * T * kBlock;
};

__global__ __launch_bounds__(256) void logits_large_kernel(LogitArgs a, int v_tiles, int band, int tiles) {
    using C = Large;
    __shared__ __attribute__((aligned(128))) unsigned char ring[2 * C::kStageBytes];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int vrow = (wave & 1) * 128, rrow = (wave >> 1) * 128;
    const unsigned pitch = (unsigned)a.blocks * kBlock;

    // Places as in logits_kernel; of the padded ones there may be none.
    const int r_tiles = (a.R + C::T - 1) / C::T, v_per = (v_tiles + 7) / 8;
    struct Place {
        int v0, r0;
    };
    auto place = [&](int id) {
        const int xcd = id & 7, at = id >> 3;
        const int b0 = at / (v_per * band) * band, in_band = min(band, r_tiles - b0), rest = at - b0 * v_per;
        return Place{(rest / in_band * 8 + xcd) * C::T, (b0 + rest % in_band) * C::T};
    };
    auto valid = [&](int id) {                              // the first from id on that is one
        while (id < tiles && place(id).v0 >= a.V) id += gridDim.x;
        return id;
    };
    int id = valid(blockIdx.x);
    if (id >= tiles) return;

    // What a tile reads. Rows past an operand read as zeros; of no tile none is read.
    struct Source {
        const uint8_t *w, *h;
        unsigned wn, hn;
    };
    auto source = [&](const Place& p, bool some) {
        return Source{a.w + (long long)p.v0 * pitch, a.h + (long long)p.r0 * pitch,
                      some ? (unsigned)min(C::T, a.V - p.v0) * pitch : 0u,
                      some ? (unsigned)min(C::T, a.R - p.r0) * pitch : 0u};
    };
    const unsigned lane_off = (lane >> 3) * pitch + (((lane & 7) ^ (lane >> 3)) * 16);
    // Load n of a wave: rows 8 (n kWaves + wave) .. + 7 of the stage, the head's first.
    auto fetch = [&](const Source& s, int n, int k, int slot) {
        const int row = 8 * (n * C::kWaves + wave);
        const bool head = n * C::kWaves * 8 < C::T;
        const unsigned off = lane_off + (unsigned)(head ? row : row - C::T) * pitch + k * kBlock;
        svdma::load16(head ? svdma::rsrc(s.w, s.wn) : svdma::rsrc(s.h, s.hn), off,
                      ring + slot * C::kStageBytes + row * kBlock);
    };
    // Where a tile's scales start.
    struct Scales {
        unsigned w, h[C::M];
    };
    auto scales_of = [&](const Place& p) {
        Scales s;
        s.w = (unsigned)(min(p.v0 + vrow, a.V - 1) / kBlock * a.blocks);
        #pragma unroll
        for (int j = 0; j < C::M; ++j) s.h[j] = (unsigned)(min(p.r0 + rrow + 32 * j + (lane & 31), a.R - 1) * a.blocks);
        return s;
    };
    Scales at;                                              // of the next stage
    unsigned sw, sh[C::M];
    auto load_scales = [&]() {
        sw = a.ws[at.w];
        #pragma unroll
        for (int j = 0; j < C::M; ++j) sh[j] = a.hs[at.h[j]];
    };

    i32x8 wf[2][C::M], hf[2][C::M];
    const unsigned lds_row = (lane & 31) * kBlock;
    auto read = [&](int slot, int half, int n) {            // fragment n: rows', then columns'
        const int c0 = 4 * half + 2 * (lane >> 5);
        const int p0 = (c0 ^ (lane & 7)) * 16, p1 = ((c0 + 1) ^ (lane & 7)) * 16;
        const unsigned char* row = ring + slot * C::kStageBytes + lds_row +
                                   (n < C::M ? C::T + rrow + 32 * n : vrow + 32 * (n - C::M)) * kBlock;
        const i32x8 f = __builtin_bit_cast(i32x8, __builtin_shufflevector(
            *reinterpret_cast<const u32x4*>(row + p0), *reinterpret_cast<const u32x4*>(row + p1),
            0, 1, 2, 3, 4, 5, 6, 7));
        if (n < C::M) hf[half][n] = f;
        else wf[half][n - C::M] = f;
    };
    f32x16 acc[C::M][C::M];
    unsigned sw_now, sh_now[C::M];
    // Waits for them here rather than behind a tile's stores.
    auto use_scales = [&]() {
        sw_now = sw;
        asm volatile("" : "+v"(sw_now));
        #pragma unroll
        for (int j = 0; j < C::M; ++j) {
            sh_now[j] = sh[j];
            asm volatile("" : "+v"(sh_now[j]));
        }
    };
    auto product = [&](int half, int n) {
        const int i = n / C::M, j = n % C::M;
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            wf[half][i], hf[half][j], acc[i][j], 0, 0, 0, (int)sw_now, 0, (int)sh_now[j]);
        __builtin_amdgcn_sched_barrier(0);
    };

    Place now = place(id);
    Source from = source(now, true);
    at = scales_of(now);
    load_scales();
    #pragma unroll
    for (int n = 0; n < C::kLoads; ++n) fetch(from, n, 0, 0);
    #pragma unroll
    for (int n = 0; n < C::kLoads; ++n) fetch(from, n, 1, 1);
    svdma::wait_vm<C::kLoads>();
    svdma::ring_barrier();
    #pragma unroll
    for (int n = 0; n < 2 * C::M; ++n) read(0, 0, n);
    use_scales();
    int slot = 0;
    for (;;) {
        const int next = valid(id + gridDim.x);
        const bool some = next < tiles;
        const Place then = some ? place(next) : now;
        const Source then_from = source(then, some);
        const Scales then_at = scales_of(then);
        #pragma unroll
        for (int i = 0; i < C::M; ++i) {
            #pragma unroll
            for (int j = 0; j < C::M; ++j) acc[i][j] = f32x16{};
        }
        int k = 0;
        do {
            __builtin_amdgcn_sched_barrier(0);
            #pragma unroll
            for (int n = 0; n < C::M * C::M; ++n) {
                product(0, n);
                if (n < 2 * C::M) read(slot, 1, n);
                __builtin_amdgcn_sched_barrier(0);
            }
            // A branch here would make a second loop of the last stage, and copies
            // of the accumulators between the two.
            const bool last = k + 1 == a.blocks;
            at.w = last ? then_at.w : at.w + 1;
            #pragma unroll
            for (int j = 0; j < C::M; ++j) at.h[j] = last ? then_at.h[j] : at.h[j] + 1;
            const bool wrap = k + 2 >= a.blocks;
            const Source s = wrap ? then_from : from;
            const int ks = wrap ? k + 2 - a.blocks : k + 2;
            __builtin_amdgcn_sched_barrier(0);
            // The next stage has arrived: its loads were issued a phase ago, and
            // nothing since. (A count that left the scales' loads outstanding
            // would rest on how many of them the compiler makes.)
            svdma::wait_vm<0>();
            __builtin_amdgcn_sched_barrier(0);
            load_scales();                                  // of the next stage
            svdma::ring_barrier();
            __builtin_amdgcn_sched_barrier(0);
            #pragma unroll
            for (int n = 0; n < C::M * C::M; ++n) {
                product(1, n);
                if (n < 2 * C::M) read(slot ^ 1, 0, n);
                fetch(s, n, ks, slot);
                __builtin_amdgcn_sched_barrier(0);
            }
            use_scales();
            slot ^= 1;
        } while (++k < a.blocks);
        // A lane holds row lane % 32 of every 32 x 32 tile and columns 8 g + 4
        // (lane / 32) .. + 3: swapping halves gives it eight in a row.
        const int col0 = vrow + 8 * (lane >> 5), cols = a.V - now.v0;
        const __amdgpu_buffer_rsrc_t dst = svdma::rsrc(
            static_cast<const uint16_t*>(a.out) + (long long)now.r0 * a.V + now.v0,
            ((unsigned)min(C::T, a.R - now.r0) * (unsigned)a.V - (unsigned)now.v0) * 2);
        #pragma unroll
        for (int j = 0; j < C::M; ++j) {
            const unsigned off = ((unsigned)(rrow + 32 * j + (lane & 31)) * (unsigned)a.V + (unsigned)col0) * 2;
            #pragma unroll
            for (int i = 0; i < C::M; ++i) {
                // Read one by one: the compiler would take them all over into
                // ordinary registers, in the loop over stages.
                asm volatile("" : "+a"(acc[i][j]));
                __builtin_amdgcn_sched_barrier(0);
                #pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const f32x16& v = acc[i][j];
                    const float lo[4] = {v[8 * m], v[8 * m + 1], v[8 * m + 2], v[8 * m + 3]};
                    const float hi[4] = {v[8 * m + 4], v[8 * m + 5], v[8 * m + 6], v[8 * m + 7]};
                    const uint2 x = pack4(lo, uint16_t{}), y = pack4(hi, uint16_t{});
                    const auto p = __builtin_amdgcn_permlane32_swap(x.x, y.x, false, false);
                    const auto q = __builtin_amdgcn_permlane32_swap(x.y, y.y, false, false);
                    const int c = 32 * i + 16 * m;
                    // Past the last row or column: past the end of the buffer, dropped.
                    __builtin_amdgcn_raw_buffer_store_b128(u32x4{p[0], q[0], p[1], q[1]}, dst,
                                                           col0 + c < cols ? (int)(off + 2 * c) : -1, 0, 0);
                }
            }
        }
        if (!some) break;
        id = next;
        now = then;
        from = then_from;
    }
    svdma::wait_vm<0>();            // no load into LDS outlives the workgroup
}

void launch_large(const LogitArgs& a, hipStream_t s) {
    const int v_tiles = (a.V + Large::T - 1) / Large::T, r_tiles = (a.R + Large::T - 1) / Large::T;
    const int bands = (r_tiles + 7) / 8, band = (r_tiles + bands - 1) / bands;
    const int tiles = (v_tiles + 7) / 8 * 8 * r_tiles;
    hipLaunchKernelGGL(logits_large_kernel, dim3((unsigned)(tiles < 256 ? tiles : 256)), dim3(256), 0, s, a,
                       v_tiles, band, tiles);
}

// Tiles by the number of rows and columns. Up to 64 rows the head's bytes
// decide and the tile is as narrow as its rows. Above, the tile whose rounds of
// workgroups take least: a round of 256 x 256 tiles (one workgroup per CU) as
// the unit, one of 128 x 128 tiles (two) measured 0.62 to 0.7 of it and one of 64
// x 64 tiles, counted as three per CU, 0.375 to 0.4 (since the rings have two
// stages five are resident; the rule was measured with what it counts). (20,000
// columns x 5,120 channels, bf16: 300 rows take 53, 44, 71 us with them, 700 rows 63, 81, 136; 151,936 columns x
// 2,560, 160 rows 126, 139, -; 2,560 columns x 4,096, 1,024 rows 44, 31, 28. The
// rule's choice was the least, or within 4 % of it, at 11 sizes in either type.)
template <bool kF8, typename O>
void launch_rows(const LogitArgs& a, hipStream_t s) {
    if (a.R <= 32) return launch_logits<Cfg<64, 32, 2, 1, kF8, O>>(a, s);
    if (a.R <= 64) {
        // Twice the columns once every CU has two such tiles (48 rows of fp32
        // logits under 151,936 columns: 97 against 104 us, 100,000: 55 and 54,
        // 65,536: 30 and 30, 40,000: 26 against 23).
        if (a.V >= 128 * 512) return launch_logits<Cfg<128, 64, 4, 1, kF8, O>>(a, s);
        return launch_logits<Cfg<64, 64, 2, 2, kF8, O>>(a, s);
    }
    auto rounds = [&](long long tile, long long held) {
        return (double)(((a.V + tile - 1) / tile * ((a.R + tile - 1) / tile) + held - 1) / held);
    };
    const double large = rounds(256, 256), middle = 0.62 * rounds(128, 512), small = 0.375 * rounds(64, 768);
    if (large <= middle && large <= small) {
        // Its outputs are 16-byte pieces, and it starts with two stages.
        if (kF8 && a.blocks > 1 && a.V % 8 == 0 && aligned(a.out, 16)) launch_large(a, s);
        else launch_logits<Cfg<256, 256, 2, 4, kF8, O>>(a, s);
    } else if (middle <= small) {
        launch_logits<Cfg<128, 128, 2, 2, kF8, O>>(a, s);
    } else {
        launch_logits<Cfg<64, 64, 2, 2, kF8, O>>(a, s);
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
    auto launch = [&](auto* p) {
        using S = std::remove_pointer_t<decltype(p)>;
        if (block_rows == kBlock) {
            hipLaunchKernelGGL((quantize_blocks_kernel<std::remove_const_t<S>>),
                               dim3((unsigned)((rows + kBlock - 1) / kBlock * blocks)), dim3(256), 0,
                               s, p, rows, H, blocks, codes, scales);
            return;
        }
        // A launch holds fewer than 2^32 threads, 16 a block.
        const int most = (int)(((1ll << 31) / 16) / blocks);
        for (int r = 0; r < rows; r += most) {
            const int n = rows - r < most ? rows - r : most;
            hipLaunchKernelGGL((quantize_rows_kernel<std::remove_const_t<S>>),
                               dim3((unsigned)(((long long)n * blocks * 16 + 255) / 256)), dim3(256), 0,
                               s, p + (long long)r * H, n, H, blocks,
                               codes + (long long)r * blocks * kBlock, scales + (long long)r * blocks);
        }
    };
    if (dtype == SV_DTYPE_F32) launch(static_cast<const float*>(src));
    else launch(static_cast<const uint16_t*>(src));
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
    if (dtype == SV_DTYPE_F32) launch_rows<false, float>(a, s);
    else launch_rows<true, uint16_t>(a, s);
    return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
