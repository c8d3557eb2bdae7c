// mx4.hip -- microscaled 4-bit floating point (OCP Microscaling Formats v1.0: E2M1 codes,
// one E8M0 scale for 32 values): rounding, its inverse, and the SwiGLU experts on MX4
// weights and activations.
#include <mutex>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "lds_ring.h"
#include "tile_list.h"
#include "variants.h"

namespace moe {

namespace {

// ---- rounding ------------------------------------------------------------------

constexpr uint8_t kNanScale = 255;

// The scale byte of a block whose largest magnitude has the bits `amax` (sign cleared):
// the exponent of the largest value less that of 4 = 2^2, the grid's top binade.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t amax) {
    if (amax >= 0x7F800000u) return kNanScale;
    const int e = (int)(amax >> 23) - 2;
    return amax == 0u ? 127u : (uint32_t)(e < 0 ? 0 : e);
}
// 2^(s - 127): s = 0 is below the normal numbers.
__device__ __forceinline__ float mx4_unit(uint32_t s) { return __uint_as_float(s == 0u ? 0x00400000u : s << 23); }

// Eight values to eight codes (value 2i in the low half of byte i), nearest even, saturating.
__device__ __forceinline__ uint32_t mx4_codes(const float (&v)[8], uint32_t s) {
    if (s == kNanScale) return 0u;
    const float unit = mx4_unit(s);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], unit, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], unit, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], unit, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], unit, 3);
    return c;
}

// Rows of values start at any element: the memory pipeline takes 16-byte accesses at every address (16384 x 7168 bf16 in
// rows of 7171 there and back 109 us, against 178 by single elements and 107 in dense rows).
typedef f32x4 f32x4u __attribute__((aligned(4)));
typedef u32x4 u32x4u __attribute__((aligned(2)));

// Row and run of run g of a matrix of rows of `runs` runs.  FLAT: the rows are whole runs without gaps, so the
// matrix is one row (16384 x 7168 there and back 2 % less time than with a division for each run).
template <bool FLAT>
__device__ __forceinline__ void mx4_place(int64_t g, int64_t total, int64_t runs, int64_t &r, int64_t &c) {
    if (FLAT) {
        r = 0;
        c = g;
    } else if (total < (1ll << 31)) {
        const uint32_t q = (uint32_t)g / (uint32_t)runs;
        r = q;
        c = (uint32_t)g - q * (uint32_t)runs;
    } else {
        r = g / runs;
        c = g - r * runs;
    }
}

// 16 lanes per run of 128 values, eight values a lane (one 16-byte load of bf16), four lanes a block, whose largest
// magnitude takes two lane exchanges; a run's codes are one whole line of 64 bytes.  Bound by memory: 16384 x 7168 bf16
// to codes 49 us, 297 MB, 6.1 TB/s.  The values are read once, and nontemporal loads keep them from displacing what the
// caches hold: 60 us without.
template <int DT, bool FLAT>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const void *__restrict__ x, int64_t ld, int64_t rows,
                                                           int64_t cols, int64_t runs, uint8_t *__restrict__ q,
                                                           uint8_t *__restrict__ sc) {
    const int64_t total = rows * runs;
    const int sub = threadIdx.x & 15;
    // the loop bound is uniform over the workgroup, so every lane reaches the lane exchanges
    for (int64_t g0 = (int64_t)blockIdx.x * 16; g0 < total; g0 += (int64_t)gridDim.x * 16) {
        const int64_t g = g0 + (threadIdx.x >> 4);
        int64_t r, c;
        mx4_place<FLAT>(g < total ? g : total - 1, total, runs, r, c);
        const int64_t c0 = c * 128 + sub * 8;
        float v[8];
        if (c0 + 8 <= cols) {
            if (DT == DT_F32) {
                const f32x4u *p = (const f32x4u *)((const float *)x + r * ld + c0);
                const f32x4 a = __builtin_nontemporal_load(p), b = __builtin_nontemporal_load(p + 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = a[i];
                    v[4 + i] = b[i];
                }
            } else {
                const u32x4 a = __builtin_nontemporal_load((const u32x4u *)((const uint16_t *)x + r * ld + c0));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = __uint_as_float(a[i] << 16);
                    v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t at = r * ld + c0 + i;
                v[i] = c0 + i >= cols ? 0.0f
                       : DT == DT_F32 ? ((const float *)x)[at] : bf16_to_f32(((const uint16_t *)x)[at]);
            }
        }
        // magnitudes order as their bits do, infinities and NaN above the rest
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
            amax = b > amax ? b : amax;
        }
        amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1, 64));
        amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2, 64));
        const uint32_t s = mx4_scale(amax);
        const uint32_t codes = mx4_codes(v, s);
        if (g < total) {
            ((uint32_t *)q)[g * 16 + sub] = codes;
            if ((sub & 3) == 0) sc[g * 4 + (sub >> 2)] = (uint8_t)s;
        }
    }
}

// Eight values a thread.  Bound by memory: 16384 x 7168 codes to bf16 49 us, 297 MB, 6.0 TB/s, four fifths of it
// writing, by nontemporal stores: 73 us without.
template <int DT, bool FLAT>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t *__restrict__ q,
                                                             const uint8_t *__restrict__ sc, int64_t rows, int64_t cols,
                                                             int64_t runs, void *__restrict__ y, int64_t ld) {
    const int64_t total = rows * runs;
    const int sub = threadIdx.x & 15;
    for (int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); g < total; g += (int64_t)gridDim.x * 16) {
        int64_t r, c;
        mx4_place<FLAT>(g, total, runs, r, c);
        const int64_t c0 = c * 128 + sub * 8;
        const uint32_t codes = ((const uint32_t *)q)[g * 16 + sub];
        const uint32_t s = sc[g * 4 + (sub >> 2)];
        const float unit = s == kNanScale ? __builtin_nanf("") : mx4_unit(s);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t c = codes >> (4 * k) & 15u, m = c & 7u;
            // magnitudes 0, 0.5, then (2 + m mod 2) 2^(m/2 - 2)
            const float mag = m < 2 ? 0.5f * (float)m : (float)(2 + (m & 1)) * __uint_as_float((m / 2 + 125u) << 23);
            v[k] = (c & 8u ? -mag : mag) * unit;
        }
        if (c0 + 8 <= cols) {
            if (DT == DT_F32) {
                f32x4u *p = (f32x4u *)((float *)y + r * ld + c0);
                const f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
                __builtin_nontemporal_store(lo, p);
                __builtin_nontemporal_store(hi, p + 1);
            } else {
                const u32x4 o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                 pack_bf16x2(v[6], v[7])};
                __builtin_nontemporal_store(o, (u32x4u *)((uint16_t *)y + r * ld + c0));
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (c0 + k >= cols) continue;
                if (DT == DT_F32) ((float *)y)[r * ld + c0 + k] = v[k];
                else ((uint16_t *)y)[r * ld + c0 + k] = (uint16_t)pack_bf16x2(v[k], 0.0f);
            }
        }
    }
}

// ---- experts -------------------------------------------------------------------
//
// Both kernels below multiply 32 x 64 blocks of weights with 64 x 32 blocks of tokens (32x32x64
// scaled MFMA: 7.0 PFLOP/s in chains of products on random codes, against 4.5 for 16x16x128).  A
// lane holds 32 codes of one row, which is one MX4 block with one scale.  The reduction is walked in
// segments of 256 values: 128 bytes of a row, of which lanes 0-31 hold the first 64 and lanes 32-63 the
// second, so that a row's segment is read as one line, the four products of a segment take a
// lane's four 16-byte pieces in order, and the lane's four scales are the bytes of one word, which
// the instruction picks from by itself.  (Any pairing of pieces gives the same sum, as long as
// weights and tokens use the same one.)
//
// A wave owns two blocks of weight rows: 32 gate rows and the matching 32 up rows, whose 32 values of H
// are one MX4 block, or 64 rows of the down weights.

struct Mx4Pass {
    int n_exp;
    const int32_t *offsets, *gather;
    const uint8_t *x, *xs;       // activation rows
    const uint8_t *w0, *w1;      // gate and up, or down
    const uint8_t *s0, *s1;
    int F;                       // output features
    int kruns;                   // runs of 128 along the reduction
    uint8_t *h, *hs;             // gate/up output
    int hruns;
    uint16_t *y;                 // down output [.][F]
    int yvec;                    // rows of y take 16-byte stores
};

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int STEP>
__device__ __forceinline__ f32x16 mx4_mfma(i32x4 a, i32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                           i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4, 4, STEP,
                                                           (int)sa, STEP, (int)sb);
}

// Keeps products where they are written: without it the compiler moves them behind the reads and barriers that they
// are meant to run beside.
__device__ __forceinline__ void mx4_pin(f32x16 &a) { asm volatile("" : "+v"(a)); }

// Buffer descriptors: offsets past a descriptor's bytes read as zero and are not written, so a lane
// without work takes kNoOffset.
constexpr uint32_t kNoOffset = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx4_rsrc(const uint8_t *p, int64_t bytes) {
    const uint64_t u = (uint64_t)p;
    const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(u >> 32)) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((int)u);
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, __builtin_amdgcn_readfirstlane((int)bytes),
                                             0x00020000);
}

// 16-byte piece p of row r in LDS: rows are 128 bytes, and the 16 lanes that LDS serves together (quads
// of a wave half with the same bit parity) hold each of the eight row pairs' low three bits once, which
// this permutation turns into eight different pieces.
__device__ __forceinline__ int mx4_swz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int mx4_lds(int r, int p) { return r * 128 + ((p ^ mx4_swz(r)) << 4); }

// A wave's 64 weight rows on their way to LDS, a segment at a time: eight loads of 1 KB (8 rows each, whole
// lines; lane l brings the piece that belongs in place l mod 8 of its row).  Rows past the features, and the
// half that an odd number of runs lacks, read as zeros.
//
// Scales: a row's eight bytes of a segment are a small part of a line, and every row is another line.  Where
// rows of scales are whole 16-byte pieces (WIDE: 512 values, aligned), one load brings 16 bytes a row, of two
// segments; otherwise two loads bring a segment's words, 32 rows each.  (Loading words for every segment made half
// of all requests to L2: 5.0 TB/s of weights in a copy to LDS against 6.2 without scales.)
constexpr int kMx4WeightBytes = 64 * 128;
constexpr int mx4_scale_bytes(bool wide) { return wide ? 16 : 8; }   // of a row, in one slot of scales

template <bool WIDE>
struct Mx4Weights {
    __amdgpu_buffer_rsrc_t w[2], s[2];
    uint32_t wo[8], so[2];
    bool once;
    template <bool GATEUP>
    __device__ __forceinline__ void aim(const Mx4Pass &a, int e, int ft, bool once_, int lane) {
        once = once_;
        const uint32_t wrow = (uint32_t)a.kruns * 64, srow = (uint32_t)a.kruns * 4;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int f0 = GATEUP ? ft * 32 : ft * 64 + i * 32;
            const int n = max(0, min(32, a.F - f0));       // rows of the block
            const int64_t r = (int64_t)e * a.F + min(f0, a.F - 1);
            w[i] = mx4_rsrc((GATEUP && i ? a.w1 : a.w0) + r * wrow, (int64_t)n * wrow);
            s[i] = mx4_rsrc((GATEUP && i ? a.s1 : a.s0) + r * srow, (int64_t)n * srow);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = j * 8 + (lane >> 3);
                wo[i * 4 + j] = row < n ? (uint32_t)row * wrow + (((lane & 7) ^ mx4_swz(row)) << 4) : kNoOffset;
            }
            const int row = WIDE ? lane & 31 : lane >> 1;
            so[i] = row < n ? (uint32_t)row * srow + (WIDE ? 0 : (lane & 1) * 4) : kNoOffset;
        }
    }
    // Codes of segment k.  Rows that this tile alone reads (an expert of one row block) are loaded with the
    // nontemporal policy, so that L2 keeps the tokens: 256 experts of 7168 x 2048, 4 rows each, 928 us against 999.
    __device__ __forceinline__ void load(const Mx4Pass &a, int k, char *dst, int lane) const {
        const bool tail = 2 * k + 1 == a.kruns;
        auto each = [&](auto once) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const bool none = tail && (((lane & 7) ^ mx4_swz((q & 3) * 8 + (lane >> 3))) & 4);
                if (decltype(once)::value) buffer_dma16_stream(w[q >> 2], none ? kNoOffset : wo[q], k * 128, dst + q * 1024);
                else buffer_dma16(w[q >> 2], none ? kNoOffset : wo[q], k * 128, dst + q * 1024);
            }
        };
        if (once) each(std::true_type{});
        else each(std::false_type{});
    }
    // scales of segment k, or (WIDE) of segments k and k + 1; two loads
    __device__ __forceinline__ void load_scales(const Mx4Pass &a, int k, char *dst, int lane) const {
        const bool tail = 2 * k + 1 == a.kruns;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (!WIDE) buffer_dma4(s[i], tail && (lane & 1) ? kNoOffset : so[i], k * 8, dst + i * 256);
            else if (lane < 32) buffer_dma16(s[i], so[i], k * 8, dst + i * 512);
        }
    }
};

// Where a tile's results go: descriptors based at its first row.
struct Mx4Out {
    __amdgpu_buffer_rsrc_t o, s;
};

template <bool GATEUP>
__device__ __forceinline__ Mx4Out mx4_out(const Mx4Pass &a, int64_t row0, int rows) {
    const uint32_t hrow = (uint32_t)a.hruns * 64;
    Mx4Out O;
    if (GATEUP) {
        O.o = mx4_rsrc(a.h + row0 * hrow, (int64_t)rows * hrow);
        O.s = mx4_rsrc(a.hs + row0 * (hrow >> 4), (int64_t)rows * (hrow >> 4));
    } else {
        O.o = mx4_rsrc((const uint8_t *)(a.y + row0 * a.F), (int64_t)rows * a.F * 2);
        O.s = O.o;
    }
    return O;
}

// g / (1 + exp(-g)), each operation rounded to fp32, so that a code of H is the one the formula gives in fp32: an
// exponential by one rounded product with log2(e) errs by up to 2^-23 |g|, which moved one code in some 10^7 (and next
// to a middle of two codes, g from -85 to 20, one in eight).  exp(x) = 2^n 2^f, n whole and |f| <= 1/2, with f's
// argument in two parts: within 0.87 ulp (tried against 64 bits at every float from -87 to 87).  Against the one product
// it costs 0.5 to 1 % of a call's time, 4 % at 24 experts of 1000 x 360 (25.6 us).
__device__ __forceinline__ float mx4_silu(float g) {
#pragma clang fp contract(off)
    constexpr float kLog2e = 0x1.715476p+0f, kLog2eTail = 0x1.4ae0bfp-26f;
    const float x = __builtin_amdgcn_fmed3f(-g, -200.0f, 200.0f);   // past either end the result is 0 or infinity
    const float p = x * kLog2e, n = __builtin_rintf(p);
    const float f = (p - n) + __builtin_fmaf(x, kLog2eTail, __builtin_fmaf(x, kLog2e, -p));
    return g / (1.0f + __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n));
}

// Results of 32 tokens from row r of the tile on: lane l holds, of token l & 31, features
// 8 q + 4 (l >> 5) + 0..3 (q = 0..3) of each of its two blocks.  Rows past the tile's lie past the
// descriptor and are not written.
template <bool GATEUP>
__device__ __forceinline__ void mx4_store(const Mx4Pass &a, const Mx4Out &O, const f32x16 &p, const f32x16 &u, int ft,
                                          int r, int lane) {
    const int half = lane >> 5;
    if (GATEUP) {
        float h[16];
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = mx4_silu(p[i]) * u[i];
            h[i] = ft * 32 + 8 * (i >> 2) + 4 * half + (i & 3) < a.F ? v : 0.0f;
            amax = max(amax, __float_as_uint(h[i]) & 0x7FFFFFFFu);
        }
        const auto other = __builtin_amdgcn_permlane32_swap(amax, amax, false, false);
        const uint32_t s = mx4_scale(max(other[0], other[1]));
        const float lo[8] = {h[0], h[1], h[2], h[3], h[4], h[5], h[6], h[7]};
        const float hi[8] = {h[8], h[9], h[10], h[11], h[12], h[13], h[14], h[15]};
        const uint32_t c0 = mx4_codes(lo, s), c1 = mx4_codes(hi, s);   // 16 bits for each q
        // the token's 16 bytes in the first lane: its own 16 bits below the other lane's
        const auto e0 = __builtin_amdgcn_permlane32_swap(c0, c0, false, false);
        const auto e1 = __builtin_amdgcn_permlane32_swap(c1, c1, false, false);
        const uint32_t a0 = e0[0], b0 = e0[1], a1 = e1[0], b1 = e1[1];
        const u32x4 o = {(a0 & 0xFFFFu) | b0 << 16, a0 >> 16 | (b0 & 0xFFFF0000u), (a1 & 0xFFFFu) | b1 << 16,
                         a1 >> 16 | (b1 & 0xFFFF0000u)};
        const uint32_t hrow = (uint32_t)a.hruns * 64;
        __builtin_amdgcn_raw_buffer_store_b128(o, O.o, half ? kNoOffset : (uint32_t)r * hrow + ft * 16, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b8((uint8_t)s, O.s, half ? kNoOffset : (uint32_t)r * (hrow >> 4) + ft, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x16 &v = i ? u : p;
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
                // groups q and q + 1 of eight features: the first lane takes group q whole, the second q + 1
                const uint32_t a0 = pack_bf16x2(v[4 * q], v[4 * q + 1]), a1 = pack_bf16x2(v[4 * q + 2], v[4 * q + 3]);
                const uint32_t b0 = pack_bf16x2(v[4 * q + 4], v[4 * q + 5]),
                               b1 = pack_bf16x2(v[4 * q + 6], v[4 * q + 7]);
                const auto x0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
                const auto x1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
                const u32x4 o = {x0[0], x1[0], x0[1], x1[1]};
                const int f = ft * 64 + i * 32 + 8 * (q + half);
                const uint32_t at = ((uint32_t)r * a.F + f) * 2;
                if (a.yvec) {
                    __builtin_amdgcn_raw_buffer_store_b128(o, O.o, f < a.F ? at : kNoOffset, 0, 0);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(o[k >> 1] >> (16 * (k & 1))), O.o,
                                                              f + k < a.F ? at + 2 * k : kNoOffset, 0, 0);
                }
            }
        }
    }
}

constexpr int kMx4Threads = 256;
constexpr int kMx4Waves = kMx4Threads / 64;

// The experts' ends in LDS, by the whole workgroup.
__device__ __forceinline__ void mx4_ends(const Mx4Pass &a, int32_t *o) {
    for (int i = threadIdx.x; i < a.n_exp; i += blockDim.x) o[i] = a.offsets[i + 1];
    __syncthreads();
}
constexpr int kMx4EndBytes = kMaxExperts * 4;

// Few tiles: bound by the time from one load to the next in each wave, so the work is cut finely.  A wave takes tiles
// of 64 weight rows and up to 32 tokens by itself; weights and tokens pass through a ring of segments in LDS that is
// the wave's own, filled by direct loads and emptied without a barrier, across the ends of tiles.  SPLIT: the four
// waves of a workgroup share a tile, each a quarter of the segments, and add up in LDS, in the order of the waves,
// which leaves room for 16 tokens.  One token, 8 experts of 7168 x 2048: gate/up 25 us, down 14 us (187 MB of
// weights at 4.8 TB/s).
constexpr int mx4_stream_tokens(bool split) { return mx4_tokens(split ? kMx4Shared : kMx4Stream); }
constexpr int mx4_slot_bytes(bool split) { return kMx4WeightBytes + mx4_stream_tokens(split) * 128; }
constexpr int kMx4ScaleSlot = (64 + 32) * 16;            // of two segments (WIDE); three of 8 bytes a row fit as well
constexpr int kMx4PartBytes = (kMx4Waves - 1) * 8 * 64 * 16;
constexpr int kMx4Slots = 3;
constexpr int mx4_wave_lds(bool split) { return kMx4Slots * mx4_slot_bytes(split) + 2 * kMx4ScaleSlot; }
constexpr int mx4_stream_lds(bool split) {
    return kMx4EndBytes + kMx4Waves * mx4_wave_lds(split) + (split ? kMx4PartBytes : 0);
}
static_assert(mx4_stream_lds(false) <= 160 * 1024 && mx4_stream_lds(true) <= 160 * 1024, "LDS");

template <bool GATEUP, bool SPLIT, bool WIDE>
__global__ __launch_bounds__(kMx4Threads, 1) void mx4_stream_kernel(const Mx4Pass a) {
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, r31 = lane & 31;
    constexpr int SLOTS = kMx4Slots, SLOT = mx4_slot_bytes(SPLIT), SB = mx4_scale_bytes(WIDE);
    constexpr int TOKENS = mx4_stream_tokens(SPLIT);
    char *ring = smem + kMx4EndBytes + wid * mx4_wave_lds(SPLIT), *scales = ring + SLOTS * SLOT;
    f32x4 *part = (f32x4 *)(smem + kMx4EndBytes + kMx4Waves * mx4_wave_lds(SPLIT));
    mx4_ends(a, (int32_t *)smem);
    // gate/up tiles also cover the padding up to whole runs, which is written as zeros
    const int ftiles = GATEUP ? a.hruns * 4 : (a.F + 63) / 64;
    TileList list;
    list.init((const int32_t *)smem, a.n_exp, TOKENS, ftiles, lane);
    const int segs = (a.kruns + 1) / 2;   // with an odd number of runs the last one has no second half
    // the wave's share of a tile's segments, in pairs where scales come for two
    constexpr int PAIR = WIDE ? 2 : 1;
    const int k0 = SPLIT ? segs / PAIR * wid / kMx4Waves * PAIR : 0;
    const int k1 = SPLIT ? segs / PAIR * (wid + 1) / kMx4Waves * PAIR : segs;
    const int step = SPLIT ? gridDim.x : gridDim.x * kMx4Waves;
    const int first = SPLIT ? blockIdx.x : blockIdx.x * kMx4Waves + wid;

    // the tile and segment whose loads are issued next
    Mx4Weights<WIDE> W;
    const uint8_t *xp[TOKENS / 8], *xsp;
    int it = first, ik = k0, nx = 0, is = 0;
    auto next_tile = [&]() {
        int e, ft, row0, valid;
        list.find(it, lane, e, ft, row0, valid);
        W.template aim<GATEUP>(a, e, ft, list.blocks(e) == 1, lane);
        // token rows past the tile's repeat its last one; their results are not used
        auto token = [&](int r) {
            const int64_t R = row0 + min(r, valid - 1);
            return a.gather ? (int64_t)a.gather[R] : R;
        };
#pragma unroll
        for (int j = 0; j < TOKENS / 8; ++j) xp[j] = a.x + token(j * 8 + (lane >> 3)) * ((int64_t)a.kruns * 64);
        xsp = a.xs + token(WIDE ? lane & 31 : lane >> 1) * ((int64_t)a.kruns * 4) + (WIDE ? 0 : (lane & 1) * 4);
        nx = (valid + 7) >> 3;
    };
    // slots of scales: one for each segment, in turn, or one for two
    auto scale_slot = [&](int s) { return scales + s * (96 * SB); };
    auto after = [&](int s) { return s + 1 == (WIDE ? 2 : SLOTS) ? 0 : s + 1; };
    // issues the next segment into a slot; the number of loads
    auto issue = [&](int slot) {
        if (it >= list.total || k0 >= k1) return 0;
        if (ik == k0) next_tile();
        char *dst = ring + slot * SLOT, *xd = dst + kMx4WeightBytes;
        const bool tail = 2 * ik + 1 == a.kruns;
        int n = 8 + nx;
        if (!WIDE || !(ik & 1)) {
            char *sd = scale_slot(is);
            is = after(is);
            W.load_scales(a, ik, sd, lane);
            if (!WIDE) dma4(xsp + (int64_t)ik * 8 - (tail && (lane & 1) ? 4 : 0), sd + 64 * SB);
            else if (lane < 32) dma16(xsp + (int64_t)ik * 8, sd + 64 * SB);
            n += 3;
        }
        W.load(a, ik, dst, lane);
#pragma unroll
        for (int j = 0; j < TOKENS / 8; ++j) {
            // the half that an odd number of runs lacks meets weights of zero: it repeats the other
            const int p = (lane & 7) ^ mx4_swz(j * 8 + (lane >> 3));
            if (j < nx) dma16(xp[j] + (int64_t)ik * 128 + (tail ? p & 3 : p) * 16, xd + j * 1024);
        }
        if (++ik == k1) {
            ik = k0;
            it += step;
        }
        return n;
    };
    // loads of the last segments issued
    issue(0);
    int n1 = issue(1), n2 = issue(2);
    const int column = r31 & (TOKENS - 1);    // further columns of the products repeat the tokens and are not used
    int slot = 0, ss = 0;
    for (int t = first; t < list.total; t += step) {
        f32x16 acc[2] = {};
        for (int k = k0; k < k1; ++k) {
            // the segment's own loads are done once only the later segments' are outstanding
            wait_vmcnt_dyn(n1 + n2);
            asm volatile("" ::: "memory");
            const char *src = ring + slot * SLOT, *xsrc = src + kMx4WeightBytes;
            const char *sc = scale_slot(ss) + (WIDE && (k & 1) ? 8 : 0) + half * 4;
            if (!WIDE || (k & 1)) ss = after(ss);
            i32x4 w[2][4], x[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                w[0][c] = *(const i32x4 *)(src + mx4_lds(r31, half * 4 + c));
                w[1][c] = *(const i32x4 *)(src + 4096 + mx4_lds(r31, half * 4 + c));
                x[c] = *(const i32x4 *)(xsrc + mx4_lds(column, half * 4 + c));
            }
            const uint32_t ws0 = *(const uint32_t *)(sc + r31 * SB), ws1 = *(const uint32_t *)(sc + (32 + r31) * SB);
            const uint32_t xs = *(const uint32_t *)(sc + (64 + column) * SB);
            wait_lgkm0();                  // the slot has been read: it can be filled again
            asm volatile("" ::: "memory");
            const int n = issue(slot);
            n1 = n2;
            n2 = n;
            acc[0] = mx4_mfma<0>(w[0][0], x[0], acc[0], ws0, xs);
            acc[1] = mx4_mfma<0>(w[1][0], x[0], acc[1], ws1, xs);
            acc[0] = mx4_mfma<1>(w[0][1], x[1], acc[0], ws0, xs);
            acc[1] = mx4_mfma<1>(w[1][1], x[1], acc[1], ws1, xs);
            acc[0] = mx4_mfma<2>(w[0][2], x[2], acc[0], ws0, xs);
            acc[1] = mx4_mfma<2>(w[1][2], x[2], acc[1], ws1, xs);
            acc[0] = mx4_mfma<3>(w[0][3], x[3], acc[0], ws0, xs);
            acc[1] = mx4_mfma<3>(w[1][3], x[3], acc[1], ws1, xs);
            slot = slot == SLOTS - 1 ? 0 : slot + 1;
        }
        if (SPLIT) {
            cta_barrier();   // the previous tile's sums have been read
            if (wid > 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        part[((wid - 1) * 8 + i * 4 + q) * 64 + lane] =
                            f32x4{acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]};
            }
            wait_lgkm0();
            cta_barrier();
            if (wid > 0) continue;
#pragma unroll 1
            for (int o = 0; o < kMx4Waves - 1; ++o)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 v = part[(o * 8 + i * 4 + q) * 64 + lane];
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[i][4 * q + k] += v[k];
                    }
        }
        int e, ft, row0, valid;
        list.find(t, lane, e, ft, row0, valid);
        mx4_store<GATEUP>(a, mx4_out<GATEUP>(a, row0, valid), acc[0], acc[1], ft, r31, lane);
    }
}

// Many tiles.  A workgroup's tile is 256 weight rows against up to CAP blocks of 32 tokens.  Four waves, one a
// SIMD, multiply (64 weight rows each, all tokens); four others, one a SIMD too, only bring segments into rings in
// LDS, across the ends of tiles, so that no product waits behind a load that finds the memory pipeline full.  One
// barrier a segment: passing it, a segment's loads are done and the places of the segment before have been read.
// CAP 4 leaves room for three segments of weights and of tokens.  CAP 5 leaves room for two of tokens, which come from L2
// and arrive in time beside weights from memory; it is for experts of about 128 rows, most of which then need
// one tile and read their weights once.
//
// 256 experts of 7168 x 2048: at 4 rows each bound by the stream of weights (5.85 GB in 894 us, 6.5 TB/s), at 128 rows by
// the stream and the products together (gate/up 940 us, down 490), neither of which the other's waits fill whole.
// 32 experts, 512 rows: products (gate/up 360 us, 2.7 of 6.7 PFLOP/s), the loads from L2 into LDS that feed them (8 of
// 16 TB/s) and the epilogue, which the multiplying waves do not overlap.
//
// Two waves a SIMD have 256 registers each.  Gate/up of 160 tokens takes all of them and keeps three values in
// scratch, read back once a tile; the loading waves, which have as many, need a few dozen.
constexpr int kMx4TileThreads = 512;
constexpr int kMx4WeightStages = 3;
constexpr int mx4_token_stages(int cap) { return cap <= 4 ? 3 : 2; }
// a slot of scales holds 16 bytes a row, of two segments (WIDE), of two slots; three of 8 bytes a row fit as well
constexpr int mx4_tile_lds(int cap) {
    return kMx4EndBytes + kMx4WeightStages * 4 * kMx4WeightBytes + mx4_token_stages(cap) * cap * 4096 +
           2 * (256 + cap * 32) * 16;
}
static_assert(mx4_tile_lds(4) <= 160 * 1024 && mx4_tile_lds(5) <= 160 * 1024, "LDS");
// the parts of LDS behind the experts' ends: weights, tokens, scales of weights, scales of tokens
template <int CAP>
struct Mx4TileParts {
    char *w, *x, *ws, *xs;
    __device__ explicit Mx4TileParts(char *smem) {
        w = smem + kMx4EndBytes;
        x = w + kMx4WeightStages * 4 * kMx4WeightBytes;
        ws = x + mx4_token_stages(CAP) * CAP * 4096;
        xs = ws + 2 * 256 * 16;
    }
};

// The loading waves; wave p brings weight rows 64 p + 0..63, token rows 8 (4 j + p) + 0..7 and the scales of token
// rows 32 p + 0..31 (wave 0 also of 128 + 0..31).
template <bool GATEUP, bool WIDE, int CAP>
__device__ __forceinline__ void mx4_tile_load(const Mx4Pass &a, const TileList &list, const Mx4TileParts<CAP> &lds,
                                              int first, int end, int step, int segs, int p, int lane) {
    constexpr int SB = mx4_scale_bytes(WIDE), XSTAGES = mx4_token_stages(CAP), SSLOTS = WIDE ? 2 : 3;
    // weights: the tile and segment that come next; places are taken in turn
    Mx4Weights<WIDE> W;
    int wt = first, wk = 0, wplace = 0, wsplace = 0;
    auto weights = [&]() {
        if (wt >= end) return 0;
        if (wk == 0) {
            int e, ft, row0, valid;
            list.find(wt, lane, e, ft, row0, valid);
            W.template aim<GATEUP>(a, e, ft * 4 + p, list.blocks(e) == 1, lane);
        }
        int n = 8;
        if (!WIDE || !(wk & 1)) {
            W.load_scales(a, wk, lds.ws + wsplace * (256 * SB) + p * (64 * SB), lane);
            wsplace = wsplace + 1 == SSLOTS ? 0 : wsplace + 1;
            n += 2;
        }
        W.load(a, wk, lds.w + (wplace * 4 + p) * kMx4WeightBytes, lane);
        wplace = wplace + 1 == kMx4WeightStages ? 0 : wplace + 1;
        if (++wk == segs) {
            wk = 0;
            wt += step;
        }
        return n;
    };
    // tokens
    const uint8_t *xp[CAP], *xsp[2];
    int xt = first, xk = 0, xplace = 0, xsplace = 0, tb = 0;
    auto tokens = [&]() {
        if (xt >= end) return 0;
        if (xk == 0) {
            int e, ft, row0, valid;
            list.find(xt, lane, e, ft, row0, valid);
            // token row r of the tile; rows past the tile's repeat its last one, their results are not used
            auto token = [&](int r) {
                const int64_t R = row0 + min(r, valid - 1);
                return a.gather ? (int64_t)a.gather[R] : R;
            };
#pragma unroll
            for (int j = 0; j < CAP; ++j) xp[j] = a.x + token((j * 4 + p) * 8 + (lane >> 3)) * ((int64_t)a.kruns * 64);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                xsp[j] = a.xs + token((j * 4 + p) * 32 + (WIDE ? lane & 31 : lane >> 1)) * ((int64_t)a.kruns * 4) +
                         (WIDE ? 0 : (lane & 1) * 4);
            tb = (valid + 31) >> 5;
        }
        const bool tail = 2 * xk + 1 == a.kruns;
        int n = tb;
        if (!WIDE || !(xk & 1)) {
            char *sd = lds.xs + xsplace * (CAP * 32 * SB);
            xsplace = xsplace + 1 == SSLOTS ? 0 : xsplace + 1;
#pragma unroll
            for (int j = 0; j < (CAP > 4 ? 2 : 1); ++j)
                if (j * 4 + p < tb) {
                    char *d = sd + (j * 4 + p) * (32 * SB);
                    if (!WIDE) dma4(xsp[j] + (int64_t)xk * 8 - (tail && (lane & 1) ? 4 : 0), d);
                    else if (lane < 32) dma16(xsp[j] + (int64_t)xk * 8, d);
                    ++n;
                }
        }
        char *xd = lds.x + xplace * (CAP * 4096);
        xplace = xplace + 1 == XSTAGES ? 0 : xplace + 1;
#pragma unroll
        for (int j = 0; j < CAP; ++j) {
            // the half that an odd number of runs lacks meets weights of zero: it repeats the other
            const int c = (lane & 7) ^ mx4_swz((j * 4 + p) * 8 + (lane >> 3));
            if (j < tb) dma16(xp[j] + (int64_t)xk * 128 + (tail ? c & 3 : c) * 16, xd + (j * 4 + p) * 1024);
        }
        if (++xk == segs) {
            xk = 0;
            xt += step;
        }
        return n;
    };
    static_assert(kMx4WeightStages == 3 && (XSTAGES == 2 || XSTAGES == 3), "order of the loads");
    // before the barrier of segment i the loads of segment i have to be done: only later ones may be outstanding,
    // those of the weights of i + 1 and, with three stages of tokens, of its tokens
    tokens();
    weights();
    int later = XSTAGES == 3 ? tokens() : 0;
    later += weights();
    for (int u = first; u < end; u += step)
        for (int i = 0; i < segs; ++i) {
            wait_vmcnt_dyn(later);
            cta_barrier();
            if (XSTAGES == 3) {
                later = weights();
                later += tokens();
            } else {
                tokens();
                later = weights();
            }
        }
    cta_barrier();   // the multiplying waves pass one behind every segment
}

template <bool GATEUP, bool WIDE, int CAP>
__global__ __launch_bounds__(kMx4TileThreads, 1) void mx4_tile_kernel(const Mx4Pass a) {
    extern __shared__ __align__(16) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Mx4TileParts<CAP> lds(smem);
    mx4_ends(a, (int32_t *)smem);
    const int wtiles = GATEUP ? a.hruns * 4 : (a.F + 63) / 64;
    TileList list;
    list.init((const int32_t *)smem, a.n_exp, CAP * 32, (wtiles + 3) / 4, lane);
    const int segs = (a.kruns + 1) / 2;   // with an odd number of runs the last one has no second half
    // workgroup b runs on XCD b mod 8: each XCD takes a contiguous eighth of the list, so that the row
    // blocks of a weight tile and the weight tiles of a row block meet in its L2
    const int per = (list.total + 7) / 8, xcd = blockIdx.x & 7;
    const int end = min(list.total, (xcd + 1) * per), first = xcd * per + (blockIdx.x >> 3), step = gridDim.x >> 3;
    if (first >= end) return;
    if (wid >= 4) {
        mx4_tile_load<GATEUP, WIDE, CAP>(a, list, lds, first, end, step, segs, wid - 4, lane);
        return;
    }

    const int half = lane >> 5, r31 = lane & 31;
    constexpr int SB = mx4_scale_bytes(WIDE), XSTAGES = mx4_token_stages(CAP);
    int slot = 0, xslot = 0, ss = 0, odd = 0, t = first;
    cta_barrier();                        // the first segment is there
    auto tile = [&](auto tbc, int ft, int row0, int valid) {
        constexpr int TB = decltype(tbc)::value;
        f32x16 acc[2][TB] = {};
        i32x4 w[2][2], b[2][TB];
        uint32_t us[2], vs[TB];
        auto read = [&](int g, int c) {
            const char *ws = lds.w + (slot * 4 + wid) * kMx4WeightBytes, *xb = lds.x + xslot * (CAP * 4096);
#pragma unroll
            for (int i = 0; i < 2; ++i) w[g][i] = *(const i32x4 *)(ws + i * 4096 + mx4_lds(r31, half * 4 + c));
#pragma unroll
            for (int j = 0; j < TB; ++j) b[g][j] = *(const i32x4 *)(xb + mx4_lds(j * 32 + r31, half * 4 + c));
        };
        auto read_scales = [&]() {
            const int at = (WIDE ? odd * 8 : 0) + half * 4;
            const char *ws = lds.ws + ss * (256 * SB) + at, *xs = lds.xs + ss * (CAP * 32 * SB) + at;
#pragma unroll
            for (int i = 0; i < 2; ++i) us[i] = *(const uint32_t *)(ws + (wid * 64 + i * 32 + r31) * SB);
#pragma unroll
            for (int j = 0; j < TB; ++j) vs[j] = *(const uint32_t *)(xs + (j * 32 + r31) * SB);
        };
        auto next_scales = [&]() {
            if (!WIDE || odd) ss = ss + 1 == (WIDE ? 2 : 3) ? 0 : ss + 1;
            odd ^= 1;
            read_scales();
        };
        read_scales();
        read(0, 0);
        for (int k = 0; k < segs; ++k) {
            const uint32_t u0 = us[0], u1 = us[1];
            uint32_t v[TB];
#pragma unroll
            for (int j = 0; j < TB; ++j) v[j] = vs[j];
            auto multiply = [&](auto sc) {
                constexpr int C = decltype(sc)::value;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    acc[0][j] = mx4_mfma<C>(w[C & 1][0], b[C & 1][j], acc[0][j], u0, v[j]);
                    acc[1][j] = mx4_mfma<C>(w[C & 1][1], b[C & 1][j], acc[1][j], u1, v[j]);
                    mx4_pin(acc[0][j]);
                    mx4_pin(acc[1][j]);
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            read(1, 1);
            multiply(std::integral_constant<int, 0>{});
            read(0, 2);
            multiply(std::integral_constant<int, 1>{});
            read(1, 3);
            multiply(std::integral_constant<int, 2>{});
            // the stage has been read; the next segment's first operands come in behind the last products (after a
            // tile's last segment they are not used)
            wait_lgkm0();
            cta_barrier();
            slot = slot == kMx4WeightStages - 1 ? 0 : slot + 1;
            xslot = xslot == XSTAGES - 1 ? 0 : xslot + 1;
            next_scales();
            read(0, 0);
            multiply(std::integral_constant<int, 3>{});
        }
        const int wt = ft * 4 + wid;
        if (wt < wtiles) {
            const Mx4Out out = mx4_out<GATEUP>(a, row0, valid);
#pragma unroll
            for (int j = 0; j < TB; ++j) mx4_store<GATEUP>(a, out, acc[0][j], acc[1][j], wt, j * 32 + r31, lane);
        }
    };
    for (; t < end; t += step) {
        int e, ft, row0, valid;
        list.find(t, lane, e, ft, row0, valid);
        if (valid <= 32) tile(std::integral_constant<int, 1>{}, ft, row0, valid);
        else if (valid <= 64) tile(std::integral_constant<int, 2>{}, ft, row0, valid);
        else if (valid <= 96) tile(std::integral_constant<int, 3>{}, ft, row0, valid);
        else if (CAP == 4 || valid <= 128) tile(std::integral_constant<int, 4>{}, ft, row0, valid);
        else tile(std::integral_constant<int, CAP>{}, ft, row0, valid);
    }
}

template <void (*KERNEL)(Mx4Pass)>
hipError_t mx4_launch(unsigned grid, int threads, int lds, const Mx4Pass &p, hipStream_t s) {
    static std::once_flag once;
    static hipError_t attr = hipSuccess;
    std::call_once(once, [&] {
        attr = hipFuncSetAttribute((const void *)KERNEL, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    });
    if (attr != hipSuccess) return attr;
    KERNEL<<<grid, threads, lds, s>>>(p);
    return hipGetLastError();
}

}  // namespace

// f(data type, whether the matrix is one row) and the shape for it.
template <class F>
static hipError_t mx4_rows_of(int dt, int64_t ld, int64_t rows, int64_t cols, F f) {
    using std::integral_constant;
    const bool flat = ld == cols && cols % 128 == 0;
    if (flat) {
        cols *= rows;
        rows = 1;
    }
    const int64_t runs = mx4_runs(cols), wgs = (rows * runs + 15) / 16;
    const unsigned grid = (unsigned)(wgs < 16384 ? wgs : 16384);
    auto with = [&](auto dtc) {
        if (flat) return f(dtc, std::true_type{}, grid, rows, cols, runs);
        return f(dtc, std::false_type{}, grid, rows, cols, runs);
    };
    return dt == DT_F32 ? with(integral_constant<int, DT_F32>{}) : with(integral_constant<int, DT_BF16>{});
}

hipError_t launch_mx4_quantize(int dt, const void *x, int64_t ld, int64_t rows, int cols, uint8_t *q, uint8_t *sc,
                               hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    return mx4_rows_of(dt, ld, rows, cols, [&](auto d, auto f, unsigned grid, int64_t rows, int64_t cols, int64_t runs) {
        mx4_quantize_kernel<decltype(d)::value, decltype(f)::value>
            <<<grid, 256, 0, s>>>(x, ld, rows, cols, runs, q, sc);
        return hipGetLastError();
    });
}

hipError_t launch_mx4_dequantize(int dt, const uint8_t *q, const uint8_t *sc, int64_t rows, int cols, void *y,
                                 int64_t ld, hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    return mx4_rows_of(dt, ld, rows, cols, [&](auto d, auto f, unsigned grid, int64_t rows, int64_t cols, int64_t runs) {
        mx4_dequantize_kernel<decltype(d)::value, decltype(f)::value>
            <<<grid, 256, 0, s>>>(q, sc, rows, cols, runs, y, ld);
        return hipGetLastError();
    });
}

hipError_t launch_mx4_ffn(const Mx4Ffn &a, hipStream_t s) {
    if (a.max_rows <= 0) return hipSuccess;
    Mx4Pass up{}, down{};
    up.n_exp = down.n_exp = a.n_exp;
    up.offsets = down.offsets = a.offsets;
    up.gather = a.gather;
    up.x = a.x;
    up.xs = a.xs;
    up.w0 = a.w[0];
    up.w1 = a.w[1];
    up.s0 = a.ws[0];
    up.s1 = a.ws[1];
    up.F = a.inter;
    up.kruns = (int)mx4_runs(a.d);
    up.h = a.h;
    up.hs = a.hs;
    up.hruns = (int)mx4_runs(a.inter);
    down.x = a.h;
    down.xs = a.hs;
    down.w0 = a.w[2];
    down.s0 = a.ws[2];
    down.F = a.d;
    down.kruns = up.hruns;
    down.y = a.y;
    down.yvec = (uintptr_t)a.y % 16 == 0 && a.d % 8 == 0;
    const int64_t cus = device_cus();
    const unsigned grid = (unsigned)((cus + 7) / 8 * 8);
    auto pass = [&](auto gateup, auto wide, const Mx4Pass &p, int64_t ftiles) {
        constexpr bool GU = decltype(gateup)::value, W = decltype(wide)::value;
        switch (mx4_variant(a.max_rows, a.n_exp, p.kruns, ftiles, cus)) {
            case kMx4Shared:
                return mx4_launch<mx4_stream_kernel<GU, true, W>>(grid, kMx4Threads, mx4_stream_lds(true), p, s);
            case kMx4Stream:
                return mx4_launch<mx4_stream_kernel<GU, false, W>>(grid, kMx4Threads, mx4_stream_lds(false), p, s);
            case kMx4Tile160:
                return mx4_launch<mx4_tile_kernel<GU, W, 5>>(grid, kMx4TileThreads, mx4_tile_lds(5), p, s);
            default:
                return mx4_launch<mx4_tile_kernel<GU, W, 4>>(grid, kMx4TileThreads, mx4_tile_lds(4), p, s);
        }
    };
    auto either = [&](auto gateup, const Mx4Pass &p, int64_t tiles) {
        const uintptr_t all = (uintptr_t)p.xs | (uintptr_t)p.s0 | (uintptr_t)p.s1;
        return p.kruns % 4 == 0 && all % 16 == 0 ? pass(gateup, std::true_type{}, p, tiles)
                                                 : pass(gateup, std::false_type{}, p, tiles);
    };
    const hipError_t e = either(std::true_type{}, up, up.hruns * 4);
    return e != hipSuccess ? e : either(std::false_type{}, down, (a.d + 63) / 64);
}

}  // namespace moe
