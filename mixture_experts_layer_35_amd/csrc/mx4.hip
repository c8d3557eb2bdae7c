// mx4.hip -- microscaled 4-bit floating point (OCP Microscaling Formats v1.0: E2M1 codes,
// one E8M0 scale for 32 values): rounding, its inverse, and the SwiGLU experts on MX4
// weights and activations.
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "lds_ring.h"

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

// 16 lanes per run of 128 values, eight values a lane, four lanes a block.
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const void *__restrict__ x, int64_t ld, int64_t rows,
                                                           int cols, int runs, uint8_t *__restrict__ q,
                                                           uint8_t *__restrict__ sc) {
    const int64_t total = rows * runs;
    const int sub = threadIdx.x & 15;
    // the loop bound is uniform over the workgroup, so every lane reaches the lane exchanges
    for (int64_t g0 = (int64_t)blockIdx.x * 16; g0 < total; g0 += (int64_t)gridDim.x * 16) {
        const int64_t g = g0 + (threadIdx.x >> 4);
        const int64_t gg = g < total ? g : total - 1;
        const int64_t r = gg / runs;
        const int c0 = (int)(gg - r * runs) * 128 + sub * 8;
        float v[8];
        if (VEC && c0 + 8 <= cols) {
            if (DT == DT_F32) {
                const f32x4 *p = (const f32x4 *)((const float *)x + r * ld + c0);
                const f32x4 a = p[0], b = p[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = a[i];
                    v[4 + i] = b[i];
                }
            } else {
                const u32x4 a = *(const u32x4 *)((const uint16_t *)x + r * ld + c0);
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

// Eight values a thread.
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t *__restrict__ q,
                                                             const uint8_t *__restrict__ sc, int64_t rows, int cols,
                                                             int runs, void *__restrict__ y, int64_t ld) {
    const int64_t total = rows * runs * 16;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / (runs * 16);
        const int c0 = (int)(i - r * (runs * 16)) * 8;
        const uint32_t codes = ((const uint32_t *)q)[i];
        const uint32_t s = sc[i >> 2];
        const float unit = s == kNanScale ? __builtin_nanf("") : mx4_unit(s);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t c = codes >> (4 * k) & 15u, m = c & 7u;
            // magnitudes 0, 0.5, then (2 + m mod 2) 2^(m/2 - 2)
            const float mag = m < 2 ? 0.5f * (float)m : (float)(2 + (m & 1)) * __uint_as_float((m / 2 + 125u) << 23);
            v[k] = (c & 8u ? -mag : mag) * unit;
        }
        if (VEC && c0 + 8 <= cols) {
            if (DT == DT_F32) {
                f32x4 *p = (f32x4 *)((float *)y + r * ld + c0);
                p[0] = f32x4{v[0], v[1], v[2], v[3]};
                p[1] = f32x4{v[4], v[5], v[6], v[7]};
            } else {
                *(u32x4 *)((uint16_t *)y + r * ld + c0) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
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

// The list of tiles: experts in order, an expert's feature tiles, a feature tile's row blocks.  Every
// wave works with it by itself: lane l adds up the tiles of experts l*P .. l*P + P-1.
struct TileList {
    const int32_t *offsets;
    int P, bm, ftiles;
    int base, count;             // this lane's first tile and tiles
    int total;
    __device__ void init(const int32_t *o, int n, int bm_, int ftiles_, int lane) {
        offsets = o;
        bm = bm_;
        ftiles = ftiles_;
        P = (n + 63) / 64;
        count = 0;
        for (int e = lane * P; e < min(n, lane * P + P); ++e) count += blocks(e) * ftiles;
        int run = count;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int up = __shfl_up(run, m, 64);
            if (lane >= m) run += up;
        }
        base = run - count;
        total = __builtin_amdgcn_readlane(run, 63);
    }
    __device__ int blocks(int e) const { return (offsets[e + 1] - offsets[e] + bm - 1) / bm; }
    // Tile t < total (the same in all lanes): expert, feature tile, first row and number of rows.  An
    // expert's rows are split evenly over its blocks.
    __device__ void find(int t, int lane, int &e, int &ft, int64_t &row0, int &valid) const {
        const uint64_t started = __ballot(count > 0 && base <= t);
        const int owner = 63 - __builtin_clzll(started);
        int le = 0, rest = t - base;
        if (lane == owner) {
            le = lane * P;
            for (int k = blocks(le) * ftiles; rest >= k; k = blocks(le) * ftiles) {
                rest -= k;
                ++le;
            }
        }
        e = __builtin_amdgcn_readlane(le, owner);
        rest = __builtin_amdgcn_readlane(rest, owner);
        const int first = __builtin_amdgcn_readfirstlane(offsets[e]);
        const int m = __builtin_amdgcn_readfirstlane(offsets[e + 1]) - first;
        const int mt = (m + bm - 1) / bm;
        // quotients are vector instructions: back to scalars, which the descriptors have to be
        ft = __builtin_amdgcn_readfirstlane(rest / mt);
        const int block = rest - ft * mt, mq = __builtin_amdgcn_readfirstlane(m / mt), mr = m - mq * mt;
        row0 = (int64_t)first + block * mq + min(block, mr);
        valid = mq + (block < mr ? 1 : 0);
    }
};

// A wave's weight rows, read through buffer descriptors: of each of its two blocks one for the codes and
// one for the scales, based at the block's first row.  Offsets past a descriptor's bytes read as zero, so
// a lane without work (kNoOffset) reads zeros at no cost: weights of 0 at a finite scale.
constexpr uint32_t kNoOffset = 0x80000000u;

struct Mx4Rows {
    __amdgpu_buffer_rsrc_t w[2], s[2];
    uint32_t wo[2], so[2];       // the lane's row and half
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx4_rsrc(const uint8_t *p, int64_t bytes) {
    const uint64_t u = (uint64_t)p;
    const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(u >> 32)) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((int)u);
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, __builtin_amdgcn_readfirstlane((int)bytes),
                                             0x00020000);
}

template <bool GATEUP>
__device__ __forceinline__ Mx4Rows mx4_rows(const Mx4Pass &a, int e, int ft, int lane) {
    const uint32_t wrow = (uint32_t)a.kruns * 64, srow = (uint32_t)a.kruns * 4;
    Mx4Rows R;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int f0 = GATEUP ? ft * 32 : ft * 64 + i * 32;
        const int n = max(0, min(32, a.F - f0));       // rows of the block
        const int64_t r = (int64_t)e * a.F + min(f0, a.F - 1);
        R.w[i] = mx4_rsrc((GATEUP && i ? a.w1 : a.w0) + r * wrow, (int64_t)n * wrow);
        R.s[i] = mx4_rsrc((GATEUP && i ? a.s1 : a.s0) + r * srow, (int64_t)n * srow);
        const bool in = (lane & 31) < n;
        R.wo[i] = in ? (lane & 31) * wrow + (lane >> 5) * 64 : kNoOffset;
        R.so[i] = in ? (lane & 31) * srow + (lane >> 5) * 4 : kNoOffset;
    }
    return R;
}

__device__ __forceinline__ i32x4 mx4_load16(__amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t so) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)vo, (int)so, 0));
}
__device__ __forceinline__ uint32_t mx4_load4(__amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t so) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, (int)vo, (int)so, 0);
}

// At the end of a loop body whose last loads are for its next round: keeps the compiler from merging them
// with the loads ahead of the loop into one at the loop's head, right before their use.
__device__ __forceinline__ void stay_here() { asm volatile("; loads of the next round are under way"); }

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
            const float g = p[i];
            // SiLU by the hardware's exponential and reciprocal, each within 2 ulp: far below the 4-bit step
            const float v = __fdividef(g, 1.0f + __expf(-g)) * u[i];
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

// Few rows an expert: bound by the stream of weights.  Waves take tiles of 64 weight rows and up to 32
// tokens by themselves, weights and tokens straight from memory to registers, each piece of the next
// segment requested as soon as this one's has been used.  SPLIT: too few tiles to occupy the GPU; the
// four waves of a workgroup then share a tile, each a quarter of the segments, and add up in LDS.
template <bool GATEUP, bool SPLIT>
__global__ __launch_bounds__(kMx4Threads, 4) void mx4_stream_kernel(const Mx4Pass a) {
    __shared__ f32x4 part[SPLIT ? (kMx4Waves - 1) * 8 * 64 : 1];
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // gate/up tiles also cover the padding up to whole runs, which is written as zeros
    const int ftiles = GATEUP ? a.hruns * 4 : (a.F + 63) / 64;
    TileList list;
    list.init(a.offsets, a.n_exp, 32, ftiles, lane);
    const int segs = (a.kruns + 1) / 2;   // with an odd number of runs the last one has no second half
    const bool second = lane >= 32;
    const int k0 = SPLIT ? segs * wid / kMx4Waves : 0, k1 = SPLIT ? segs * (wid + 1) / kMx4Waves : segs;
    const int step = SPLIT ? gridDim.x : gridDim.x * kMx4Waves;
    for (int t = SPLIT ? blockIdx.x : blockIdx.x * kMx4Waves + wid; t < list.total; t += step) {
        int e, ft, valid;
        int64_t row0;
        list.find(t, lane, e, ft, row0, valid);
        const Mx4Rows rows = mx4_rows<GATEUP>(a, e, ft, lane);
        // token columns past the tile's repeat its last one; their results are not used
        const int64_t R = row0 + min(lane & 31, valid - 1);
        const int64_t xr = a.gather ? a.gather[R] : R;
        const uint8_t *xp = a.x + xr * ((int64_t)a.kruns * 64), *xsp = a.xs + xr * ((int64_t)a.kruns * 4);
        f32x16 acc[2] = {};
        i32x4 w[2][4], x[4];
        uint32_t ws[2], xs, wo[2], so[2];
        const uint8_t *xk, *xsk;
        // where segment k lies; a segment past the end reads nothing (tokens: the last one again)
        auto aim = [&](int k) {
            const bool none = k >= k1 || (2 * k + 1 == a.kruns && second);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                wo[i] = none ? kNoOffset : rows.wo[i];
                so[i] = none ? kNoOffset : rows.so[i];
            }
            const int kx = 2 * min(k, k1 - 1) + (second && 2 * k + 1 < a.kruns ? 1 : 0);
            xk = xp + (int64_t)kx * 64;
            xsk = xsp + (int64_t)kx * 4;
        };
        auto piece = [&](int k, int c) {
            w[0][c] = mx4_load16(rows.w[0], wo[0] + c * 16, k * 128);
            w[1][c] = mx4_load16(rows.w[1], wo[1] + c * 16, k * 128);
            x[c] = *(const i32x4 *)(xk + c * 16);
        };
        auto scales = [&](int k) {
            ws[0] = mx4_load4(rows.s[0], so[0], k * 8);
            ws[1] = mx4_load4(rows.s[1], so[1], k * 8);
            xs = *(const uint32_t *)xsk;
        };
        if (k0 < k1) {
            aim(k0);
            scales(k0);
#pragma unroll
            for (int c = 0; c < 4; ++c) piece(k0, c);
        }
        for (int k = k0; k < k1; ++k) {
            const uint32_t us[2] = {ws[0], ws[1]}, vs = xs;
            aim(k + 1);
            scales(k + 1);
            auto step = [&](auto sc) {
                constexpr int S = decltype(sc)::value;
                // the order is fixed: a piece's registers are free for the next one once its products are issued
                __builtin_amdgcn_sched_barrier(0);
                acc[0] = mx4_mfma<S>(w[0][S], x[S], acc[0], us[0], vs);
                acc[1] = mx4_mfma<S>(w[1][S], x[S], acc[1], us[1], vs);
                __builtin_amdgcn_sched_barrier(0);
                piece(k + 1, S);
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            step(std::integral_constant<int, 2>{});
            step(std::integral_constant<int, 3>{});
            stay_here();
        }
        if (SPLIT) {
            __syncthreads();   // the previous tile's sums have been read
            if (wid > 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        part[((wid - 1) * 8 + i * 4 + q) * 64 + lane] =
                            f32x4{acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]};
            }
            __syncthreads();
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
        mx4_store<GATEUP>(a, mx4_out<GATEUP>(a, row0, valid), acc[0], acc[1], ft, lane & 31, lane);
    }
}

// Many rows an expert.  A workgroup's tile is 256 weight rows (64 a wave) against up to 256 tokens, one
// workgroup a compute unit: a wave then has the registers for 64 x 256 sums, two segments of
// weights on their way and the next step's tokens.  Weights go straight to the registers of the one wave
// that uses them; the tokens' segments, which all four waves use, pass through two LDS buffers.
constexpr int kMx4TileTokens = 256;

// 16-byte piece p of token row r in LDS: rows are 128 bytes, and the 16 lanes that LDS serves
// together (quads of a wave half with the same bit parity) hold each of the eight row
// pairs' low three bits once, which this permutation turns into eight different pieces.
__device__ __forceinline__ int mx4_lds(int r, int p) { return r * 128 + ((p ^ ((r >> 1) & 7)) << 4); }

template <bool GATEUP>
__global__ __launch_bounds__(kMx4Threads, 1) void mx4_tile_kernel(const Mx4Pass a) {
    __shared__ __align__(16) char xbuf[2][kMx4TileTokens * 128];
    __shared__ uint32_t sbuf[2][kMx4TileTokens * 2];
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, r31 = lane & 31;
    const int wtiles = GATEUP ? a.hruns * 4 : (a.F + 63) / 64;
    const int ftiles = (wtiles + kMx4Waves - 1) / kMx4Waves;
    TileList list;
    list.init(a.offsets, a.n_exp, kMx4TileTokens, ftiles, lane);
    const int segs = (a.kruns + 1) / 2;   // with an odd number of runs the last one has no second half
    // workgroup b runs on XCD b mod 8: each XCD takes a contiguous eighth of the list, so that the row
    // blocks of a weight tile and the weight tiles of a row block meet in its L2
    const int per = (list.total + 7) / 8, xcd = blockIdx.x & 7;
    const int end = min(list.total, (xcd + 1) * per);
    const int64_t xrow = (int64_t)a.kruns * 64;

    // staging: lane l of wave w brings piece l mod 8 of token rows 32 i + 8 w + l / 8
    const int srow = wid * 8 + (lane >> 3), sp = lane & 7;
    struct Tile {
        Mx4Rows rows;
        const uint8_t *xp[8], *xsp;
        int64_t row0;
        int valid, wt;
    } T;
    i32x4 w[2][2][4], xv[8];
    uint32_t ws[2][2], xsv[2], wo[2], so[2];
    auto setup = [&](int t) {
        int e, ft;
        list.find(t, lane, e, ft, T.row0, T.valid);
        T.wt = ft * kMx4Waves + wid;
        T.rows = mx4_rows<GATEUP>(a, e, T.wt, lane);
        // token rows past the tile's repeat its last one; their results are not used
        auto token = [&](int r) {
            const int64_t R = T.row0 + min(r, T.valid - 1);
            return a.gather ? (int64_t)a.gather[R] : R;
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) T.xp[i] = a.x + token(32 * i + srow) * xrow;
        T.xsp = a.xs + token(tid) * (xrow >> 4);
    };
    // (blocks of 32 token rows past the tile's are neither read nor written)
    auto fetch = [&](int k, auto tbc) {
        const int last = min(k, segs - 1);
        // the half that an odd number of runs lacks meets weights of zero: it repeats the other
        const int64_t o = (int64_t)last * 128 + (2 * last + 1 < a.kruns ? sp : sp & 3) * 16;
#pragma unroll
        for (int i = 0; i < decltype(tbc)::value; ++i) xv[i] = *(const i32x4 *)(T.xp[i] + o);
        const uint8_t *s = T.xsp + (int64_t)last * 8;
        xsv[0] = *(const uint32_t *)s;
        xsv[1] = *(const uint32_t *)(s + (2 * last + 1 < a.kruns ? 4 : 0));
    };
    auto keep = [&](int k, auto tbc) {
#pragma unroll
        for (int i = 0; i < decltype(tbc)::value; ++i) *(i32x4 *)(xbuf[k & 1] + mx4_lds(32 * i + srow, sp)) = xv[i];
        *(u32x2 *)(sbuf[k & 1] + 2 * tid) = u32x2{xsv[0], xsv[1]};
    };
    auto aim = [&](int k) {
        const bool none = k >= segs || (2 * k + 1 == a.kruns && half);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            wo[i] = none ? kNoOffset : T.rows.wo[i];
            so[i] = none ? kNoOffset : T.rows.so[i];
        }
    };
    auto piece = [&](int k, int g, int c) {
        w[g][0][c] = mx4_load16(T.rows.w[0], wo[0] + c * 16, k * 128);
        w[g][1][c] = mx4_load16(T.rows.w[1], wo[1] + c * 16, k * 128);
    };
    auto scales = [&](int k, int g) {
        ws[g][0] = mx4_load4(T.rows.s[0], so[0], k * 8);
        ws[g][1] = mx4_load4(T.rows.s[1], so[1], k * 8);
    };
    // the loads of a tile's first segments (of all its token rows: the tile's own loop is not chosen yet)
    auto start = [&](int t) {
        setup(t);
        fetch(0, std::integral_constant<int, 8>{});
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            aim(g);
            scales(g, g);
#pragma unroll
            for (int c = 0; c < 4; ++c) piece(g, g, c);
        }
    };

    int t = xcd * per + (blockIdx.x >> 3);
    if (t >= end) return;
    start(t);
    // One tile of up to 32 TB tokens.  Segment k's tokens are in LDS buffer k mod 2 and its weights in register
    // set k mod 2.  Meanwhile segment k + 1's tokens come in, and as a piece's products are issued, that of
    // segment k + 2; the next tile's first loads are under way while this one's results are written.
    auto tile = [&](auto tbc) {
        constexpr int TB = decltype(tbc)::value;
        f32x16 acc[2][TB] = {};
        keep(0, tbc);
        wait_lgkm0();
        cta_barrier();
        i32x4 b[2][TB];
        uint32_t xs[TB];
        auto tokens = [&](int k, int g, int s) {
#pragma unroll
            for (int j = 0; j < TB; ++j)
                b[g][j] = *(const i32x4 *)(xbuf[k & 1] + mx4_lds(j * 32 + r31, half * 4 + s));
        };
        auto token_scales = [&](int k) {
#pragma unroll
            for (int j = 0; j < TB; ++j) xs[j] = sbuf[k & 1][(j * 32 + r31) * 2 + half];
        };
        tokens(0, 0, 0);
        token_scales(0);
        auto segment = [&](int k, auto gc) {
            constexpr int G = decltype(gc)::value;
            fetch(k + 1, tbc);
            const uint32_t us[2] = {ws[G][0], ws[G][1]};
            uint32_t vs[TB];
#pragma unroll
            for (int j = 0; j < TB; ++j) vs[j] = xs[j];
            aim(k + 2);
            auto step = [&](auto sc) {
                constexpr int S = decltype(sc)::value;
                if (S < 3) {
                    tokens(k, (S + 1) & 1, S + 1);
                } else {
                    // every read of the other buffer's last segment came before the previous barrier
                    keep(k + 1, tbc);
                    wait_lgkm0();
                    cta_barrier();
                    tokens(k + 1, 0, 0);
                    token_scales(k + 1);
                    scales(k + 2, G);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    acc[0][j] = mx4_mfma<S>(w[G][0][S], b[S & 1][j], acc[0][j], us[0], vs[j]);
                    acc[1][j] = mx4_mfma<S>(w[G][1][S], b[S & 1][j], acc[1][j], us[1], vs[j]);
                }
                __builtin_amdgcn_sched_barrier(0);
                piece(k + 2, G, S);
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            step(std::integral_constant<int, 2>{});
            step(std::integral_constant<int, 3>{});
        };
        int k = 0;
        for (; k + 1 < segs; k += 2) {
            segment(k, std::integral_constant<int, 0>{});
            segment(k + 1, std::integral_constant<int, 1>{});
            stay_here();
        }
        if (k < segs) segment(k, std::integral_constant<int, 0>{});
        const Mx4Out out = mx4_out<GATEUP>(a, T.row0, T.valid);
        const int wt = T.wt;
        t += gridDim.x >> 3;
        cta_barrier();   // every wave is done with the buffers
        if (t < end) start(t);
        if (wt < wtiles) {
#pragma unroll
            for (int j = 0; j < TB; ++j) mx4_store<GATEUP>(a, out, acc[0][j], acc[1][j], wt, j * 32 + r31, lane);
        }
    };
    while (t < end) {
        if (T.valid <= 64) tile(std::integral_constant<int, 2>{});
        else if (T.valid <= 128) tile(std::integral_constant<int, 4>{});
        else if (T.valid <= 192) tile(std::integral_constant<int, 6>{});
        else tile(std::integral_constant<int, 8>{});
    }
}

}  // namespace

hipError_t launch_mx4_quantize(int dt, const void *x, int64_t ld, int64_t rows, int cols, uint8_t *q, uint8_t *sc,
                               hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const int runs = (int)mx4_runs(cols);
    const int64_t wgs = (rows * runs + 15) / 16;
    const unsigned grid = (unsigned)(wgs < 16384 ? wgs : 16384);
    const bool vec = (uintptr_t)x % 16 == 0 && ld % (dt == DT_F32 ? 4 : 8) == 0;
    if (dt == DT_F32) {
        if (vec) mx4_quantize_kernel<DT_F32, true><<<grid, 256, 0, s>>>(x, ld, rows, cols, runs, q, sc);
        else mx4_quantize_kernel<DT_F32, false><<<grid, 256, 0, s>>>(x, ld, rows, cols, runs, q, sc);
    } else {
        if (vec) mx4_quantize_kernel<DT_BF16, true><<<grid, 256, 0, s>>>(x, ld, rows, cols, runs, q, sc);
        else mx4_quantize_kernel<DT_BF16, false><<<grid, 256, 0, s>>>(x, ld, rows, cols, runs, q, sc);
    }
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(int dt, const uint8_t *q, const uint8_t *sc, int64_t rows, int cols, void *y,
                                 int64_t ld, hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const int runs = (int)mx4_runs(cols);
    const int64_t wgs = (rows * runs * 16 + 255) / 256;
    const unsigned grid = (unsigned)(wgs < 16384 ? wgs : 16384);
    const bool vec = (uintptr_t)y % 16 == 0 && ld % (dt == DT_F32 ? 4 : 8) == 0;
    if (dt == DT_F32) {
        if (vec) mx4_dequantize_kernel<DT_F32, true><<<grid, 256, 0, s>>>(q, sc, rows, cols, runs, y, ld);
        else mx4_dequantize_kernel<DT_F32, false><<<grid, 256, 0, s>>>(q, sc, rows, cols, runs, y, ld);
    } else {
        if (vec) mx4_dequantize_kernel<DT_BF16, true><<<grid, 256, 0, s>>>(q, sc, rows, cols, runs, y, ld);
        else mx4_dequantize_kernel<DT_BF16, false><<<grid, 256, 0, s>>>(q, sc, rows, cols, runs, y, ld);
    }
    return hipGetLastError();
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
    // 32 rows an expert fill one token block: up to there a tile is bound by its weights
    if (a.max_rows <= 32 * (int64_t)a.n_exp) {
        // with fewer tiles than resident waves, at most, a tile takes four waves
        const int64_t experts = a.max_rows < a.n_exp ? a.max_rows : a.n_exp;
        const unsigned grid = (unsigned)(4 * cus);
        auto go = [&](auto gateup, const Mx4Pass &p, int64_t ftiles) {
            constexpr bool GU = decltype(gateup)::value;
            if (experts * ftiles < 16 * cus) mx4_stream_kernel<GU, true><<<grid, kMx4Threads, 0, s>>>(p);
            else mx4_stream_kernel<GU, false><<<grid, kMx4Threads, 0, s>>>(p);
        };
        go(std::true_type{}, up, up.hruns * 4);
        go(std::false_type{}, down, (a.d + 63) / 64);
    } else {
        const unsigned grid = (unsigned)((cus + 7) / 8 * 8);
        mx4_tile_kernel<true><<<grid, kMx4Threads, 0, s>>>(up);
        mx4_tile_kernel<false><<<grid, kMx4Threads, 0, s>>>(down);
    }
    return hipGetLastError();
}

}  // namespace moe
