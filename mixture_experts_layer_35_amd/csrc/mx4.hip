// mx4.hip -- microscaled 4-bit floating point (OCP Microscaling Formats v1.0: E2M1 codes,
// one E8M0 scale for 32 values): rounding, its inverse, and the SwiGLU experts on MX4
// weights and activations.
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

// One pass over an expert's weights: gate/up (H = Q(SiLU(x Wg^T) * (x Wu^T))) or down (y = H Wd^T).
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
    int yvec;                    // rows of y take 8-byte stores
};

typedef uint32_t u32a __attribute__((aligned(4)));

__device__ __forceinline__ f32x4 mx4_mfma(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0},
                                                            i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, c, 4, 4, 0, sa, 0,
                                                            sb);
}

// Tile t of the list (experts in order; an expert's row blocks of `bm`, each with its ftiles feature
// tiles): the expert, its row block and feature tile.  Every wave works it out by itself: lane l
// adds up the tiles of experts l*P .. l*P + P-1.
struct TileList {
    const int32_t *offsets;
    int n, P, bm, ftiles;
    int base, count;             // this lane's first tile and tiles
    int total;
    __device__ void init(const int32_t *o, int n_, int bm_, int ftiles_, int lane) {
        offsets = o;
        n = n_;
        bm = bm_;
        ftiles = ftiles_;
        P = (n + 63) / 64;
        count = 0;
        for (int e = lane * P; e < min(n, lane * P + P); ++e) count += tiles(e);
        int run = count;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int up = __shfl_up(run, m, 64);
            if (lane >= m) run += up;
        }
        base = run - count;
        total = __builtin_amdgcn_readlane(run, 63);
    }
    __device__ int tiles(int e) const { return (offsets[e + 1] - offsets[e] + bm - 1) / bm * ftiles; }
    // t < total, the same in all lanes
    __device__ void find(int t, int lane, int &e, int &block, int &ft) const {
        const uint64_t started = __ballot(count > 0 && base <= t);
        const int owner = 63 - __builtin_clzll(started);
        int le = 0, rest = t - base;
        if (lane == owner) {
            le = lane * P;
            for (int k = tiles(le); rest >= k; k = tiles(le)) {
                rest -= k;
                ++le;
            }
        }
        e = __builtin_amdgcn_readlane(le, owner);
        rest = __builtin_amdgcn_readlane(rest, owner);
        block = rest / ftiles;
        ft = rest - block * ftiles;
    }
};

constexpr int kMx4Waves = 4;
constexpr int kMx4Threads = 64 * kMx4Waves;

// A workgroup's tile: 64 weight rows (gate/up: 32 gate rows and the matching 32 up rows) against
// up to 16 * NB tokens of one expert.  The four waves split the reduction and add their sums in LDS.
template <bool GATEUP, int NB>
__global__ __launch_bounds__(kMx4Threads) void mx4_expert_kernel(const Mx4Pass a) {
    __shared__ f32x4 part[kMx4Waves][4][NB][64];
    const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
    const int r15 = lane & 15, g = lane >> 4;
    constexpr int FT = GATEUP ? 32 : 64;
    // gate/up tiles also cover the padding up to whole runs, which is written as zeros
    const int ftiles = GATEUP ? a.hruns * 4 : (a.F + FT - 1) / FT;
    TileList list;
    list.init(a.offsets, a.n_exp, 16 * NB, ftiles, lane);
    const int64_t wrow = (int64_t)a.kruns * 64, srow = (int64_t)a.kruns * 4;

    for (int t = blockIdx.x; t < list.total; t += gridDim.x) {
        int e, block, ft;
        list.find(t, lane, e, block, ft);
        const int64_t row0 = a.offsets[e] + (int64_t)block * 16 * NB;
        const int valid = min(16 * NB, a.offsets[e + 1] - (int)row0);
        // rows past the features or the tokens repeat the last one; their results are not used
        const uint8_t *wp[4], *sp[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int f = min(ft * FT + (GATEUP ? (i & 1) : i) * 16 + r15, a.F - 1);
            const int64_t r = (int64_t)e * a.F + f;
            wp[i] = (GATEUP && i >= 2 ? a.w1 : a.w0) + r * wrow + g * 16;
            sp[i] = (GATEUP && i >= 2 ? a.s1 : a.s0) + r * srow;
        }
        const uint8_t *xp[NB], *xsp[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int64_t R = row0 + min(j * 16 + r15, valid - 1);
            const int64_t xr = a.gather ? a.gather[R] : R;
            xp[j] = a.x + xr * wrow + g * 16;
            xsp[j] = a.xs + xr * srow;
        }
        f32x4 acc[4][NB];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
        for (int k = wid; k < a.kruns; k += kMx4Waves) {
            i32x4 wa[4], xb[NB];
            uint32_t ws[4], xs[NB];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wa[i] = *(const i32x4 *)(wp[i] + (int64_t)k * 64);
                ws[i] = *(const uint32_t *)(sp[i] + (int64_t)k * 4) >> (8 * g);
            }
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                xb[j] = *(const i32x4 *)(xp[j] + (int64_t)k * 64);
                xs[j] = *(const uint32_t *)(xsp[j] + (int64_t)k * 4) >> (8 * g);
            }
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = mx4_mfma(wa[i], xb[j], acc[i][j], ws[i], xs[j]);
        }
        __syncthreads();   // the previous tile's sums have been read
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) part[wid][i][j][lane] = acc[i][j];
        __syncthreads();
        // token block j's results: lane holds features 4g .. 4g+3 of each 16-row block, token r15
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            if (j % kMx4Waves != wid) continue;
            f32x4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = part[0][i][j][lane];
#pragma unroll
                for (int k = 1; k < kMx4Waves; ++k) v[i] += part[k][i][j][lane];
            }
            const bool live = j * 16 + r15 < valid;
            const int64_t R = row0 + j * 16 + r15;
            if (GATEUP) {
                // the tile's 32 features are one MX4 block of H
                float h[8];
                uint32_t amax = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float av = v[i][q], bv = v[i + 2][q];
                        const bool in = ft * 32 + i * 16 + 4 * g + q < a.F;
                        h[i * 4 + q] = in ? av / (1.0f + expf(-av)) * bv : 0.0f;
                        amax = max(amax, __float_as_uint(h[i * 4 + q]) & 0x7FFFFFFFu);
                    }
                amax = max(amax, (uint32_t)__shfl_xor((int)amax, 16, 64));
                amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32, 64));
                const uint32_t s = mx4_scale(amax), c = mx4_codes(h, s);
                if (live) {
                    uint16_t *p = (uint16_t *)(a.h + (R * a.hruns * 64 + ft * 16 + 2 * g));
                    p[0] = (uint16_t)c;           // features 4g .. 4g+3 of the first 16
                    p[4] = (uint16_t)(c >> 16);   // and of the second
                    if (g == 0) a.hs[R * a.hruns * 4 + ft] = (uint8_t)s;
                }
            } else if (live) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int f = ft * 64 + i * 16 + 4 * g;
                    uint16_t *p = a.y + R * a.F + f;
                    if (a.yvec && f < a.F) {
                        *(u32x2 *)p = u32x2{pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3])};
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (f + q < a.F) p[q] = (uint16_t)pack_bf16x2(v[i][q], 0.0f);
                    }
                }
            }
        }
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
    down.yvec = (uintptr_t)a.y % 8 == 0 && a.d % 4 == 0;
    const unsigned grid = 4 * (unsigned)device_cus();
    if (a.max_rows <= 16 * (int64_t)a.n_exp) {
        mx4_expert_kernel<true, 1><<<grid, kMx4Threads, 0, s>>>(up);
        mx4_expert_kernel<false, 1><<<grid, kMx4Threads, 0, s>>>(down);
    } else {
        mx4_expert_kernel<true, 2><<<grid, kMx4Threads, 0, s>>>(up);
        mx4_expert_kernel<false, 2><<<grid, kMx4Threads, 0, s>>>(down);
    }
    return hipGetLastError();
}

}  // namespace moe
