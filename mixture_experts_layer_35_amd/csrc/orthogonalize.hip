// orthogonalize.hip -- an update's matrices brought near the nearest orthogonal ones by Newton-Schulz steps:
//   X_0 = G / (|G|_F + eps);   S = X X^T,  P = b S + c S S,  X <- a X + P X
// with G transposed where it has more rows than columns.
//
// Products take pairs of bf16, hi = the nearest bf16 and lo = that of what is left, which keep 16 significant bits: a product of
// pairs is three matrix products, hi hi + hi lo + lo hi, summed in fp32 (lo lo is below what a pair drops).  Rows of pairs hold
// 32 hi and then 32 lo of 32 values in turn, 128 bytes, which is what a step of the reduction takes from a row.  Sides are padded
// to multiples of 32 with zeros.
//
// Plain bf16 would leave a few percent: a step multiplies the smallest singular values, and errors beside them, by up to
// a = 3.4, five steps by 485.  What is multiplied so are errors outside both the rows' and the columns' space of X.  a X brings
// such; P X lies in X's spaces on one side at least, whatever rounding P or X took, but for the dropped lo lo, ten times less.
// So S and P are held in pairs, and the X that a multiplies in all of fp32's 24 bits, its last 8 (`rest`, a bf16 that is exact)
// where y will be, as long as the steps left multiply by more than kRestGrowth: a pair loses 2^-18 of a value, which 64 times as
// large is a seventh of what the result's rounding to bf16 loses.  Against 64 bits, before that rounding (1.7e-3), 512 x 1024:
// rank 1 2.4e-4, rank 3 1.6e-4, full rank 3e-5; with X in pairs alone 1.7e-3, 1.1e-3 and 3e-5, with all bits in every step
// 1.8e-4, 7.5e-5 and 3e-5, with everything in fp32 1.0e-4, 4.5e-5 and 2e-6.  8 matrices of 2048 x 7168 take 11.2 ms so and 11.0
// with X in pairs alone, 24 of 1000 x 360 498 us and 478.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "lds_ring.h"
#include "strided.h"
#include "variants.h"

namespace moe {

namespace {

constexpr int kOrthThreads = 512;
constexpr double kRestGrowth = 64.0;

// hi and lo of a value (lo is rounded where it is stored); one that is not finite gives NaN in lo and so in every sum it meets.
__device__ __forceinline__ void split_pair(float v, float &hi, float &lo) {
    hi = bf16_to_f32((uint16_t)pack_bf16x2(v, 0.0f));
    lo = v - hi;
}

// What hi and lo leave of a value: 8 bits, exact in bf16.
__device__ __forceinline__ float rest_of(float lo) { return lo - bf16_to_f32((uint16_t)pack_bf16x2(lo, 0.0f)); }

// ---- norms and the first X ---------------------------------------------------

constexpr int kNormThreads = 256;

// part[m][p]: the sum of the squares of a share of matrix m, in 64 bits (no square of an fp32 value leaves them).
template <int DT>
__global__ __launch_bounds__(kNormThreads) void orth_norm_kernel(const void *__restrict__ g, int64_t size, int parts,
                                                                 double *__restrict__ part) {
    const int m = blockIdx.x / parts, p = blockIdx.x % parts;
    const int64_t eights = (size + 7) / 8, from = eights * p / parts, to = eights * (p + 1) / parts;
    double sum = 0.0;
    for (int64_t i = from + threadIdx.x; i < to; i += kNormThreads) {
        float v[8];
        load8<DT>(g, m * size + i * 8, size - i * 8, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += (double)v[k] * v[k];
    }
    __shared__ double all[kNormThreads];
    all[threadIdx.x] = sum;
    __syncthreads();
    for (int w = kNormThreads / 2; w > 0; w >>= 1) {
        if ((int)threadIdx.x < w) all[threadIdx.x] += all[threadIdx.x + w];
        __syncthreads();
    }
    if (threadIdx.x == 0) part[blockIdx.x] = all[0];
}

// 1 / (norm + eps) of matrix m from its at most 64 parts, in every lane.
__device__ __forceinline__ double orth_inverse(const double *part, int m, int parts, double eps) {
    const int lane = threadIdx.x & 63;
    double sum = lane < parts ? part[m * (int64_t)parts + lane] : 0.0;
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) sum += __shfl_xor(sum, w, 64);
    return 1.0 / (sqrt(sum) + eps);
}

// Eight values of a row of X as pairs: `at` is a multiple of 8.
__device__ __forceinline__ void store_pairs(uint16_t *row, int at, const float (&v)[8]) {
    u32x4 oh, ol;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float hi[2], lo[2];
        split_pair(v[2 * k], hi[0], lo[0]);
        split_pair(v[2 * k + 1], hi[1], lo[1]);
        oh[k] = pack_bf16x2(hi[0], hi[1]);
        ol[k] = pack_bf16x2(lo[0], lo[1]);
    }
    uint16_t *to = row + (at >> 5) * 64 + (at & 31);
    *(u32x4 *)to = oh;
    *(u32x4 *)(to + 32) = ol;
}

// What pairs leave of eight values, `n` of which are there, to y (if any).
__device__ __forceinline__ void store_rests(uint16_t *y, int64_t at, int n, const float (&v)[8]) {
    if (!y) return;
    float rest[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float hi, lo;
        split_pair(v[k], hi, lo);
        rest[k] = rest_of(lo);
    }
    if (n >= 8) {
        *(u32x4_any *)(y + at) = u32x4{pack_bf16x2(rest[0], rest[1]), pack_bf16x2(rest[2], rest[3]),
                                       pack_bf16x2(rest[4], rest[5]), pack_bf16x2(rest[6], rest[7])};
        return;
    }
#pragma unroll
    for (int k = 0; k < 7; ++k)
        if (k < n) y[at + k] = (uint16_t)pack_bf16x2(rest[k], 0.0f);
}

// X_0 in pairs, and what they leave in y, which lies as G does and may be G: a thread writes there what it has read.
// A workgroup takes 64 x 64 values; those of G^T (TALL) are turned over in LDS.
template <int DT, bool TALL>
__global__ __launch_bounds__(256) void orth_first_kernel(const void *g, const double *__restrict__ part, int parts,
                                                         double eps, int r, int c, int rp, int cp,
                                                         uint16_t *__restrict__ x, uint16_t *y) {
    const int m = blockIdx.z, c0 = blockIdx.x * 64, r0 = blockIdx.y * 64;
    const double inv = orth_inverse(part, m, parts, eps);
    const int64_t base = (int64_t)m * r * c;
    __shared__ float turned[TALL ? 64 * 65 : 1];
    const int row = threadIdx.x >> 3, eight = (threadIdx.x & 7) * 8;
    if (TALL) {
        // rows of G are columns of X
#pragma unroll
        for (int k = 0; k < 64; k += 32) {
            const int j = c0 + row + k, i = r0 + eight;
            float v[8];
            load8<DT>(g, base + (int64_t)j * r + i, j < c ? r - i : 0, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                v[q] = (float)((double)v[q] * inv);
                turned[(eight + q) * 65 + row + k] = v[q];
            }
            store_rests(y, base + (int64_t)j * r + i, j < c ? r - i : 0, v);
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < 64; k += 32) {
        const int i = r0 + row + k, j = c0 + eight;
        float v[8];
        if (TALL) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = turned[(row + k) * 65 + eight + q];
        } else {
            load8<DT>(g, base + (int64_t)i * c + j, i < r ? c - j : 0, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = (float)((double)v[q] * inv);
            store_rests(y, base + (int64_t)i * c + j, i < r ? c - j : 0, v);
        }
        if (i < rp && j < cp) store_pairs(x + ((int64_t)m * rp + i) * cp * 2, j, v);
    }
}

// ---- products ----------------------------------------------------------------

// out[b][a] = sum over k of A(a, k) B(b, k):
//   GRAM    A, B: rows of X, k along them         S, symmetric
//   SQUARE  A, B: rows of S                       P = c S S + b S, symmetric
//   UPDATE  A: columns of X (k: its rows), B: rows of P      a X + P X
// SINGLE: the update of matrices whose y is taken value by value: X lies across it, or has fewer than four columns.
enum { ORTH_GRAM, ORTH_SQUARE, ORTH_UPDATE, ORTH_UPDATE_SINGLE };

struct OrthPass {
    int n;
    int A, B, K;                // sides of out, padded, and the reduction's length
    const uint16_t *a, *b;      // pairs; rows of K (A: UPDATE rows of A)
    const uint16_t *c;          // what the epilogue adds, as out
    float alpha, beta;          // out = alpha * sum + beta * c
    uint16_t *out;              // pairs
    uint16_t *y;                // UPDATE: [rows][cols] of G,
    int rest_in, rest_out;      // what pairs leave of c and then of out,
    int last;                   // or the result in bf16 (out is not written)
    int r, cc, tall;            // sides of X without padding
};

// Eight waves, WA along a by 8 / WA along b (16-row blocks of b in turn), each with RB blocks of 16 values of a and CB of b.
template <int RB, int CB, int WA>
struct OrthTile {
    static constexpr int WB = 8 / WA, TA = RB * 16 * WA, TB = CB * 16 * WB;
    static constexpr int stage_a = TA * 128, stage = stage_a + TB * 128;
    static constexpr int scratch = 8 * 16 * 17 * 4;     // a 16 x 16 block of each wave, turned over
    static constexpr int slots = (160 * 1024 - scratch) / stage < 8 ? (160 * 1024 - scratch) / stage : 8;
    static constexpr int lds = slots * stage + scratch;
};

template <int OP, int RB, int CAP, int WA>
__global__ __launch_bounds__(kOrthThreads, 1) void orth_kernel(const OrthPass a) {
    typedef OrthTile<RB, CAP, WA> T;
    constexpr bool SINGLE = OP == ORTH_UPDATE_SINGLE, UPDATE = OP == ORTH_UPDATE || SINGLE, SYM = !UPDATE, ASTRIDED = UPDATE;
    constexpr int SLOTS = T::slots, STAGE = T::stage, WB = T::WB, QA = T::TA / 64, QB = T::TB / 64, N = QA + QB;
    constexpr int ROW = T::TA * 4, LANES = ROW / 16;   // a staged row of the reduction: bytes, lanes that bring it
    static_assert(T::TA % 64 == 0 && T::TB % 64 == 0 && RB % 2 == 0 && SLOTS >= 2, "loads of a step are shared evenly");
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    char *const ring = smem;
    const int filled = lds_place(ring);              // the ring for direct loads
    uint32_t *const turn = (uint32_t *)(smem + SLOTS * STAGE) + wid * (16 * 17);
    const int at = (a.A + T::TA - 1) / T::TA, bt = (a.B + T::TB - 1) / T::TB;
    // symmetric: the tiles that reach the diagonal or lie below it (b >= a), for each column of tiles a run of them
    auto tiles_below = [&](int ia) { return bt - min(bt, ia * T::TA / T::TB); };
    int per_matrix = at * bt;
    if (SYM) {
        per_matrix = 0;
        for (int i = 0; i < at; ++i) per_matrix += tiles_below(i);
    }
    const int total = a.n * per_matrix;
    const int per = (total + 7) / 8, xcd = blockIdx.x & 7;
    const int end = min(total, (xcd + 1) * per), first = xcd * per + (blockIdx.x >> 3), step = gridDim.x >> 3;
    if (first >= end) return;
    auto find = [&](int t, int &m, int &a0, int &b0) __attribute__((always_inline)) {
        m = __builtin_amdgcn_readfirstlane(t / per_matrix);
        int rest = t - m * per_matrix, ia = 0;
        if (SYM) {
            for (int k = tiles_below(0); rest >= k; k = tiles_below(ia)) {
                rest -= k;
                ++ia;
            }
            b0 = (bt - tiles_below(ia) + rest) * T::TB;
        } else {
            ia = __builtin_amdgcn_readfirstlane(rest / bt);
            b0 = (rest - ia * bt) * T::TB;
        }
        a0 = ia * T::TA;
    };
    const int steps = a.K / 32;

    // ---- loads ----
    int it = first, ik = 0;
    i32x4s ar, br;
    uint32_t avoff[QA], bvoff[QB];
    const int a_step = ASTRIDED ? 32 * a.A * 4 : 128;
    auto bytes_at = [&](int row) { return ((lane & 7) ^ swz<128>(row)) << 4; };
    auto aim = [&]() __attribute__((always_inline)) {
        int m, a0, b0;
        find(it, m, a0, b0);
        const int64_t amat = (int64_t)(ASTRIDED ? a.K : a.A) * (ASTRIDED ? a.A : a.K) * 2, bmat = (int64_t)a.B * a.K * 2;
        ar = words_of(a.a + m * amat, amat * 2);
        br = words_of(a.b + m * bmat, bmat * 2);
#pragma unroll
        for (int q = 0; q < QA; ++q) {
            if (ASTRIDED) {
                const int k = (wid * QA + q) * (64 / LANES) + lane / LANES;
                const int col = a0 * 4 + (((lane % LANES) ^ strided_slot(k)) << 4);
                avoff[q] = col < a.A * 4 ? (uint32_t)(k * a.A * 4 + col) : kNoOffset;
            } else {
                const int row = (wid * QA + q) * 8 + (lane >> 3);
                avoff[q] = a0 + row < a.A ? (uint32_t)((a0 + row) * a.K * 4 + bytes_at(row)) : kNoOffset;
            }
        }
#pragma unroll
        for (int q = 0; q < QB; ++q) {
            const int row = (q * 8 + wid) * 8 + (lane >> 3);
            bvoff[q] = b0 + row < a.B ? (uint32_t)((b0 + row) * a.K * 4 + bytes_at(row)) : kNoOffset;
        }
    };
    // issues a step's N loads; 0 behind the last tile
    auto issue = [&](int slot) __attribute__((always_inline)) {
        if (it >= end) return 0;
        if (ik == 0) aim();
        const int as = filled + slot * STAGE + wid * (QA * 1024), bs = filled + slot * STAGE + T::stage_a + wid * 1024;
#pragma unroll
        for (int q = 0; q < QA; ++q) fill16(ar, avoff[q], ik * a_step, as + q * 1024);
#pragma unroll
        for (int q = 0; q < QB; ++q) fill16(br, bvoff[q], ik * 128, bs + q * 8192);
        if (++ik == steps) {
            ik = 0;
            it += step;
        }
        return N;
    };

    // ---- products ----
    const int wf = wid / WB, wm = wid % WB, r15 = lane & 15, g = lane >> 4;
    const int arow = wf * (RB * 16) + r15, brow = wm * 16 + r15;
    const int alo = arow * 128 + ((g ^ swz<128>(arow)) << 4), blo = brow * 128 + ((g ^ swz<128>(brow)) << 4);
    int aofs[RB][2];
    if (ASTRIDED) {
        const int jj = (lane >> 2) & 3, aa = lane & 3, k = 8 * g + jj;
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int col = wf * (RB * 16) + i * 16 + 4 * aa;
                const int piece = ((col >> 5) * 128 + p * 64 + (col & 31) * 2) >> 4;
                aofs[i][p] = k * ROW + ((piece ^ strided_slot(k)) << 4) + 8 * (aa & 1);
            }
    }
    int slot = 0;
    auto next = [](int s, int d) { return s + d >= SLOTS ? s + d - SLOTS : s + d; };
    int later[SLOTS - 1] = {};       // loads of the steps under way, the next one's first
    issue(0);
#pragma unroll
    for (int s = 1; s < SLOTS - 1; ++s) later[s - 1] = issue(s);
    for (int t = first; t < end; t += step) {
        f32x4 acc[RB][CAP] = {};
        for (int k = 0; k < steps; ++k) {
            int n = 0;
#pragma unroll
            for (int s = 0; s < SLOTS - 2; ++s) n += later[s];
            wait_vmcnt_dyn(n);
            wait_lgkm0();
            cta_barrier();
#pragma unroll
            for (int s = 0; s + 1 < SLOTS - 2; ++s) later[s] = later[s + 1];
            n = issue(next(slot, SLOTS - 1));
            if (SLOTS > 2) later[SLOTS > 2 ? SLOTS - 3 : 0] = n;
            const char *as = ring + slot * STAGE, *bs = as + T::stage_a;
            bf16x8 ah[RB], al[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                if constexpr (ASTRIDED) {
                    ah[i] = read_strided<ROW>(as + aofs[i][0]);
                    al[i] = read_strided<ROW>(as + aofs[i][1]);
                } else {
                    ah[i] = *(const bf16x8 *)(as + alo + i * 2048);
                    al[i] = *(const bf16x8 *)(as + (alo ^ 64) + i * 2048);
                }
            }
#pragma unroll
            for (int j = 0; j < CAP; ++j) {
                const bf16x8 bh = *(const bf16x8 *)(bs + blo + j * (WB * 2048));
                const bf16x8 bl = *(const bf16x8 *)(bs + (blo ^ 64) + j * (WB * 2048));
#pragma unroll
                for (int i = 0; i < RB; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ah[i], bh, acc[i][j], 0, 0, 0);
#pragma unroll
                for (int i = 0; i < RB; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ah[i], bl, acc[i][j], 0, 0, 0);
#pragma unroll
                for (int i = 0; i < RB; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(al[i], bh, acc[i][j], 0, 0, 0);
            }
            slot = next(slot, 1);
        }
        // ---- results ----
        int m, a0, b0;
        find(t, m, a0, b0);
        const bool mirror = SYM && b0 >= a0 + T::TA;
        const int64_t ld = (int64_t)a.A * 2, mat = (int64_t)m * a.B * ld;
        // What is added to the sums of two blocks, the i-th and next of column j: loads without branches, two blocks ahead of the
        // stores that they may not pass.  Rows and columns past the matrix repeat its last ones, and their sums are not stored;
        // past X without padding rests are 0 (SINGLE loads read zeros past the matrix, and are masked like the others).
        struct Added {
            u32x2 hi[2], lo[2];
            uint32_t rest[2][SINGLE ? 4 : 2];
        } added[2];
        // the matrix's X and y: bytes from their first value fit 32 bits
        const char *const cm = (const char *)(a.c + mat);
        char *const ym = (char *)(a.y + (int64_t)m * a.r * a.cc);
        const uint32_t yb = a.tall ? 2 : 2 * (uint32_t)a.cc, yf = a.tall ? 2 * (uint32_t)a.r : 2;
        __amdgpu_buffer_rsrc_t yr;
        if constexpr (SINGLE) yr = buffer_of(ym, (int64_t)a.r * a.cc * 2);
        auto load_added = [&](int j, int i0, Added &in) __attribute__((always_inline)) {
            const int b = b0 + (j * WB + wm) * 16 + r15;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int f = a0 + wf * (RB * 16) + (i0 + i) * 16 + 4 * g;
                const char *at = cm + ((uint32_t)min(b, a.B - 1) * a.A * 4 + min(f & ~31, a.A - 32) * 4 + (f & 31) * 2);
                in.hi[i] = *(const u32x2 *)at;
                in.lo[i] = *(const u32x2 *)(at + 64);
                if (!UPDATE || !a.rest_in) continue;
                if constexpr (UPDATE && SINGLE) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        in.rest[i][q] = __builtin_amdgcn_raw_buffer_load_b16(yr, b * yb + f * yf + q * yf, 0, 0);
                } else if constexpr (UPDATE) {
                    const u32x2 w = *(const u32x2_any *)(ym + (min(b, a.r - 1) * yb + min(f, a.cc - 4) * 2));
                    in.rest[i][0] = w[0];
                    in.rest[i][1] = w[1];
                }
            }
        };
        // four rests of X's row b from column f on, as they were loaded
        auto rests = [&](const uint32_t *w, int b, int f, float (&v)[4]) __attribute__((always_inline)) {
            uint64_t u;
            if constexpr (SINGLE) {
                u = (uint64_t)(w[2] | w[3] << 16) << 32 | (w[0] | w[1] << 16);
            } else {
                u = (uint64_t)w[1] << 32 | w[0];
                const int past = f - min(f, a.cc - 4);
                u = past >= 4 ? 0 : u >> (16 * past);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] = a.rest_in && b < a.r && f + q < a.cc ? bf16_to_f32((uint16_t)(u >> (16 * q))) : 0.0f;
        };
        // four values of y: each by the lane that has read it
        auto y_store = [&](int b, int f, u32x2 w) __attribute__((always_inline)) {
            if constexpr (SINGLE) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(w[q >> 1] >> (16 * (q & 1))), yr,
                                                          b < a.r && f + q < a.cc ? b * yb + f * yf + q * yf : kNoOffset, 0, 0);
            } else if (b < a.r) {
                if (f + 4 <= a.cc) {
                    *(u32x2_any *)(ym + (b * yb + f * 2)) = w;
                    return;
                }
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    if (f + q < a.cc) *(uint16_t *)(ym + (b * yb + (f + q) * 2)) = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
            }
        };
        if (OP != ORTH_GRAM) load_added(0, 0, added[0]);
#pragma unroll
        for (int j = 0; j < CAP; ++j) {
            const int bb = b0 + (j * WB + wm) * 16, b = bb + r15;
#pragma unroll
            for (int i = 0; i < RB; i += 2) {
                const int f0 = a0 + wf * (RB * 16) + i * 16;           // a run of 32 values of a
                const int u = (j * RB + i) / 2;
                if (OP != ORTH_GRAM && u + 1 < CAP * RB / 2) load_added((i + 2) / RB + j, (i + 2) % RB, added[(u + 1) & 1]);
                const bool there = b < a.B && f0 < a.A;
                float v[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const Added &in = added[u & 1];
                    float rest[4] = {};
                    if constexpr (UPDATE) rests(in.rest[h], b, f0 + h * 16 + 4 * g, rest);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        v[h][q] = a.alpha * acc[i + h][j][q];
                        if constexpr (OP != ORTH_GRAM) {
                            const float hi = bf16_to_f32((uint16_t)(in.hi[h][q >> 1] >> (16 * (q & 1))));
                            const float lo = bf16_to_f32((uint16_t)(in.lo[h][q >> 1] >> (16 * (q & 1))));
                            v[h][q] += a.beta * (hi + lo + rest[q]);
                        }
                    }
                }
                if (UPDATE && a.last) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        y_store(b, f0 + h * 16 + 4 * g, u32x2{pack_bf16x2(v[h][0], v[h][1]), pack_bf16x2(v[h][2], v[h][3])});
                    continue;
                }
                float hi[2][4], lo[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) split_pair(v[h][q], hi[h][q], lo[h][q]);
                    if (UPDATE && a.rest_out)
                        y_store(b, f0 + h * 16 + 4 * g, u32x2{pack_bf16x2(rest_of(lo[h][0]), rest_of(lo[h][1])),
                                                              pack_bf16x2(rest_of(lo[h][2]), rest_of(lo[h][3]))});
                }
                const u32x4 oh = pair_bf16_value(hi[0], hi[1], lane), ol = pair_bf16_value(lo[0], lo[1], lane);
                if (there) {
                    uint16_t *row = a.out + mat + b * ld + f0 * 2 + pair_bf16_col(0, lane);
                    *(u32x4 *)row = oh;
                    *(u32x4 *)(row + 32) = ol;
                }
                if (mirror) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // the block [b][a] turned over in the wave's own LDS: lane 4 a + k then holds b = 4 k .. 4 k + 3
#pragma unroll
                        for (int q = 0; q < 4; ++q) turn[(4 * g + q) * 17 + r15] = pack_bf16x2(hi[h][q], lo[h][q]);
                        asm volatile("" ::: "memory");      // LDS serves a wave's writes and reads in order
                        uint32_t w[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) w[q] = turn[(lane >> 2) * 17 + (lane & 3) * 4 + q];
                        asm volatile("" ::: "memory");
                        const int f = f0 + h * 16 + (lane >> 2);
                        if (f < a.A && bb < a.B) {
                            uint16_t *row = a.out + mat + f * ld + (bb >> 5) * 64 + (bb & 31) + (lane & 3) * 4;
                            *(u32x2 *)row = u32x2{w[0] & 0xFFFF | w[1] << 16, w[2] & 0xFFFF | w[3] << 16};
                            *(u32x2 *)(row + 32) = u32x2{w[0] >> 16 | w[1] & 0xFFFF0000u, w[2] >> 16 | w[3] & 0xFFFF0000u};
                        }
                    }
                }
            }
        }
    }
}

template <void (*KERNEL)(OrthPass)>
hipError_t orth_launch(unsigned grid, int lds, const OrthPass &p, hipStream_t s) {
    static std::atomic<uint64_t> allowed{0};
    const hipError_t e = allow_lds((const void *)KERNEL, lds, allowed);
    if (e != hipSuccess) return e;
    KERNEL<<<grid, kOrthThreads, lds, s>>>(p);
    return hipGetLastError();
}

template <int OP>
hipError_t orth_product(const OrthPass &p, hipStream_t s) {
    const unsigned grid = (unsigned)((device_cus() + 7) / 8 * 8);
    switch (orth_variant(p.n, p.A, p.B, OP == ORTH_GRAM || OP == ORTH_SQUARE, grid)) {
        case kOrth256x256: return orth_launch<orth_kernel<OP, 4, 8, 4>>(grid, OrthTile<4, 8, 4>::lds, p, s);
        case kOrth256x128: return orth_launch<orth_kernel<OP, 4, 4, 4>>(grid, OrthTile<4, 4, 4>::lds, p, s);
        case kOrth128x128: return orth_launch<orth_kernel<OP, 2, 4, 4>>(grid, OrthTile<2, 4, 4>::lds, p, s);
        default: return orth_launch<orth_kernel<OP, 2, 1, 2>>(grid, OrthTile<2, 1, 2>::lds, p, s);
    }
}

}  // namespace

OrthSizes orth_sizes(int64_t n, int64_t rows, int64_t cols) {
    OrthSizes z{};
    z.tall = rows > cols;
    z.r = z.tall ? cols : rows;
    z.c = z.tall ? rows : cols;
    z.rp = (z.r + 31) / 32 * 32;
    z.cp = (z.c + 31) / 32 * 32;
    z.parts = (int)(z.r * z.c / 16384 + 1 < 64 ? z.r * z.c / 16384 + 1 : 64);
    z.x = (size_t)n * z.rp * z.cp * 4;
    z.s = (size_t)n * z.rp * z.rp * 4;
    z.norm = ((size_t)n * z.parts * 8 + 255) / 256 * 256;
    return z;
}

hipError_t launch_orthogonalize(const OrthProblem &q, hipStream_t s) {
    const OrthSizes z = orth_sizes(q.n, q.rows, q.cols);
    char *ws = (char *)q.ws;
    double *part = (double *)ws;
    ws += z.norm;
    uint16_t *x[2], *gram, *poly;
    auto take = [&](size_t bytes) { uint16_t *p = (uint16_t *)ws; ws += (bytes + 255) / 256 * 256; return p; };
    x[0] = take(z.x);
    x[1] = take(z.x);
    gram = take(z.s);
    poly = take(z.s);
    const int n = (int)q.n, r = (int)z.r, c = (int)z.c, rp = (int)z.rp, cp = (int)z.cp;
    const dim3 blocks((cp + 63) / 64, (rp + 63) / 64, n);
    // the largest factor by which the steps from k on multiply what rounding adds to X_k
    auto growth = [&](int k) {
        double by = 1.0;
        for (; k < q.steps; ++k) by *= fabs((double)q.coeffs[3 * k]);
        return by;
    };
    uint16_t *const rests = growth(0) > kRestGrowth ? (uint16_t *)q.y : nullptr;
    auto first = [&](auto dtc) {
        constexpr int D = decltype(dtc)::value;
        orth_norm_kernel<D><<<n * z.parts, kNormThreads, 0, s>>>(q.g, z.r * z.c, z.parts, part);
        if (z.tall) orth_first_kernel<D, true><<<blocks, 256, 0, s>>>(q.g, part, z.parts, q.eps, r, c, rp, cp, x[0], rests);
        else orth_first_kernel<D, false><<<blocks, 256, 0, s>>>(q.g, part, z.parts, q.eps, r, c, rp, cp, x[0], rests);
    };
    if (q.dt == DT_F32) first(std::integral_constant<int, DT_F32>{});
    else first(std::integral_constant<int, DT_BF16>{});
    hipError_t e = hipGetLastError();
    for (int k = 0; k < q.steps && e == hipSuccess; ++k) {
        const float *co = q.coeffs + 3 * k;
        OrthPass p{};
        p.n = n;
        p.A = p.B = rp;
        p.K = cp;
        p.a = p.b = x[k & 1];
        p.alpha = 1.0f;
        p.out = gram;
        e = orth_product<ORTH_GRAM>(p, s);
        if (e != hipSuccess) break;
        p.K = rp;
        p.a = p.b = p.c = gram;
        p.alpha = co[2];
        p.beta = co[1];
        p.out = poly;
        e = orth_product<ORTH_SQUARE>(p, s);
        if (e != hipSuccess) break;
        p.A = cp;
        p.a = p.c = x[k & 1];
        p.b = poly;
        const bool last = k == q.steps - 1;
        const float scale = last ? q.scale : 1.0f;
        p.alpha = scale;
        p.beta = co[0] * scale;
        p.out = x[(k + 1) & 1];
        p.y = (uint16_t *)q.y;
        p.last = last;
        p.rest_in = growth(k) > kRestGrowth;
        p.rest_out = !last && growth(k + 1) > kRestGrowth;
        p.r = r;
        p.cc = c;
        p.tall = z.tall;
        e = z.tall || z.c < 4 ? orth_product<ORTH_UPDATE_SINGLE>(p, s) : orth_product<ORTH_UPDATE>(p, s);
    }
    return e;
}

}  // namespace moe
