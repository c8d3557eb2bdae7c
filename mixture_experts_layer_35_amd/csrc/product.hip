// product.hip -- products of routed experts by themselves: y = W x for the rows of each expert in bf16 and in 8-bit
// integers, the gradient at x, the gradient at W, and the rounding of rows to 8-bit integers.
#include <atomic>
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "lds_ring.h"
#include "strided.h"
#include "tile_list.h"
#include "variants.h"

namespace moe {

namespace {

// out[b][a] = sum over k of A(a, k) B(b, k), a being the output's contiguous index:
//   product   a: features of W[e], k: inputs       b: rows of x   A's rows hold the reduction
//   dx        a: inputs,           k: features     b: rows of dy  the reduction runs over the rows of W[e]
//   dw        a: inputs,           k: rows of e    b: features    it runs over the rows of x and of dy
//
// A tile is 256 values of a against up to 256 of b.  The reduction is walked 128 bytes of a row (64 bf16, 128 integers) or
// 64 rows at a time through a ring of stages in LDS; products are 16x16x32 (bf16) and 16x16x64 (integers), A's values the
// row operand, so that a lane holds four consecutive outputs of one row.  Eight waves, 4 along a by 2 along b, the two
// taking 16-row blocks of b in turn.
constexpr int kTileA = 256;
constexpr int kProductThreads = 512;
constexpr int kProductStageA = kTileA * 128;
constexpr int kEndBytes = kMaxExperts * 4;

template <int CAP>
constexpr int product_slots() { return CAP <= 5 ? 3 : 2; }
template <int CAP>
constexpr int product_stage() { return kProductStageA + CAP * 4096; }
template <int CAP>
constexpr int product_lds() { return kEndBytes + product_slots<CAP>() * product_stage<CAP>(); }
static_assert(product_lds<4>() <= 160 * 1024 && product_lds<5>() <= 160 * 1024 && product_lds<8>() <= 160 * 1024, "LDS");

template <int DT>
struct Product;
template <>
struct Product<DT_BF16> {
    typedef bf16x8 frag;
    typedef f32x4 acc;
    static constexpr int esz = 2;
    __device__ static acc mma(frag a, frag b, acc c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};
template <>
struct Product<DT_I8> {
    typedef i32x4 frag;
    typedef i32x4 acc;
    static constexpr int esz = 1;
    __device__ static acc mma(frag a, frag b, acc c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0); }
};

// 16 bytes that lanes without data read.
__device__ const u32x4 product_zeros = {0, 0, 0, 0};

// Values e0 .. e0 + 7 of a bf16 row of `n` values at any address, zeros past its end.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
__device__ __forceinline__ u32x4 row_chunk(const uint16_t *row, int64_t e0, int64_t n) {
    if (e0 + 8 <= n) return *(const u32x4_any *)(row + e0);
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (e0 + k < n) v[k >> 1] |= (uint32_t)row[e0 + k] << (16 * (k & 1));
    return v;
}

template <int DT, int OP, int CAP, bool DIRECT>
__global__ __launch_bounds__(kProductThreads, 1) void product_kernel(const ProductPass a) {
    typedef Product<DT> P;
    constexpr int esz = P::esz, SLOTS = DIRECT ? product_slots<CAP>() : 2, STAGE = product_stage<CAP>();
    constexpr bool DW = OP == PRODUCT_DW, ASTRIDED = OP != PRODUCT_Y;
    constexpr int QB = CAP / 2 + CAP % 2;            // loads of B a wave issues for a step, at most
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    int32_t *const ends = (int32_t *)smem;
    char *const ring = smem + kEndBytes;
    for (int i = tid; i < a.n_exp; i += kProductThreads)
        ends[i] = (int)max((int64_t)0, min((int64_t)a.offsets[i + 1], a.max_rows));
    __syncthreads();
    const int atiles = (a.A + kTileA - 1) / kTileA, btiles = DW ? (a.B + 255) / 256 : 0;
    TileList list;
    int total;
    if (DW) {
        list.ends = ends;
        total = a.n_exp * atiles * btiles;
    } else {
        list.init(ends, a.n_exp, CAP * 32, atiles, lane);
        total = list.total;
    }
    // workgroup b runs on XCD b mod 8: each XCD takes a contiguous eighth of the list, so that tiles that share
    // operands meet in its L2
    const int per = (total + 7) / 8, xcd = blockIdx.x & 7;
    const int end = min(total, (xcd + 1) * per), first = xcd * per + (blockIdx.x >> 3), step = gridDim.x >> 3;
    if (first >= end) return;

    // tile t: expert, first value of a, first row (of the rows, or of dw's features) and their number
    auto find = [&](int t, int &e, int &a0, int &row0, int &valid) {
        if (DW) {
            e = t / (atiles * btiles);
            const int rest = t - e * (atiles * btiles), bt = rest / atiles;
            a0 = (rest - bt * atiles) * kTileA;
            row0 = bt * 256;
            valid = min(256, a.B - row0);
        } else {
            int ft;
            list.find(t, lane, e, ft, row0, valid);
            a0 = ft * kTileA;
        }
    };
    // reduction rows of expert e (dw) or the reduction's length
    auto first_of = [&](int e) { return __builtin_amdgcn_readfirstlane(list.start(e)); };
    auto rows_of = [&](int e) { return __builtin_amdgcn_readfirstlane(ends[e]) - first_of(e); };
    constexpr int KSTEP = 128 / esz;                  // of the reduction
    auto steps_of = [&](int e) { return DW ? max(1, (rows_of(e) + KSTEP - 1) / KSTEP) : (a.K + KSTEP - 1) / KSTEP; };

    // ---- loads: the tile and step that come next ----
    int it = first, ik = 0, isteps = 0, ie = 0, ia0 = 0, irow0 = 0, ivalid = 0;
    __amdgpu_buffer_rsrc_t ar;
    uint32_t avoff[4];
    const char *bptr[QB];
    // places in a stage: A's load q of the wave brings 1 KB to (wid * 4 + q) * 1024, B's to (q * 8 + wid) * 1024
    const int arow0 = wid * 32 + (lane >> 3);         // rows that hold the reduction: row of load q = 0
    const int ak0 = wid * 8 + (lane >> 5);            // rows of the reduction
    auto bytes_at = [&](int row) { return ((lane & 7) ^ swz<128>(row)) << 4; };           // within 128 bytes of a row
    auto values_at = [&](int k) { return ((lane & 31) ^ strided_slot(k)) * 8; };           // within 256 values
    auto aim = [&]() {
        find(it, ie, ia0, irow0, ivalid);
        isteps = steps_of(ie);
        if (!DW) {
            const char *base = (const char *)a.a + (int64_t)ie * a.a_mat * esz;
            const int n = min(kTileA, a.A - ia0);
            if (!ASTRIDED) {
                base += (int64_t)ia0 * a.a_ld * esz;
                ar = buffer_of(base, (int64_t)n * a.a_ld * esz);
            } else {
                ar = buffer_of(base, a.a_mat * esz);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (!ASTRIDED) {
                    const int row = arow0 + q * 8;
                    avoff[q] = row < n ? (uint32_t)((int64_t)row * a.a_ld * esz) + bytes_at(row) : kNoOffset;
                } else {
                    const int k = ak0 + q * 2, c = ia0 + values_at(k);
                    avoff[q] = c < a.A ? (uint32_t)(((int64_t)k * a.a_ld + c) * esz) : kNoOffset;
                }
            }
#pragma unroll
            for (int q = 0; q < QB; ++q) {
                // rows past the tile's repeat its last one; their results are not used
                const int row = (q * 8 + wid) * 8 + (lane >> 3);
                const int64_t R = irow0 + min(row, ivalid - 1);
                const int64_t token = a.gather ? (int64_t)a.gather[R] : R;
                bptr[q] = (const char *)a.b + token * a.b_ld * esz + bytes_at(row);
            }
        }
    };
    // A strided operand's 16 bytes of load q in step k (dw): row r of the reduction, values c .. c + 7
    auto dw_chunk = [&](int q, bool isA, const uint16_t *&row, int &c) {
        const int k = ak0 + q * 2, r = ik * 64 + k, m = rows_of(ie);
        const int64_t R = first_of(ie) + min(r, max(m - 1, 0));
        c = (isA ? ia0 : irow0) + values_at(k);
        row = nullptr;
        if (r < m && c < (isA ? a.A : a.B)) {
            const int64_t src = isA && a.gather ? (int64_t)a.gather[R] : R;
            row = isA ? (const uint16_t *)a.a + src * a.a_ld : (const uint16_t *)a.b + src * a.b_ld;
        }
    };
    const int64_t kbytes = (int64_t)a.K * esz;
    // issues a step's loads into a stage; the number of loads
    auto issue = [&](char *stage) {
        if (it >= end) return 0;
        if (ik == 0) aim();
        char *as = stage + wid * 4096, *bs = stage + kProductStageA + wid * 1024;
        int n = 4;
        if constexpr (DW) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint16_t *row;
                int c;
                dw_chunk(q, true, row, c);
                dma16(row ? (const void *)(row + c) : (const void *)&product_zeros, as + q * 1024);
                dw_chunk(q, false, row, c);
                dma16(row ? (const void *)(row + c) : (const void *)&product_zeros,
                      stage + kProductStageA + wid * 4096 + q * 1024);
            }
            n = 8;
        } else {
            const bool tail = ik == isteps - 1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t vo = avoff[q];
                if (!ASTRIDED) {
                    if (tail && (int64_t)ik * 128 + bytes_at(arow0 + q * 8) >= kbytes) vo = kNoOffset;
                    buffer_dma16(ar, vo, ik * 128, as + q * 1024);
                } else {
                    if (tail && ik * 64 + ak0 + q * 2 >= a.K) vo = kNoOffset;
                    buffer_dma16(ar, vo, (int)(ik * 64 * a.a_ld * esz), as + q * 1024);
                }
            }
            const int blocks = (ivalid + 31) >> 5;
#pragma unroll
            for (int q = 0; q < QB; ++q)
                if (q * 8 + wid < blocks * 4) {
                    const int at = bytes_at((q * 8 + wid) * 8 + (lane >> 3));
                    const void *src = bptr[q] + (int64_t)ik * 128;
                    if (tail && (int64_t)ik * 128 + at >= kbytes) src = &product_zeros;
                    dma16(src, bs + q * 8192);
                    ++n;
                }
        }
        if (++ik == isteps) {
            ik = 0;
            it += step;
        }
        return n;
    };
    // the same through registers, for rows that do not lie at multiples of 16 bytes
    u32x4 areg[4], breg[DW ? 4 : QB];
    int iblocks = 0;
    auto fetch = [&]() {
        iblocks = 0;
        if (it >= end) return;
        if (ik == 0) aim();
        if constexpr (DW) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint16_t *row;
                int c;
                dw_chunk(q, true, row, c);
                areg[q] = row ? row_chunk(row, c, a.A) : u32x4{0, 0, 0, 0};
                dw_chunk(q, false, row, c);
                breg[q] = row ? row_chunk(row, c, a.B) : u32x4{0, 0, 0, 0};
            }
            iblocks = 8;
        } else {
            const uint16_t *m = (const uint16_t *)a.a + (int64_t)ie * a.a_mat;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (!ASTRIDED) {
                    const int row = arow0 + q * 8;
                    areg[q] = ia0 + row < a.A ? row_chunk(m + (int64_t)(ia0 + row) * a.a_ld,
                                                          (int64_t)ik * 64 + bytes_at(row) / 2, a.K)
                                              : u32x4{0, 0, 0, 0};
                } else {
                    const int k = ak0 + q * 2;
                    areg[q] = ik * 64 + k < a.K ? row_chunk(m + (int64_t)(ik * 64 + k) * a.a_ld, ia0 + values_at(k), a.A)
                                                : u32x4{0, 0, 0, 0};
                }
            }
            iblocks = (ivalid + 31) >> 5;
#pragma unroll
            for (int q = 0; q < QB; ++q)
                if (q * 8 + wid < iblocks * 4) {
                    const int at = bytes_at((q * 8 + wid) * 8 + (lane >> 3)) / 2;
                    breg[q] = row_chunk((const uint16_t *)bptr[q] - at, (int64_t)ik * 64 + at, a.K);
                }
        }
        if (++ik == isteps) {
            ik = 0;
            it += step;
        }
    };
    auto put = [&](char *stage) {
        if (!iblocks) return;
        char *as = stage + wid * 4096 + lane * 16, *bs = stage + kProductStageA + lane * 16;
#pragma unroll
        for (int q = 0; q < 4; ++q) *(u32x4 *)(as + q * 1024) = areg[q];
        if constexpr (DW) {
#pragma unroll
            for (int q = 0; q < 4; ++q) *(u32x4 *)(bs + wid * 4096 + q * 1024) = breg[q];
        } else {
#pragma unroll
            for (int q = 0; q < QB; ++q)
                if (q * 8 + wid < iblocks * 4) *(u32x4 *)(bs + (q * 8 + wid) * 1024) = breg[q];
        }
    };

    // ---- products ----
    const int wf = wid >> 1, wm = wid & 1, r15 = lane & 15, g = lane >> 4;
    // lane offsets of the operands' 16-byte reads: sub-step 0; sub-step 1 is 64 bytes or 32 rows on
    const int arow = wf * 64 + r15, brow = wm * 16 + r15;
    const int alo = arow * 128 + ((g ^ swz<128>(arow)) << 4), blo = brow * 128 + ((g ^ swz<128>(brow)) << 4);
    int aofs[4], bofs[4];
    if (ASTRIDED) {
        const int jj = (lane >> 2) & 3, aa = lane & 3, k = 8 * g + jj;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ca = wf * 8 + i * 2 + (aa >> 1), cb = i * 4 + wm * 2 + (aa >> 1);
            aofs[i] = k * 512 + ((ca ^ strided_slot(k)) << 4) + 8 * (aa & 1);
            bofs[i] = k * 512 + ((cb ^ strided_slot(k)) << 4) + 8 * (aa & 1);
        }
    }
    int slot = 0, n1 = 0;
    auto next = [](int s) { return s + 1 == SLOTS ? 0 : s + 1; };
    auto tile = [&](auto tbc, int steps, int e, int a0, int row0, int valid) {
        constexpr int TB = decltype(tbc)::value;
        typename P::acc acc[4][TB] = {};
        for (int k = 0; k < steps; ++k) {
            // the stage's loads are done once only the later stages' are outstanding; past the barrier every wave's are, and
            // the stage before has been read
            if (DIRECT) {
                if (SLOTS == 3) wait_vmcnt_dyn(n1);
                else wait_vmcnt<0>();
            }
            wait_lgkm0();
            cta_barrier();
            if (DIRECT) n1 = issue(ring + (SLOTS == 3 ? next(next(slot)) : next(slot)) * STAGE);
            else fetch();
            const char *as = ring + slot * STAGE, *bs = as + kProductStageA;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                typename P::frag af[4], bf[TB];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (ASTRIDED) af[i] = read_strided<512>(as + aofs[i] + s * (32 * 512));
                    else af[i] = *(const typename P::frag *)(as + (alo ^ (s * 64)) + i * 2048);
                }
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    if constexpr (DW) bf[j] = read_strided<512>(bs + bofs[j & 3] + (j >> 2) * 256 + s * (32 * 512));
                    else bf[j] = *(const typename P::frag *)(bs + (blo ^ (s * 64)) + j * 4096);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < TB; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i][j] = P::mma(af[i], bf[j], acc[i][j]);
            }
            if (!DIRECT) put(ring + next(slot) * STAGE);
            slot = next(slot);
        }
        // ---- results ----
        const int f0 = a0 + wf * 64;
#pragma unroll
        for (int j = 0; j < TB; ++j) {
            const int b = (j * 2 + wm) * 16 + r15;
            const bool there = b < valid;
            float v[4][4];
            float sb = 1.0f;
            if constexpr (DT == DT_I8) {
                const int64_t R = row0 + min(b, valid - 1);
                sb = a.sb[a.gather ? (int64_t)a.gather[R] : R];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (DT == DT_I8) {
                        const int f = f0 + i * 16 + 4 * g + q;
                        v[i][q] = (float)acc[i][j][q] * sb * a.sa[(int64_t)e * a.A + min(f, a.A - 1)];
                    } else {
                        v[i][q] = acc[i][j][q];
                    }
                }
            const int64_t at = (DW ? ((int64_t)e * a.B + row0 + b) : (int64_t)row0 + b) * a.out_ld;
            if (a.out_f32) {
                float *row = (float *)a.out + at;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int f = f0 + i * 16 + 4 * g;
                    if (!there) continue;
                    if (a.wide && f < a.A) {
                        f32x4 o = {v[i][0], v[i][1], v[i][2], v[i][3]};
                        if (a.accumulate) o += *(const f32x4 *)(row + f);
                        *(f32x4 *)(row + f) = o;
                    } else if (!a.wide) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (f + q < a.A) row[f + q] = v[i][q] + (a.accumulate ? row[f + q] : 0.0f);
                    }
                }
            } else {
                uint16_t *row = (uint16_t *)a.out + at;
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    if (a.wide) {
                        const u32x4 o = pair_bf16_value(v[i], v[i + 1], lane);
                        const int f = pair_bf16_col(f0 + i * 16, lane);
                        if (there && f < a.A) *(u32x4 *)(row + f) = o;
                    } else if (there) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const int f = f0 + (i + h) * 16 + 4 * g + q;
                                if (f < a.A) row[f] = (uint16_t)pack_bf16x2(v[i + h][q], 0.0f);
                            }
                    }
                }
            }
        }
    };
    if (DIRECT) {
        issue(ring);
        if (SLOTS == 3) n1 = issue(ring + STAGE);
    } else {
        fetch();
        put(ring);
    }
    for (int t = first; t < end; t += step) {
        int e, a0, row0, valid;
        find(t, e, a0, row0, valid);
        const int steps = steps_of(e);
        auto run = [&](auto tb) { tile(tb, steps, e, a0, row0, valid); };
        using std::integral_constant;
        if (DW) {
            run(integral_constant<int, CAP>{});
        } else {
            const int blocks = (valid + 31) >> 5;
            if (blocks == 1) run(integral_constant<int, 1>{});
            else if (blocks == 2) run(integral_constant<int, 2>{});
            else if (CAP <= 4 && blocks == 3) run(integral_constant<int, 3>{});
            else if (CAP == 4 || blocks <= 4) run(integral_constant<int, 4>{});
            else if (CAP == 5 || blocks == 5) run(integral_constant<int, CAP < 5 ? CAP : 5>{});
            else if (blocks == 6) run(integral_constant<int, CAP < 6 ? CAP : 6>{});
            else run(integral_constant<int, CAP>{});
        }
    }
}

template <void (*KERNEL)(ProductPass)>
hipError_t product_launch(unsigned grid, int lds, const ProductPass &p, hipStream_t s) {
    static std::atomic<uint64_t> allowed{0};
    const hipError_t e = allow_lds((const void *)KERNEL, lds, allowed);
    if (e != hipSuccess) return e;
    KERNEL<<<grid, kProductThreads, lds, s>>>(p);
    return hipGetLastError();
}

// ---- rounding to 8-bit integers ----------------------------------------------

// A row's largest magnitude, then its codes; a wave takes a row.
template <int DT>
__global__ __launch_bounds__(256) void int8_quantize_kernel(const void *__restrict__ x, int64_t ld, int64_t rows, int cols,
                                                            int run, int8_t *__restrict__ q, float *__restrict__ s) {
    const int lane = threadIdx.x & 63;
    for (int64_t r = blockIdx.x * 4ll + (threadIdx.x >> 6); r < rows; r += gridDim.x * 4ll) {
        auto at = [&](int c) {
            return DT == DT_F32 ? ((const float *)x)[r * ld + c] : bf16_to_f32(((const uint16_t *)x)[r * ld + c]);
        };
        float top = 0.0f;
        bool bad = false;
        for (int c = lane; c < cols; c += 64) {
            const float v = fabsf(at(c));
            bad |= !(v <= 3.4028235e38f);
            top = fmaxf(top, v);
        }
        bad = __ballot(bad) != 0;
        top = fmaxf(wave_max_f32(top), 0x1p-100f);
        const float inv = bad ? 0.0f : 127.0f / top;
        for (int c = lane; c < run; c += 64)
            q[r * run + c] = c < cols && !bad ? (int8_t)(int)rintf(at(c) * inv) : (int8_t)0;
        if (lane == 0) s[r] = bad ? __uint_as_float(0x7FC00000u) : top / 127.0f;
    }
}

}  // namespace

hipError_t launch_product(int dt, int op, const ProductPass &p, hipStream_t s) {
    const unsigned grid = (unsigned)((device_cus() + 7) / 8 * 8);
    const int esz = dt == DT_I8 ? 1 : 2;
    auto aligned = [&](const void *ptr, int64_t ld) { return (uintptr_t)ptr % 16 == 0 && ld * esz % 16 == 0; };
    // loads of whole 16-byte pieces; a piece has to lie in its row
    const bool direct = aligned(p.a, p.a_ld) && aligned(p.b, p.b_ld) && p.a_mat * esz % 16 == 0 &&
                        (op == PRODUCT_DW ? p.A % 8 == 0 && p.B % 8 == 0
                                          : (int64_t)p.K * esz % 16 == 0 && (op == PRODUCT_Y || p.A % 8 == 0));
    const bool many = p.max_rows > 160ll * p.n_exp;
    if (op == PRODUCT_DW) {
        if (direct) return product_launch<product_kernel<DT_BF16, PRODUCT_DW, 8, true>>(grid, product_lds<8>(), p, s);
        return product_launch<product_kernel<DT_BF16, PRODUCT_DW, 8, false>>(grid, product_lds<8>(), p, s);
    }
    if (op == PRODUCT_DX) {
        if (!direct) return product_launch<product_kernel<DT_BF16, PRODUCT_DX, 4, false>>(grid, product_lds<4>(), p, s);
        if (many) return product_launch<product_kernel<DT_BF16, PRODUCT_DX, 8, true>>(grid, product_lds<8>(), p, s);
        return product_launch<product_kernel<DT_BF16, PRODUCT_DX, 4, true>>(grid, product_lds<4>(), p, s);
    }
    if (dt == DT_I8) {
        if (many) return product_launch<product_kernel<DT_I8, PRODUCT_Y, 8, true>>(grid, product_lds<8>(), p, s);
        return product_launch<product_kernel<DT_I8, PRODUCT_Y, 4, true>>(grid, product_lds<4>(), p, s);
    }
    if (!direct) return product_launch<product_kernel<DT_BF16, PRODUCT_Y, 4, false>>(grid, product_lds<4>(), p, s);
    if (many) return product_launch<product_kernel<DT_BF16, PRODUCT_Y, 8, true>>(grid, product_lds<8>(), p, s);
    return product_launch<product_kernel<DT_BF16, PRODUCT_Y, 4, true>>(grid, product_lds<4>(), p, s);
}

hipError_t launch_int8_quantize(int dt, const void *x, int64_t ld, int64_t rows, int cols, int8_t *q, float *sc,
                                hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const int run = (int)int8_row(cols);
    const unsigned grid = (unsigned)(rows < 65536 ? (rows + 3) / 4 : 16384);
    if (dt == DT_F32) int8_quantize_kernel<DT_F32><<<grid, 256, 0, s>>>(x, ld, rows, cols, run, q, sc);
    else int8_quantize_kernel<DT_BF16><<<grid, 256, 0, s>>>(x, ld, rows, cols, run, q, sc);
    return hipGetLastError();
}

}  // namespace moe
