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

// Values e0 .. e0 + 7 of a bf16 row of `n` values at any address, zeros past its end.  The load of a piece that ends past the row
// is moved back to the row's last eight values, which are then shifted: no lane branches around its load.
__device__ __forceinline__ u32x4 row_chunk(const uint16_t *row, int e0, int n) {
    if (n < 8) {
        u32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (e0 + k < n) v[k >> 1] |= (uint32_t)row[e0 + k] << (16 * (k & 1));
        return v;
    }
    const int e = min(e0, n - 8), d = min(e0 - e, 8);
    u32x4 v = *(const u32x4_any *)(row + e);
    if (d > 0) {
        uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
        if (d >= 4) {
            lo = d == 8 ? 0 : hi >> (16 * (d - 4));
            hi = 0;
        } else {
            lo = lo >> (16 * d) | hi << (64 - 16 * d);
            hi >>= 16 * d;
        }
        v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
    return v;
}

// Writes a wave's results: 16-value blocks of a from f0 on, 16-row blocks of b in turn with the other wave's.
template <int DT, int RB, int TB, bool DW, class Acc>
__device__ __forceinline__ void product_store(const ProductPass &a, const Acc (&acc)[RB][TB], int e, int f0, int row0,
                                              int valid, int wb, int lane) {
    const int r15 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < TB; ++j) {
        const int b = (j * 2 + wb) * 16 + r15;
        const bool there = b < valid;
        float v[RB][4];
        float sb = 1.0f;
        if constexpr (DT == DT_I8) {
            const int64_t R = row0 + min(b, valid - 1);
            sb = a.sb[a.gather ? (int64_t)a.gather[R] : R];
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
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
        // 16-byte stores at any address (the memory pipeline takes them); single values where a row ends within one
        if (a.out_f32) {
            float *row = (float *)a.out + at;
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                const int f = f0 + i * 16 + 4 * g;
                if (!there) continue;
                if (f + 4 <= a.A) {
                    f32x4 o = {v[i][0], v[i][1], v[i][2], v[i][3]};
                    if (DW && a.accumulate) o += *(const f32x4_any *)(row + f);
                    *(f32x4_any *)(row + f) = o;
                } else {
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        if (f + q < a.A) row[f + q] = v[i][q] + (DW && a.accumulate ? row[f + q] : 0.0f);
                }
            }
        } else {
            uint16_t *row = (uint16_t *)a.out + at;
#pragma unroll
            for (int i = 0; i < RB; i += 2) {
                const u32x4 o = pair_bf16_value(v[i], v[i + 1], lane);
                const int f = pair_bf16_col(f0 + i * 16, lane);
                if (!there) continue;
                if (f + 8 <= a.A) {
                    *(u32x4_any *)(row + f) = o;
                } else {
#pragma unroll
                    for (int q = 0; q < 7; ++q)
                        if (f + q < a.A) row[f + q] = (uint16_t)(o[q >> 1] >> (16 * (q & 1)));
                }
            }
        }
    }
}

template <int DT, int OP, int CAP, bool DIRECT>
__global__ __launch_bounds__(kProductThreads, 1) void product_kernel(const ProductPass a) {
    typedef Product<DT> P;
    constexpr int esz = P::esz, SLOTS = DIRECT ? product_slots<CAP>() : 2;
    constexpr bool DW = OP == PRODUCT_DW, ASTRIDED = OP != PRODUCT_Y;
    constexpr int STAGE = DW ? 2 * kProductStageA : product_stage<CAP>();
    static_assert(!DW || !DIRECT, "product_dw_kernel");
    constexpr int QB = CAP / 2 + CAP % 2;            // loads of B a wave issues for a step, at most
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    int32_t *const ends = (int32_t *)smem;
    char *const ring = smem + kEndBytes;
    const int filled = lds_place(ring);              // the ring for direct loads
    for (int i = tid; i < a.n_exp; i += kProductThreads)
        ends[i] = (int)max((int64_t)0, min((int64_t)a.offsets[i + 1], a.max_rows));
    __syncthreads();
    const int atiles = (a.A + kTileA - 1) / kTileA, btiles = DW ? (a.B + CAP * 32 - 1) / (CAP * 32) : 0;
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
    auto find = [&](int t, int &e, int &a0, int &row0, int &valid) __attribute__((always_inline)) {
        if (DW) {
            e = t / (atiles * btiles);
            const int rest = t - e * (atiles * btiles), bt = rest / atiles;
            a0 = (rest - bt * atiles) * kTileA;
            row0 = bt * (CAP * 32);
            valid = min(CAP * 32, a.B - row0);
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
    auto steps_of = [&](int e) __attribute__((always_inline)) {
        const int n = DW ? max(1, parts_of(rows_of(e), KSTEP)) : (a.K + KSTEP - 1) / KSTEP;
        return DIRECT ? n : (n + 1) & ~1;             // through registers in twos, the last one of zeros
    };

    // added to: an expert without rows keeps its values to the bit, so its tiles are passed over by loads and products alike
    auto kept = [&](int t) { return DW && a.accumulate && rows_of(t / (atiles * btiles)) <= 0; };

    // ---- loads: the tile and step that come next ----
    int it = first, ik = 0, isteps = 0, ie = 0, ia0 = 0, irow0 = 0, ivalid = 0;
    i32x4s ar;
    uint32_t avoff[4];
    const char *bptr[QB];
    // places in a stage: A's load q of the wave brings 1 KB to (wid * 4 + q) * 1024, B's to (q * 8 + wid) * 1024
    const int arow0 = wid * 32 + (lane >> 3);         // rows that hold the reduction: row of load q = 0
    const int ak0 = wid * 8 + (lane >> 5);            // rows of the reduction
    auto bytes_at = [&](int row) { return ((lane & 7) ^ swz<128>(row)) << 4; };           // within 128 bytes of a row
    auto values_at = [&](int k) { return ((lane & 31) ^ strided_slot(k)) * 8; };           // within 256 values
    auto aim = [&]() __attribute__((always_inline)) {
        find(it, ie, ia0, irow0, ivalid);
        isteps = steps_of(ie);
        if (!DW) {
            const char *base = (const char *)a.a + (int64_t)ie * a.a_mat * esz;
            const int n = min(kTileA, a.A - ia0);
            if (!ASTRIDED) {
                base += (int64_t)ia0 * a.a_ld * esz;
                ar = words_of(base, (int64_t)n * a.a_ld * esz);
            } else {
                ar = words_of(base, a.a_mat * esz);
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
                arrived(bptr[q]);
            }
        }
    };
    const int64_t kbytes = (int64_t)a.K * esz;
    // issues a step's loads into a stage; the number of loads
    auto issue = [&](int stage) __attribute__((always_inline)) {
        if (it >= end) return 0;
        if (ik == 0) aim();
        const int as = stage + wid * 4096, bs = stage + kProductStageA + wid * 1024;
        int n = 4;
        if constexpr (!DW) {
            const bool tail = ik == isteps - 1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t vo = avoff[q];
                if (!ASTRIDED) {
                    if (tail && (int64_t)ik * 128 + bytes_at(arow0 + q * 8) >= kbytes) vo = kNoOffset;
                    fill16(ar, vo, ik * 128, as + q * 1024);
                } else {
                    if (tail && ik * 64 + ak0 + q * 2 >= a.K) vo = kNoOffset;
                    fill16(ar, vo, (int)(ik * 64 * a.a_ld * esz), as + q * 1024);
                }
            }
            const int blocks = (ivalid + 31) >> 5;
#pragma unroll
            for (int q = 0; q < QB; ++q)
                if (q * 8 + wid < blocks * 4) {
                    const int at = bytes_at((q * 8 + wid) * 8 + (lane >> 3));
                    const void *src = bptr[q] + (int64_t)ik * 128;
                    if (tail && (int64_t)ik * 128 + at >= kbytes) src = &product_zeros;
                    fill16(src, bs + q * 8192);
                    ++n;
                }
        }
        if (++ik == isteps) {
            ik = 0;
            it += step;
        }
        return n;
    };
    // the same through registers, for rows that do not lie at multiples of 16 bytes: two sets, so that a step's loads have two
    // steps' time (4 rows to 4 experts of 6581 x 1793, the gradient at x: 79 us, with one set 141).  The second set does not quite
    // fit: the product spills 14 registers and the gradient at x 21, 60 and 88 bytes of scratch a lane
    u32x4 areg[2][4], breg[2][DW ? 4 : QB];
    int iblocks[2] = {0, 0};
    auto fetch = [&](auto setc) __attribute__((always_inline)) {
        constexpr int S = decltype(setc)::value;
        iblocks[S] = 0;
        if (DW && ik == 0)
            while (it < end && kept(it)) it += step;
        if (it >= end) return;
        if (ik == 0) aim();
        constexpr u32x4 none = {0, 0, 0, 0};
        if constexpr (DW) {
            const int m = rows_of(ie), lo = first_of(ie);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                areg[S][q] = breg[S][q] = none;
                if (ik * 64 + wid * 8 + q * 2 < m) {             // the load's first row, the same in all lanes
                    const int k = ak0 + q * 2, r = ik * 64 + k;
                    const int64_t R = lo + min(r, m - 1), src = a.gather ? (int64_t)a.gather[R] : R;
                    const u32x4 x = row_chunk((const uint16_t *)a.a + src * a.a_ld, ia0 + values_at(k), a.A);
                    const u32x4 y = row_chunk((const uint16_t *)a.b + R * a.b_ld, irow0 + values_at(k) % (CAP * 32), a.B);
                    areg[S][q] = r < m ? x : none;
                    breg[S][q] = r < m ? y : none;
                }
            }
            iblocks[S] = 8;
        } else {
            const uint16_t *m = (const uint16_t *)a.a + (int64_t)ie * a.a_mat;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (!ASTRIDED) {
                    const int row = arow0 + q * 8;
                    areg[S][q] = none;
                    if (ia0 + wid * 32 + q * 8 < a.A) {          // the load's first row, the same in all lanes
                        const uint16_t *from = m + (int64_t)min(ia0 + row, a.A - 1) * a.a_ld;
                        const u32x4 v = row_chunk(from, ik * 64 + bytes_at(row) / 2, a.K);
                        areg[S][q] = ia0 + row < a.A ? v : none;
                    }
                } else {
                    const int k = ik * 64 + ak0 + q * 2;
                    areg[S][q] = none;
                    if (ik * 64 + wid * 8 + q * 2 < a.K) {
                        const u32x4 v = row_chunk(m + (int64_t)min(k, a.K - 1) * a.a_ld, ia0 + values_at(ak0 + q * 2), a.A);
                        areg[S][q] = k < a.K ? v : none;
                    }
                }
            }
            iblocks[S] = (ivalid + 31) >> 5;
#pragma unroll
            for (int q = 0; q < QB; ++q)
                if (q * 8 + wid < iblocks[S] * 4) {
                    const int at = bytes_at((q * 8 + wid) * 8 + (lane >> 3)) / 2;
                    breg[S][q] = row_chunk((const uint16_t *)bptr[q] - at, ik * 64 + at, a.K);
                }
        }
        if (++ik == isteps) {
            ik = 0;
            it += step;
        }
    };
    auto put = [&](auto setc, char *stage) __attribute__((always_inline)) {
        constexpr int S = decltype(setc)::value;
        if (!iblocks[S]) return;
        char *as = stage + wid * 4096 + lane * 16, *bs = stage + kProductStageA + lane * 16;
#pragma unroll
        for (int q = 0; q < 4; ++q) *(u32x4 *)(as + q * 1024) = areg[S][q];
        if constexpr (DW) {
#pragma unroll
            for (int q = 0; q < 4; ++q) *(u32x4 *)(bs + wid * 4096 + q * 1024) = breg[S][q];
        } else {
#pragma unroll
            for (int q = 0; q < QB; ++q)
                if (q * 8 + wid < iblocks[S] * 4) *(u32x4 *)(bs + (q * 8 + wid) * 1024) = breg[S][q];
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
    auto tile = [&](auto tbc, int steps, int e, int a0, int row0, int valid) __attribute__((always_inline)) {
        constexpr int TB = decltype(tbc)::value;
        typename P::acc acc[4][TB] = {};
        auto products = [&]() __attribute__((always_inline)) {
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
        };
        if constexpr (DIRECT) {
            for (int k = 0; k < steps; ++k) {
                // the stage's loads are done once only the later stages' are outstanding; past the barrier every wave's are,
                // and the stage before has been read
                if (SLOTS == 3) wait_vmcnt_dyn(n1);
                else wait_vmcnt<0>();
                wait_lgkm0();
                cta_barrier();
                n1 = issue(filled + (SLOTS == 3 ? next(next(slot)) : next(slot)) * STAGE);
                products();
                slot = next(slot);
            }
        } else {
            using std::integral_constant;
            // past the barrier the slot is filled and the other one has been read; set p of registers goes to slot p
            for (int k = 0; k < steps; k += 2) {
                wait_lgkm0();
                cta_barrier();
                fetch(integral_constant<int, 0>{});
                products();
                put(integral_constant<int, 1>{}, ring + STAGE);
                slot = 1;
                wait_lgkm0();
                cta_barrier();
                fetch(integral_constant<int, 1>{});
                products();
                put(integral_constant<int, 0>{}, ring);
                slot = 0;
            }
        }
        product_store<DT, 4, TB, DW>(a, acc, e, a0 + wf * 64, row0, valid, wm, lane);
    };
    if (DIRECT) {
        issue(filled);
        if (SLOTS == 3) n1 = issue(filled + STAGE);
    } else {
        fetch(std::integral_constant<int, 0>{});
        put(std::integral_constant<int, 0>{}, ring);
        fetch(std::integral_constant<int, 1>{});
    }
    for (int t = first; t < end; t += step) {
        if (kept(t)) continue;
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

// dw for operands and results at multiples of 16 bytes.  A tile is 256 inputs by 256 features of one expert; the expert's rows
// are taken 32 at a time through a ring of four stages, of which three are under way (with two stages of 64 rows, whose gather
// indexes were vector loads that every load under way had to end for, 32 experts of 512 rows took 1165 us).  The rows' indexes
// come by scalar loads a stage ahead.  Results leave by stores without branches, so that their number is known: a stage's loads
// are waited for by counting what was issued behind them, and the stores of one tile drain under the next.  Tiles are listed in
// groups of 8 along a, so that the 32 of an XCD share 8 blocks of x and 4 of dy.  32 experts of 512 rows, 7168 by 2048: 845 us
// in fp32 (1.9 GB of results; 0.57 PFLOP/s), 664 in bf16, 1270 in fp32 added to what is there.
constexpr int kDwStage = 2 * 32 * 512;
constexpr int kDwSlots = 4;
constexpr int kDwLds = kEndBytes + kDwSlots * kDwStage;

template <bool ACCUMULATE>
__global__ __launch_bounds__(kProductThreads, 1) void product_dw_kernel(const ProductPass a) {
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    int32_t *const ends = (int32_t *)smem;
    const char *const ring = smem + kEndBytes;
    const int filled = lds_place(ring);              // the ring for direct loads
    for (int i = tid; i < a.n_exp; i += kProductThreads)
        ends[i] = (int)max((int64_t)0, min((int64_t)a.offsets[i + 1], a.max_rows));
    __syncthreads();
    const int atiles = (a.A + 255) / 256, btiles = (a.B + 255) / 256, total = a.n_exp * atiles * btiles;
    // workgroup b runs on XCD b mod 8: each XCD takes a contiguous eighth of the list
    const int per = (total + 7) / 8, xcd = blockIdx.x & 7;
    const int end = min(total, (xcd + 1) * per), first = xcd * per + (blockIdx.x >> 3), step = gridDim.x >> 3;
    if (first >= end) return;
    auto find = [&](int t, int &e, int &a0, int &b0) __attribute__((always_inline)) {
        e = __builtin_amdgcn_readfirstlane(t / (atiles * btiles));
        const int rest = t - e * (atiles * btiles), group = __builtin_amdgcn_readfirstlane(rest / (8 * btiles));
        const int in = rest - group * (8 * btiles), wide = min(8, atiles - group * 8);
        const int bt = __builtin_amdgcn_readfirstlane(in / wide);
        a0 = (group * 8 + in - bt * wide) * 256;
        b0 = bt * 256;
    };
    auto start_of = [&](int e) { return e ? __builtin_amdgcn_readfirstlane(ends[e - 1]) : 0; };
    auto rows_of = [&](int e) { return max(0, __builtin_amdgcn_readfirstlane(ends[e]) - start_of(e)); };
    // an expert without rows takes one step of zeros, or none: added to, it keeps its values to the bit, so its tiles are passed
    // over by loads and products alike
    auto kept = [&](int t) {
        return ACCUMULATE && rows_of(__builtin_amdgcn_readfirstlane(t / (atiles * btiles))) == 0;
    };
    auto steps_of = [&](int rows) { return max(1, parts_of(rows, 32)); };

    // ---- loads: the tile and step that come next, and the rows of x that this wave's loads of it bring ----
    const int k0 = wid * 4 + (lane >> 5);             // the lane's row of a step, in load 0; load 1 is two on
    int it = first, ik = 0, isteps = 0, lo = 0, rows = 0, index[4] = {0, 0, 0, 0};
    int64_t aoff[2], boff[2];                         // bytes within rows; -1: past the row's values
    auto look = [&]() __attribute__((always_inline)) {
        if (ik == 0)
            while (it < end && kept(it)) it += step;
        if (it >= end) return;
        if (ik == 0) {
            int e, a0, b0;
            find(it, e, a0, b0);
            lo = start_of(e);
            rows = rows_of(e);
            isteps = steps_of(rows);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int c = ((lane & 31) ^ strided_slot(k0 + q * 2)) * 8;
                aoff[q] = a0 + c < a.A ? (a0 + c) * 2ll : -1;
                boff[q] = b0 + c < a.B ? (b0 + c) * 2ll : -1;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = lo + min(ik * 32 + wid * 4 + i, rows - 1);
            index[i] = rows > 0 && a.gather ? scalar_load(a.gather, r) : r;
        }
    };
    int ops = 0;                                      // vector memory instructions so far
    auto issue = [&](int stage) __attribute__((always_inline)) {
        if (it >= end) return;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = ik * 32 + k0 + q * 2;
            const bool there = r < rows;
            const int64_t xrow = lane >> 5 ? index[q * 2 + 1] : index[q * 2];
            const char *x = (const char *)a.a + xrow * a.a_ld * 2 + aoff[q];
            const char *y = (const char *)a.b + (int64_t)((uint32_t)lo + (uint32_t)r) * a.b_ld * 2 + boff[q];
            fill16(there && aoff[q] >= 0 ? x : (const char *)&product_zeros, stage + wid * 2048 + q * 1024);
            fill16(there && boff[q] >= 0 ? y : (const char *)&product_zeros, stage + kDwStage / 2 + wid * 2048 + q * 1024);
        }
        ops += 4;
        if (++ik == isteps) {
            ik = 0;
            it += step;
        }
        look();
    };

    const int wf = wid >> 1, wm = wid & 1, r15 = lane & 15, g = lane >> 4;
    int aofs[4], bofs[4];
    {
        const int jj = (lane >> 2) & 3, aa = lane & 3, k = 8 * g + jj;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ca = wf * 8 + i * 2 + (aa >> 1), cb = i * 4 + wm * 2 + (aa >> 1);
            aofs[i] = k * 512 + ((ca ^ strided_slot(k)) << 4) + 8 * (aa & 1);
            bofs[i] = k * 512 + ((cb ^ strided_slot(k)) << 4) + 8 * (aa & 1) + kDwStage / 2;
        }
    }
    look();
    int slot = 0, mark[kDwSlots - 1];                 // `ops` behind the loads of the steps that come
#pragma unroll
    for (int i = 0; i < kDwSlots - 1; ++i) {
        issue(filled + i * kDwStage);
        mark[i] = ops;
    }
    for (int t = first; t < end; t += step) {
        if (kept(t)) continue;
        int e, a0, b0;
        find(t, e, a0, b0);
        const int steps = steps_of(rows_of(e));
        f32x4 acc[4][8] = {};
        for (int k = 0; k < steps; ++k) {
            wait_vmcnt_dyn(ops - mark[0]);
            wait_lgkm0();
            cta_barrier();
            // past the barrier every wave's loads of the stage are done, and the stage before has been read
            issue(filled + ((slot + kDwSlots - 1) & (kDwSlots - 1)) * kDwStage);
            mark[0] = mark[1];
            mark[1] = mark[2];
            mark[2] = ops;
            const char *st = ring + slot * kDwStage;
            bf16x8 af[4], bf[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) af[i] = read_strided<512>(st + aofs[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) bf[j] = read_strided<512>(st + bofs[j & 3] + (j >> 2) * 256);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = Product<DT_BF16>::mma(af[i], bf[j], acc[i][j]);
            slot = (slot + 1) & (kDwSlots - 1);
        }
        const int f0 = a0 + wf * 64, osz = a.out_f32 ? 4 : 2, valid = min(256, a.B - b0);
        const __amdgpu_buffer_rsrc_t out =
            buffer_of((const char *)a.out + ((int64_t)e * a.B + b0) * a.A * osz, (int64_t)valid * a.A * osz);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int b = (j * 2 + wm) * 16 + r15;
            const uint32_t row = b < valid ? (uint32_t)(b * a.A * osz) : kNoOffset;
            if (a.out_f32) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int f = f0 + i * 16 + 4 * g;
                    const uint32_t at = f < a.A ? row + f * 4 : kNoOffset;
                    f32x4 v = acc[i][j];
                    if (ACCUMULATE) v += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(out, at, 0, 0));
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), out, at, 0, 0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const float va[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                    const float vb[4] = {acc[i + 1][j][0], acc[i + 1][j][1], acc[i + 1][j][2], acc[i + 1][j][3]};
                    const int f = pair_bf16_col(f0 + i * 16, lane);
                    __builtin_amdgcn_raw_buffer_store_b128(pair_bf16_value(va, vb, lane), out,
                                                           f < a.A ? row + f * 2 : kNoOffset, 0, 0);
                }
            }
        }
        ops += a.out_f32 ? 32 : 16;
    }
}

// Few tiles: a single token to its experts, small matrices.  Bound by the time from one load to the next, so the work is cut
// finely: a tile is 64 values of a by up to 8 rows of b, and the four waves of a workgroup share it, each a quarter of the steps,
// which pass through a ring in LDS of the wave's own without barriers.  The sums meet in LDS, in the order of the waves.
// One token, 8 experts of 7168 x 2048 (235 MB): 43 us with other experts in each call (36 with the same ones, whose weights the
// last cache then holds in part), 69 in tiles of 256 by 160 rows.
constexpr int kStreamThreads = 256;
constexpr int kStreamRows = product_rows(kProductStream);
constexpr int kStreamStageA = 64 * 128, kStreamStage = kStreamStageA + kStreamRows * 128, kStreamSlots = 4;
constexpr int kStreamParts = 3 * 4 * 64 * 16;
constexpr int kStreamLds = kEndBytes + 4 * kStreamSlots * kStreamStage + kStreamParts;
static_assert(kStreamLds <= 160 * 1024, "LDS");

// rows of 128 bytes: as strided_slot, with the row's lowest bit in the place of the 128
__device__ __forceinline__ int stream_slot(int k) { return 2 * (((k >> 1) & 1) | (((k >> 3) & 1) << 1)); }

template <int DT, bool ASTRIDED>
__global__ __launch_bounds__(kStreamThreads, 1) void product_stream_kernel(const ProductPass a) {
    typedef Product<DT> P;
    typedef typename P::frag frag;
    constexpr int esz = P::esz;
    extern __shared__ __align__(1024) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    int32_t *const ends = (int32_t *)smem;
    const char *const ring = smem + kEndBytes + wid * (kStreamSlots * kStreamStage);
    const int filled = lds_place(ring);
    u32x4 *const parts = (u32x4 *)(smem + kEndBytes + 4 * kStreamSlots * kStreamStage);
    for (int i = tid; i < a.n_exp; i += kStreamThreads)
        ends[i] = (int)max((int64_t)0, min((int64_t)a.offsets[i + 1], a.max_rows));
    __syncthreads();
    TileList list;
    list.init(ends, a.n_exp, kStreamRows, (a.A + 63) / 64, lane);
    const int steps = (int)(((int64_t)a.K * esz + 127) / 128), part = (int)((int64_t)a.K * esz % 128);
    const int klo = steps * wid / 4, khi = steps * (wid + 1) / 4;

    // ---- loads: the tile and step that come next ----
    int it = blockIdx.x, ik = klo;
    i32x4s ar = {};
    uint32_t avoff[8];
    const char *brow = nullptr;
    const int piece = ((lane & 7) ^ swz<128>(lane >> 3)) << 4;
    int ops = 0;
    auto issue = [&](int stage) __attribute__((always_inline)) {
        if (it >= list.total || klo >= khi) return;
        if (ik == klo) {
            int e, ft, row0, valid;
            list.find(it, lane, e, ft, row0, valid);
            const int a0 = ft * 64;
            const char *base = (const char *)a.a + (int64_t)e * a.a_mat * esz;
            if (!ASTRIDED) ar = words_of(base + (int64_t)a0 * a.a_ld * esz, (int64_t)min(64, a.A - a0) * a.a_ld * esz);
            else ar = words_of(base, a.a_mat * esz);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int row = q * 8 + (lane >> 3);
                if (!ASTRIDED) {
                    avoff[q] = a0 + row < a.A ? (uint32_t)((int64_t)row * a.a_ld * esz) + piece : kNoOffset;
                } else {
                    const int c = a0 + ((lane & 7) ^ stream_slot(row)) * 8;
                    avoff[q] = c < a.A ? (uint32_t)(((int64_t)row * a.a_ld + c) * esz) : kNoOffset;
                }
            }
            // rows past the tile's repeat its last one; their results are not used
            int token = row0 + min(lane >> 3, valid - 1);
            if (a.gather) token = a.gather[token];
            brow = (const char *)a.b + (int64_t)token * a.b_ld * esz + piece;
            arrived(brow);
        }
        const bool tail = part && ik == steps - 1;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            uint32_t vo = avoff[q];
            if (!ASTRIDED) {
                if (tail) vo = piece >= part ? kNoOffset : vo;
                fill16(ar, vo, ik * 128, stage + q * 1024);
            } else {
                if (tail) vo = ik * 64 + q * 8 + (lane >> 3) >= a.K ? kNoOffset : vo;
                fill16(ar, vo, (int)(ik * 64 * a.a_ld * esz), stage + q * 1024);
            }
        }
        const char *src = brow + (int64_t)ik * 128;
        if (tail) src = piece >= part ? (const char *)&product_zeros : src;
        fill16(src, stage + kStreamStageA);
        ops += 9;
        if (++ik == khi) {
            ik = klo;
            it += gridDim.x;
        }
    };

    const int r15 = lane & 15, g = lane >> 4, row8 = r15 & (kStreamRows - 1);
    const int alo = r15 * 128 + ((g ^ swz<128>(r15)) << 4), blo = kStreamStageA + row8 * 128 + ((g ^ swz<128>(row8)) << 4);
    int aofs[4];
    {
        const int jj = (lane >> 2) & 3, aa = lane & 3, k = 8 * g + jj;
#pragma unroll
        for (int i = 0; i < 4; ++i) aofs[i] = k * 128 + (((i * 2 + (aa >> 1)) ^ stream_slot(k)) << 4) + 8 * (aa & 1);
    }
    int slot = 0, mark[kStreamSlots - 1];
#pragma unroll
    for (int i = 0; i < kStreamSlots - 1; ++i) {
        issue(filled + i * kStreamStage);
        mark[i] = ops;
    }
    for (int t = blockIdx.x; t < list.total; t += gridDim.x) {
        typename P::acc acc[4][1] = {};
        for (int k = klo; k < khi; ++k) {
            // the step's loads are done once only those behind them are outstanding; the slot before has been read
            wait_vmcnt_dyn(ops - mark[0]);
            asm volatile("" ::: "memory");
            issue(filled + ((slot + kStreamSlots - 1) & (kStreamSlots - 1)) * kStreamStage);
            mark[0] = mark[1];
            mark[1] = mark[2];
            mark[2] = ops;
            const char *st = ring + slot * kStreamStage;
            frag af[2][4], bf[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (ASTRIDED) af[s][i] = read_strided<128>(st + aofs[i] + s * (32 * 128));
                    else af[s][i] = *(const frag *)(st + (alo ^ (s * 64)) + i * 2048);
                }
                bf[s] = *(const frag *)(st + (blo ^ (s * 64)));
            }
            wait_lgkm0();
            asm volatile("" ::: "memory");
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][0] = P::mma(af[s][i], bf[s], acc[i][0]);
            slot = (slot + 1) & (kStreamSlots - 1);
        }
        cta_barrier();                                // the previous tile's sums have been read
        if (wid > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) parts[((wid - 1) * 4 + i) * 64 + lane] = __builtin_bit_cast(u32x4, acc[i][0]);
        }
        wait_lgkm0();
        cta_barrier();
        if (wid > 0) continue;
#pragma unroll
        for (int w = 0; w < 3; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i][0] += __builtin_bit_cast(typename P::acc, parts[(w * 4 + i) * 64 + lane]);
        int e, ft, row0, valid;
        list.find(t, lane, e, ft, row0, valid);
        product_store<DT, 4, 1, false>(a, acc, e, ft * 64, row0, valid, 0, lane);
    }
}

template <void (*KERNEL)(ProductPass)>
hipError_t product_launch(unsigned grid, int threads, int lds, const ProductPass &p, hipStream_t s) {
    static std::atomic<uint64_t> allowed{0};
    const hipError_t e = allow_lds((const void *)KERNEL, lds, allowed);
    if (e != hipSuccess) return e;
    KERNEL<<<grid, threads, lds, s>>>(p);
    return hipGetLastError();
}

// ---- rounding to 8-bit integers ----------------------------------------------

// A row's largest magnitude, then its codes.  WAVES waves take a row, eight values a lane at a time; up to four times eight stay
// in registers between the two, longer rows are read again.  By one wave and by four: 4096 rows of 512 4.5 and 8.8 us, of 2048
// 5.3 and 9.7, of 4096 9.8 and 12.2, of 7168 20.2 and 17.3; 64 rows of 4096 5.2 and 4.6, of 7168 8.0 and 4.6 (4.5 is the host's
// call).  One wave takes what it can hold: up to 2048 values.
constexpr int kInt8Held = 4;

template <int DT, int WAVES>
__global__ __launch_bounds__(256) void int8_quantize_kernel(const void *__restrict__ x, int64_t ld, int64_t rows, int cols,
                                                            int run, int8_t *__restrict__ q, float *__restrict__ s) {
    constexpr int ROWS = 4 / WAVES, LANES = WAVES * 64;
    __shared__ float tops[4];
    const int in = threadIdx.x % LANES, wave = threadIdx.x >> 6;
    for (int64_t r0 = blockIdx.x * (int64_t)ROWS; r0 < rows; r0 += gridDim.x * (int64_t)ROWS) {
        const int64_t r = r0 + threadIdx.x / LANES;
        const bool there = r < rows;
        float held[kInt8Held][8];
        // the largest magnitude as bits: those of an infinity or NaN are larger than any number's
        uint32_t top = __float_as_uint(0x1p-100f);
        auto look = [&](const float (&v)[8]) {
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7FFFFFFFu);
        };
#pragma unroll
        for (int i = 0; i < kInt8Held; ++i) {
            const int c = (i * LANES + in) * 8;
            load8<DT>(x, r * ld + c, there ? min(8, cols - c) : 0, held[i]);
            look(held[i]);
        }
        for (int c = (kInt8Held * LANES + in) * 8; there && c < cols; c += LANES * 8) {
            float v[8];
            load8<DT>(x, r * ld + c, cols - c, v);
            look(v);
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m, kWave));
        if (WAVES > 1) {
            __syncthreads();                        // the row before has been read
            tops[wave] = __uint_as_float(top);
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WAVES; ++w) top = max(top, __float_as_uint(tops[w]));
        }
        if (!there) continue;
        const bool bad = top >= 0x7F800000u;
        const float most = __uint_as_float(top), inv = 127.0f / most;
        auto codes = [&](const float (&v)[8], int c) {
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k >> 2] |= ((uint32_t)(int)rintf(v[k] * inv) & 0xFFu) << (8 * (k & 3));
            if (c < run) *(u32x2 *)(q + r * run + c) = bad ? u32x2{0, 0} : u32x2{w[0], w[1]};
        };
#pragma unroll
        for (int i = 0; i < kInt8Held; ++i) codes(held[i], (i * LANES + in) * 8);
        for (int c = (kInt8Held * LANES + in) * 8; c < run; c += LANES * 8) {
            float v[8];
            load8<DT>(x, r * ld + c, cols - c, v);
            codes(v, c);
        }
        if (in == 0) s[r] = bad ? __uint_as_float(0x7FC00000u) : most / 127.0f;
    }
}

}  // namespace

constexpr int kDwAnyLds = kEndBytes + 2 * 2 * kProductStageA;   // both operands' stages hold 256 values a row

hipError_t launch_product(int dt, int op, const ProductPass &p, hipStream_t s) {
    using std::integral_constant;
    const int64_t cus = device_cus();
    const unsigned grid = (unsigned)((cus + 7) / 8 * 8);
    const int esz = dt == DT_I8 ? 1 : 2;
    auto aligned = [&](const void *ptr, int64_t ld) { return (uintptr_t)ptr % 16 == 0 && ld * esz % 16 == 0; };
    // loads of whole 16-byte pieces: a piece has to lie in its row
    const bool pieces = aligned(p.a, p.a_ld) && aligned(p.b, p.b_ld) && p.a_mat * esz % 16 == 0 &&
                        (op == PRODUCT_DW ? p.A % 8 == 0 && p.B % 8 == 0
                                          : (int64_t)p.K * esz % 16 == 0 && (op == PRODUCT_Y || p.A % 8 == 0));
    if (op == PRODUCT_DW) {
        if (pieces && p.wide)
            return p.accumulate ? product_launch<product_dw_kernel<true>>(grid, kProductThreads, kDwLds, p, s)
                                : product_launch<product_dw_kernel<false>>(grid, kProductThreads, kDwLds, p, s);
        return product_launch<product_kernel<DT_BF16, PRODUCT_DW, 4, false>>(grid, kProductThreads, kDwAnyLds, p, s);
    }
    auto of = [&](auto dtc, auto opc) {
        constexpr int D = decltype(dtc)::value, O = decltype(opc)::value;
        switch (product_variant(p.max_rows, p.n_exp, p.A, pieces, cus)) {
            case kProductStream:
                return product_launch<product_stream_kernel<D, O == PRODUCT_DX>>(grid, kStreamThreads, kStreamLds, p, s);
            case kProduct160:
                return product_launch<product_kernel<D, O, 5, true>>(grid, kProductThreads, product_lds<5>(), p, s);
            case kProduct256:
                return product_launch<product_kernel<D, O, 8, true>>(grid, kProductThreads, product_lds<8>(), p, s);
            default:
                // codes of 8 bits always lie in pieces
                if constexpr (D == DT_I8) return hipErrorInvalidValue;
                else return product_launch<product_kernel<D, O, 4, false>>(grid, kProductThreads, product_lds<4>(), p, s);
        }
    };
    if (dt == DT_I8) return of(integral_constant<int, DT_I8>{}, integral_constant<int, PRODUCT_Y>{});
    if (op == PRODUCT_DX) return of(integral_constant<int, DT_BF16>{}, integral_constant<int, PRODUCT_DX>{});
    return of(integral_constant<int, DT_BF16>{}, integral_constant<int, PRODUCT_Y>{});
}

hipError_t launch_int8_quantize(int dt, const void *x, int64_t ld, int64_t rows, int cols, int8_t *q, float *sc,
                                hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const int run = (int)int8_row(cols);
    auto launch = [&](auto dtc, auto waves) {
        constexpr int D = decltype(dtc)::value, W = decltype(waves)::value;
        const int64_t groups = (rows * W + 3) / 4;
        int8_quantize_kernel<D, W><<<(unsigned)(groups < 65536 ? groups : 65536), 256, 0, s>>>(x, ld, rows, cols, run, q, sc);
        return hipGetLastError();
    };
    using std::integral_constant;
    auto of = [&](auto dtc) {
        return cols <= 512 * kInt8Held ? launch(dtc, integral_constant<int, 1>{}) : launch(dtc, integral_constant<int, 4>{});
    };
    return dt == DT_F32 ? of(integral_constant<int, DT_F32>{}) : of(integral_constant<int, DT_BF16>{});
}

}  // namespace moe
