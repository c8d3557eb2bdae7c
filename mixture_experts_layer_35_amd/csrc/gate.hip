// gate.hip -- routing from logits: softmax or sigmoid scores, a bias for balance,
// groups, top-K, renormalised weights ("DeepSeek-V3 Technical Report", §2.1.2, for the
// sigmoid form), and the gradient of the weights at the logits.
//
// A token belongs to L lanes of a wave, lane l holding experts l*V .. l*V + V-1 in
// registers, so that lane order is index order and a tie's lower index is the lower lane.
#include <type_traits>

#include "common.h"
#include "internal.h"
#include "variants.h"

// A product and a sum that the definition rounds one after the other stay two roundings.
#pragma clang fp contract(off)

namespace moe {

namespace {

constexpr int kGateThreads = 256;
constexpr int kMaxK = 32;   // slots of a token, at most

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// v combined over the L lanes of a token, in all of them.  Steps inside a row of 16 lanes are DPP
// moves, the two across rows lane swaps, so no step goes through LDS.
template <int L, class Op>
__device__ __forceinline__ uint32_t lanes_reduce(uint32_t v, Op op) {
    auto dpp = [](uint32_t x, auto ctrl) {
        return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, decltype(ctrl)::value, 0xF, 0xF, false);
    };
    v = op(v, dpp(v, std::integral_constant<int, 0xB1>{}));               // lane ^ 1
    v = op(v, dpp(v, std::integral_constant<int, 0x4E>{}));               // lane ^ 2
    if (L >= 8) v = op(v, dpp(v, std::integral_constant<int, 0x141>{}));  // the other quad of 8
    if (L >= 16) v = op(v, dpp(v, std::integral_constant<int, 0x140>{})); // the other half of 16
    if (L >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    if (L >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(r[0], r[1]);
    }
    return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    return lanes_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
    return __uint_as_float(lanes_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    return __uint_as_float(lanes_reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
// The same steps on both halves of a double.
template <int L>
__device__ __forceinline__ double lanes_sum(double v) {
    auto dpp = [](double x, auto ctrl) {
        const u32x2 h = __builtin_bit_cast(u32x2, x);
        const u32x2 o = {(uint32_t)__builtin_amdgcn_update_dpp((int)h[0], (int)h[0], decltype(ctrl)::value, 0xF, 0xF, false),
                         (uint32_t)__builtin_amdgcn_update_dpp((int)h[1], (int)h[1], decltype(ctrl)::value, 0xF, 0xF, false)};
        return __builtin_bit_cast(double, o);
    };
    v += dpp(v, std::integral_constant<int, 0xB1>{});
    v += dpp(v, std::integral_constant<int, 0x4E>{});
    if (L >= 8) v += dpp(v, std::integral_constant<int, 0x141>{});
    if (L >= 16) v += dpp(v, std::integral_constant<int, 0x140>{});
    if (L >= 32) {
        const u32x2 h = __builtin_bit_cast(u32x2, v);
        const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
        v = __builtin_bit_cast(double, u32x2{lo[0], hi[0]}) + __builtin_bit_cast(double, u32x2{lo[1], hi[1]});
    }
    if (L >= 64) {
        const u32x2 h = __builtin_bit_cast(u32x2, v);
        const auto lo = __builtin_amdgcn_permlane32_swap(h[0], h[0], false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap(h[1], h[1], false, false);
        v = __builtin_bit_cast(double, u32x2{lo[0], hi[0]}) + __builtin_bit_cast(double, u32x2{lo[1], hi[1]});
    }
    return v;
}

// A token's lanes lie in one wave, whose LDS accesses run in order: what they wrote is there for
// what they read next, and only the compiler has to keep the order.
__device__ __forceinline__ void token_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Order of choice values (never -0: a score is not) as unsigned integers; 0 stands below all of them.
__device__ __forceinline__ uint32_t choice_key(float c) {
    const uint32_t b = __float_as_uint(c);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
constexpr uint32_t kKeyNone = 0x007FFFFFu;   // choice_key(-infinity)
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// An expert is in use unless its logit is -infinity or NaN.
__device__ __forceinline__ bool in_use(float z) { return z > neg_inf(); }
__device__ __forceinline__ float sigmoid_score(float z) { return in_use(z) ? 1.0f / (1.0f + expf(-z)) : 0.0f; }
// exp(z - m) of a softmax whose largest logit in use is m (m itself may be +infinity).
__device__ __forceinline__ float softmax_exp(float z, float m) {
    return !in_use(z) ? 0.0f : z == m ? 1.0f : expf(z - m);
}

// sigmoid_score of V logits, the same bits.  With r within one ulp of 1/d, r + r (1 - d r) is 1/d
// correctly rounded (Markstein); tried against the division at every float d >= 1 it fails only above
// 2^126, where r itself is no normal number.  A third of the division's instructions, where all lanes of the wave have
// logits above -87: experts out of use, and lanes' places past E, count as -infinity and take the division.
template <int V>
__device__ __forceinline__ void sigmoid_scores(const float (&z)[V], float (&s)[V]) {
    float top = 0.0f;
#pragma unroll
    for (int r = 0; r < V; ++r) {
        s[r] = 1.0f + expf(-(in_use(z[r]) ? z[r] : neg_inf()));
        top = fmaxf(top, s[r]);
    }
    if (__any(top > 0x1p126f)) {
#pragma unroll
        for (int r = 0; r < V; ++r) s[r] = 1.0f / s[r];
    } else {
#pragma unroll
        for (int r = 0; r < V; ++r) {
            const float q = __builtin_amdgcn_rcpf(s[r]);
            s[r] = __builtin_fmaf(__builtin_fmaf(-s[r], q, 1.0f), q, q);
        }
    }
}

template <int DT>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    return DT == DT_F32 ? ((const float *)p)[i] : bf16_to_f32(((const uint16_t *)p)[i]);
}

// A lane's V values of a row of n, four at a time: chunk r of lane l starts at chunk_at<L, V, SPREAD>(l, r).  In
// order (a lane's values are neighbours), or spread (the lanes' chunks are, which the memory pipeline likes
// better).  `fill` past element n.
template <int L, int V, bool SPREAD>
__device__ __forceinline__ int chunk_at(int l, int r) { return SPREAD ? (r * L + l) * 4 : l * V + r * 4; }

template <int DT, int L, int V, bool SPREAD>
__device__ __forceinline__ void load_row(const void *row, int l, int n, bool vec, float fill, float (&v)[V]) {
#pragma unroll
    for (int r = 0; r < V / 4; ++r) {
        const int i = chunk_at<L, V, SPREAD>(l, r);
        float *o = v + 4 * r;
        if (vec && i + 4 <= n) {
            if (DT == DT_F32) {
                const f32x4 x = *(const f32x4 *)((const float *)row + i);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = x[k];
            } else {
                const u32x2 x = *(const u32x2 *)((const uint16_t *)row + i);
                o[0] = __uint_as_float(x[0] << 16);
                o[1] = __uint_as_float(x[0] & 0xFFFF0000u);
                o[2] = __uint_as_float(x[1] << 16);
                o[3] = __uint_as_float(x[1] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = i + k < n ? load1<DT>(row, i + k) : fill;
        }
    }
}

template <int DT, int L, int V, bool SPREAD>
__device__ __forceinline__ void store_row(void *row, int l, int n, bool vec, const float (&v)[V]) {
#pragma unroll
    for (int r = 0; r < V / 4; ++r) {
        const int i = chunk_at<L, V, SPREAD>(l, r);
        const float *o = v + 4 * r;
        if (vec && i + 4 <= n) {
            if (DT == DT_F32) *(f32x4 *)((float *)row + i) = f32x4{o[0], o[1], o[2], o[3]};
            else *(u32x2 *)((uint16_t *)row + i) = u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (i + k >= n) continue;
                if (DT == DT_F32) ((float *)row)[i + k] = o[k];
                else ((uint16_t *)row)[i + k] = (uint16_t)pack_bf16x2(o[k], 0.0f);
            }
        }
    }
}

struct GateArgs {
    int64_t T, ld, dld, t0;   // t0: the launch's first token
    int E, G, M, K;
    bool softmax, renorm, group_max;
    // whether rows of the logits, of scores / ds, of dlogits and the bias take four-value accesses
    bool vec, svec, dvec, bvec;
    float scale;
    const void *logits;
    const float *bias;
    float *scores;
    int32_t *idx;           // the forward's outputs
    float *w;
    const int32_t *cidx;    // the backward's inputs
    const float *cw, *dw, *ds;
    void *dlogits;
};

// Softmax statistics of a token: the exponentials e, the largest logit in use, and 1 / sum of e (0
// where no expert is in use).
template <int L, int V>
__device__ __forceinline__ void softmax_stats(const float (&z)[V], float (&e)[V], float &m, float &inv) {
    float t = neg_inf();
#pragma unroll
    for (int r = 0; r < V; ++r) t = fmaxf(t, z[r]);   // fmaxf passes over NaN
    m = lanes_max<L>(t);
    // the sum is held in 64 bits and rounded once, so that no order of the additions can move a choice
    double sum = 0.0;
    if (__any(m == -neg_inf())) {
#pragma unroll
        for (int r = 0; r < V; ++r) e[r] = softmax_exp(z[r], m);
    } else {
        const float base = m == neg_inf() ? 0.0f : m;
#pragma unroll
        for (int r = 0; r < V; ++r) e[r] = expf((in_use(z[r]) ? z[r] : neg_inf()) - base);   // softmax_exp's bits
    }
#pragma unroll
    for (int r = 0; r < V; ++r) sum += e[r];
    const float total = (float)lanes_sum<L>(sum);
    inv = total > 0.0f ? 1.0f / total : 0.0f;
}

// LDS of a token: the slots' keys and indices, with a bias the scores, and the experts' keys, for groups that do not
// lie in whole lanes each group a word apart from the next one's bank and the groups' own keys behind them.
__host__ __device__ inline int gate_lds_words(int E, int G, bool bias) {
    return 2 * kMaxK + (bias ? (E + 3) & ~3 : 0) + (G > 1 ? (E + 2 * G + 3) & ~3 : (E + 3) & ~3);
}

// The two largest keys of the `width` lanes (a power of two) around a lane, in all of them.
__device__ __forceinline__ void lanes_top2(uint32_t &k1, uint32_t &k2, int width) {
    auto join = [&](uint32_t o1, uint32_t o2) {
        k2 = max(min(k1, o1), max(k2, o2));
        k1 = max(k1, o1);
    };
    auto dpp = [&](auto ctrl) {
        join((uint32_t)__builtin_amdgcn_update_dpp((int)k1, (int)k1, decltype(ctrl)::value, 0xF, 0xF, false),
             (uint32_t)__builtin_amdgcn_update_dpp((int)k2, (int)k2, decltype(ctrl)::value, 0xF, 0xF, false));
    };
    if (width >= 2) dpp(std::integral_constant<int, 0xB1>{});
    if (width >= 4) dpp(std::integral_constant<int, 0x4E>{});
    if (width >= 8) dpp(std::integral_constant<int, 0x141>{});
    if (width >= 16) dpp(std::integral_constant<int, 0x140>{});
    if (width >= 32) join((uint32_t)__shfl_xor((int)k1, 16, 64), (uint32_t)__shfl_xor((int)k2, 16, 64));
}

// One pass over the logits: scores s (sigmoid, or softmax with its maximum and sum over the token's lanes), choice
// values s + b as ordered integers, groups by the sum of their two largest (or the largest), then K rounds of a maximum
// over the token's lanes, and the slots' weights, over their sum where that is asked for.  Nothing but the logits is
// read and nothing but the outputs written.
//
// 16384 tokens, 8 of 256 experts, 4 of 8 groups, fp32: 12.8 us for 17.9 MB, bound by vector instructions (four tokens
// a wave, four waves a SIMD): of 1183 a wave the 8 rounds take some 400, the exponentials 260, the groups 180, the keys
// 100, the reciprocals 50.  65521 tokens, 6 of 64 by softmax, bf16: 11 us for 11.5 MB.  One token: 4.2 us, the
// launch and one chain of dependent steps.
template <int DT, int L, int V>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(const GateArgs a) {
    constexpr int TPB = kGateThreads / L;                 // tokens per workgroup
    constexpr int Q = L < kMaxK ? kMaxK / L : 1;          // slots a lane handles, at most
    extern __shared__ __align__(16) uint32_t lds[];
    const int sub = threadIdx.x / L, l = threadIdx.x % L, lane = threadIdx.x & 63, base = lane / L * L;
    const int E = a.E, K = a.K, G = a.G, E4 = (E + 3) & ~3;
    const bool bias = a.bias != nullptr;
    uint32_t *slot_key = lds + sub * gate_lds_words(E, G, bias);
    int *slot_idx = (int *)(slot_key + kMaxK);
    float *sval = (float *)(slot_idx + kMaxK);
    uint32_t *ckey = (uint32_t *)(sval + (bias ? E4 : 0));
    uint32_t *gkey = ckey + E + G;
    // the wave's tokens past T work on the last one and store nothing
    const int64_t t0 = a.t0 + (int64_t)blockIdx.x * TPB + sub;
    const bool live = t0 < a.T;
    const int64_t t = live ? t0 : a.T - 1;
    const char *row = (const char *)a.logits + t * a.ld * (DT == DT_F32 ? 4 : 2);
    const int i0 = l * V;

    float z[V], b[V], s[V];
    load_row<DT, L, V, false>(row, l, E, a.vec, neg_inf(), z);
    if (bias) load_row<DT_F32, L, V, false>(a.bias, l, E, a.bvec, 0.0f, b);
    if (a.softmax) {
        float m, inv;
        softmax_stats<L, V>(z, s, m, inv);
#pragma unroll
        for (int r = 0; r < V; ++r) s[r] *= inv;
    } else {
        sigmoid_scores<V>(z, s);
    }
    // an expert out of use, or whose choice value is NaN (which fmaxf passes over), orders as -infinity
    uint32_t key[V];
    if (bias) {
#pragma unroll
        for (int r = 0; r < V; ++r) key[r] = choice_key(in_use(z[r]) ? fmaxf(s[r] + b[r], neg_inf()) : neg_inf());
#pragma unroll
        for (int r = 0; r < V; r += 4)
            if (i0 + r < E) *(f32x4 *)(sval + i0 + r) = f32x4{s[r], s[r + 1], s[r + 2], s[r + 3]};
    } else {
#pragma unroll
        for (int r = 0; r < V; ++r) key[r] = in_use(z[r]) ? __float_as_uint(s[r]) | 0x80000000u : kKeyNone;
    }
    if (E != L * V) {
#pragma unroll
        for (int r = 0; r < V; ++r)
            if (i0 + r >= E) key[r] = 0u;
    }
    if (a.scores && live) store_row<DT_F32, L, V, false>(a.scores + t * E, l, E, a.svec, s);

    if (G > 1) {
        const int gs = E / G;
        auto group_key = [&](uint32_t k1, uint32_t k2) {
            return !a.group_max && k2 > kKeyNone ? choice_key(key_value(k1) + key_value(k2)) : k1;
        };
        if (E == L * V && gs % V == 0 && G <= 16) {
            // a group is L / G whole lanes: its keys stay in registers (16384 tokens, 8 groups of 32: 2.1 us less
            // than by way of LDS; each lane compares with all G groups, hence the limit)
            const int width = L / G, mine = l / width;
            uint32_t k1 = 0, k2 = 0;
#pragma unroll
            for (int r = 0; r < V; ++r) {
                k2 = max(k2, min(k1, key[r]));
                k1 = max(k1, key[r]);
            }
            lanes_top2(k1, k2, width);
            const uint32_t k = group_key(k1, k2);
            // kept when fewer than M groups come before it
            int before = 0;
            for (int o = 0; o < G; ++o) {
                const uint32_t other = (uint32_t)__shfl((int)k, base + o * width, 64);
                before += other > k || (other == k && o < mine) ? 1 : 0;
            }
            const uint32_t most = before < a.M ? 0xFFFFFFFFu : kKeyNone;
#pragma unroll
            for (int r = 0; r < V; ++r) key[r] = min(key[r], most);
        } else {
            int g = i0 / gs, left = (g + 1) * gs - i0;
#pragma unroll
            for (int r = 0; r < V; ++r) {
                if (i0 + r < E) ckey[i0 + r + g] = key[r];
                if (--left == 0) {
                    ++g;
                    left = gs;
                }
            }
            token_lds_order();
            // a group's two largest keys, by one lane
            for (int o = l; o < G; o += L) {
                uint32_t k1 = 0, k2 = 0;
                const uint32_t *p = ckey + o * (gs + 1);
#pragma unroll 8
                for (int i = 0; i < gs; ++i) {
                    const uint32_t c = p[i];
                    k2 = max(k2, min(k1, c));
                    k1 = max(k1, c);
                }
                gkey[o] = group_key(k1, k2);
            }
            token_lds_order();
            // a group is kept when fewer than M others come before it
            uint32_t lo = 0, hi = 0;
            for (int o = l; o < G; o += L) {
                const uint32_t k = gkey[o];
                int before = 0;
#pragma unroll 8
                for (int p = 0; p < G; ++p) before += gkey[p] > k || (gkey[p] == k && p < o) ? 1 : 0;
                if (before < a.M) {
                    if (o < 32) lo |= 1u << o;
                    else hi |= 1u << (o - 32);
                }
            }
            auto either = [](uint32_t x, uint32_t y) { return x | y; };
            lo = lanes_reduce<L>(lo, either);
            if (G > 32) hi = lanes_reduce<L>(hi, either);
            const uint64_t kept = (uint64_t)hi << 32 | lo;
            g = i0 / gs;
            left = (g + 1) * gs - i0;
#pragma unroll
            for (int r = 0; r < V; ++r) {
                if (!((kept >> (g & 63)) & 1)) key[r] = min(key[r], kKeyNone);
                if (--left == 0) {
                    ++g;
                    left = gs;
                }
            }
        }
    }

    // K rounds: the lane with the largest key (the lowest such lane) gives up its first such expert
    auto winner = [&](uint32_t best, uint32_t &top) {
        top = lanes_max<L>(best);
        const uint64_t who = __ballot(best == top);
        return lane == base + __builtin_ctzll(who >> base);
    };
    if (V >= 16) {
        // many keys a lane: they lie in LDS, and registers keep the largest of every four (16384 tokens, 8 of 256: 12.7 us
        // against 14.3 with all keys in registers, where a round has to look through them all)
        uint32_t most[V / 4];
#pragma unroll
        for (int r = 0; r < V / 4; ++r) {
            const u32x4 k = {key[4 * r], key[4 * r + 1], key[4 * r + 2], key[4 * r + 3]};
            most[r] = max(max(k[0], k[1]), max(k[2], k[3]));
            if (i0 + 4 * r < E) *(u32x4 *)(ckey + i0 + 4 * r) = k;
        }
        token_lds_order();
        for (int j = 0; j < K; ++j) {
            uint32_t best = most[0], top;
#pragma unroll
            for (int r = 1; r < V / 4; ++r) best = max(best, most[r]);
            if (winner(best, top)) {
                int four = V / 4 - 1;
#pragma unroll
                for (int r = V / 4 - 2; r >= 0; --r) four = most[r] == top ? r : four;
                const int at = i0 + 4 * four;
                u32x4 k = *(const u32x4 *)(ckey + at);
                const int i = k[0] == top ? 0 : k[1] == top ? 1 : k[2] == top ? 2 : 3;
                ckey[at + i] = 0u;
#pragma unroll
                for (int r = 0; r < 4; ++r) k[r] = r == i ? 0u : k[r];
                const uint32_t left = max(max(k[0], k[1]), max(k[2], k[3]));
#pragma unroll
                for (int r = 0; r < V / 4; ++r) most[r] = r == four ? left : most[r];
                slot_key[j] = top;
                slot_idx[j] = at + i;
            }
        }
    } else {
        for (int j = 0; j < K; ++j) {
            uint32_t best = key[0], top;
#pragma unroll
            for (int r = 1; r < V; ++r) best = max(best, key[r]);
            if (winner(best, top)) {
                int at = 0;
                bool found = false;
#pragma unroll
                for (int r = 0; r < V; ++r) {
                    const bool take = key[r] == top && !found;
                    found = found || take;
                    at = take ? r : at;
                    key[r] = take ? 0u : key[r];
                }
                slot_key[j] = top;
                slot_idx[j] = i0 + at;
            }
        }
    }
    token_lds_order();
    // the slots' weights (without a bias a key is its score), and their sum from left to right
    float w[Q];
    int ix[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int j = min(l + q * L, K - 1);
        ix[q] = slot_idx[j];
        const uint32_t k = slot_key[j];
        w[q] = k == kKeyNone ? 0.0f : bias ? sval[ix[q]] : key_value(k);
    }
    if (a.renorm) {
        token_lds_order();
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (l + q * L < K) slot_key[l + q * L] = __float_as_uint(w[q]);
        token_lds_order();
        float total = 0.0f;
#pragma unroll 8
        for (int j = 0; j < K; ++j) total += __uint_as_float(slot_key[j]);
#pragma unroll
        for (int q = 0; q < Q; ++q) w[q] = total > 0.0f ? w[q] / total : 0.0f;
    }
    if (!live) return;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int j = l + q * L;
        if (j < K) {
            a.idx[t * K + j] = ix[q];
            a.w[t * K + j] = w[q] * a.scale;
        }
    }
}

__host__ __device__ inline int gate_backward_lds_words(int E) { return (E + 3) & ~3; }

// With D the sum of the chosen scores, w_j = c s_j / D gives dL/ds_j = c (g_j - sum_i g_i s_i / D) / D, without
// renormalisation c g_j; the scores' own gradient is added to that, and
// dL/dz = ds s (1 - s) for sigmoid scores, s (ds - sum_e ds_e s_e) for softmax ones.
// Near the smallest floats 1 / D and ds overflow, though s ds is of the order of g for any D.  There (D < 2^-64) the chosen
// scores are taken 2^100 times as large, which is exact, so that ds comes out 2^100 times smaller, and s ds is formed from
// the two before anything is added.
//
// Every row of dlogits is written whole, zeros included.  16384 tokens, 8 of 256, sigmoid, fp32: 6 us for 19 MB, mostly
// those zeros.  65521 tokens of 64 experts, softmax and a gradient at every score, bf16: 10.7 us for 38 MB.
//
// DENSE: softmax scores, or a gradient at every score.  Otherwise only the chosen logits have a
// gradient, and only they are read.
template <int DT, int L, int V, bool DENSE>
__global__ __launch_bounds__(kGateThreads) void gate_backward_kernel(const GateArgs a) {
    constexpr int TPB = kGateThreads / L;
    constexpr int Q = L < kMaxK ? kMaxK / L : 1;
    extern __shared__ __align__(16) uint32_t lds[];
    const int sub = threadIdx.x / L, l = threadIdx.x % L;
    const int E = a.E, K = a.K;
    float *dsl = (float *)(lds + sub * gate_backward_lds_words(E));   // the slots' part of ds, of s ds, or of dz
    const int64_t t0 = a.t0 + (int64_t)blockIdx.x * TPB + sub;
    const bool live = t0 < a.T;
    const int64_t t = live ? t0 : a.T - 1;
    const char *row = (const char *)a.logits + t * a.ld * (DT == DT_F32 ? 4 : 2);

    float z[V], d[V], m = 0.0f, inv = 0.0f;
    int ij[Q];
    float sj[Q], gj[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int j = l + q * L;
        const int64_t at = t * K + min(j, K - 1);
        const float w = a.cw[at];
        ij[q] = a.cidx[at];
        gj[q] = a.dw[at];
        if (j >= K || w == 0.0f || (unsigned)ij[q] >= (unsigned)E) ij[q] = -1;
    }
    const float w0 = a.cw[t * K], dw0 = a.dw[t * K];
    if (DENSE) {
        load_row<DT, L, V, true>(row, l, E, a.vec, neg_inf(), z);
        if (a.ds) load_row<DT_F32, L, V, true>(a.ds + t * E, l, E, a.svec, 0.0f, d);
    }
    // the slots' logits; slots without a weight read the first one and do not use it
#pragma unroll
    for (int q = 0; q < Q; ++q) sj[q] = load1<DT>(row, max(ij[q], 0));
#pragma unroll
    for (int r = 0; r < V / 4; ++r) {
        const int i = chunk_at<L, V, true>(l, r);
        if (i < E) *(f32x4 *)(dsl + i) = f32x4{0, 0, 0, 0};
    }

    float s[V];
    if (DENSE) {
        if (a.softmax) {
            softmax_stats<L, V>(z, s, m, inv);
#pragma unroll
            for (int r = 0; r < V; ++r) s[r] *= inv;
        } else {
            sigmoid_scores<V>(z, s);
        }
    }
    // Slots: s_j and g_j.  The weights' sum is fixed under renormalisation, so a common part of the g
    // moves nothing: taking g_0 away first keeps the difference below exact where the g are alike
    // (K = 1 gives 0).
    const float g0 = a.renorm && w0 != 0.0f ? dw0 : 0.0f;
    float sum_s = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const bool on = ij[q] >= 0;
        sj[q] = !on ? 0.0f : a.softmax ? softmax_exp(sj[q], m) * inv : sigmoid_score(sj[q]);
        gj[q] = on ? gj[q] - g0 : 0.0f;
        sum_s += sj[q];
    }
    float invd = 1.0f, mean = 0.0f, up = 1.0f;
    if (a.renorm) {
        const float D = lanes_sum<L>(sum_s);
        up = D < 0x1p-64f ? 0x1p100f : 1.0f;
        invd = D > 0.0f ? 1.0f / (D * up) : 0.0f;
#pragma unroll
        for (int q = 0; q < Q; ++q) mean += gj[q] * (sj[q] * up);
        mean = lanes_sum<L>(mean) * invd;
    }
    const bool tiny = up != 1.0f;
    token_lds_order();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if (ij[q] < 0) continue;
        const float ds = (gj[q] - mean) * invd * a.scale, sds = ds * (sj[q] * up);
        dsl[ij[q]] = !DENSE ? sds * (1.0f - sj[q]) : tiny ? sds : ds;
    }
    token_lds_order();

    float o[V];
#pragma unroll
    for (int r = 0; r < V / 4; ++r) {
        const int i = chunk_at<L, V, true>(l, r);
        const f32x4 x = i < E ? *(const f32x4 *)(dsl + i) : f32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) o[4 * r + k] = x[k];
    }
    if (DENSE) {
        float dot = 0.0f;
        // an expert out of use takes no gradient, whatever the caller's dscores holds there
        if (__any(tiny)) {
            float sds[V];
#pragma unroll
            for (int r = 0; r < V; ++r) {
                const float own = a.ds && in_use(z[r]) ? d[r] : 0.0f;
                o[r] = !in_use(z[r]) ? 0.0f : tiny ? o[r] : o[r] + own;
                sds[r] = tiny ? own * s[r] + o[r] : o[r] * s[r];
                dot += sds[r];
            }
            if (a.softmax) dot = lanes_sum<L>(dot);
#pragma unroll
            for (int r = 0; r < V; ++r)
                o[r] = !a.softmax ? sds[r] * (1.0f - s[r]) : tiny ? sds[r] - s[r] * dot : s[r] * (o[r] - dot);
        } else {
#pragma unroll
            for (int r = 0; r < V; ++r) {
                o[r] = in_use(z[r]) ? (a.ds ? d[r] + o[r] : o[r]) : 0.0f;
                dot += o[r] * s[r];
            }
            if (a.softmax) dot = lanes_sum<L>(dot);
#pragma unroll
            for (int r = 0; r < V; ++r) o[r] = a.softmax ? s[r] * (o[r] - dot) : o[r] * s[r] * (1.0f - s[r]);
        }
    }
    if (live) store_row<DT, L, V, true>((char *)a.dlogits + t * a.dld * (DT == DT_F32 ? 4 : 2), l, E, a.dvec, o);
}

// f(L, V) for the token's width.
template <class F>
hipError_t with_width(int64_t T, int E, F f) {
    const GateWidth w = gate_width(T, E, device_cus());
    hipError_t e = hipErrorInvalidValue;
    auto width = [&](auto l, auto v) {
        if (w.lanes == decltype(l)::value && w.values == decltype(v)::value) e = f(l, v);
    };
    using std::integral_constant;
    width(integral_constant<int, 8>{}, integral_constant<int, 4>{});
    width(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    width(integral_constant<int, 32>{}, integral_constant<int, 4>{});
    width(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    width(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    width(integral_constant<int, 16>{}, integral_constant<int, 8>{});
    width(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    width(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    width(integral_constant<int, 32>{}, integral_constant<int, 16>{});
    width(integral_constant<int, 64>{}, integral_constant<int, 16>{});
    return e;
}

// A launch holds fewer than 2^32 threads: f(first token, grid) for parts of the batch of TPB tokens a workgroup.
template <class F>
hipError_t in_launches(int64_t T, int TPB, F f) {
    const int64_t part = (int64_t)((1ll << 32) / kGateThreads - 1) * TPB;
    for (int64_t t = 0; t < T; t += part) {
        const int64_t n = T - t < part ? T - t : part;
        f(t, (unsigned)((n + TPB - 1) / TPB));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Whether every row of a matrix can be read four values at a time.
bool rows_of_four(const void *p, int64_t ld, int esz) { return (uintptr_t)p % (4 * esz) == 0 && ld % 4 == 0; }

GateArgs gate_args(const GateProblem &p) {
    GateArgs a{};
    a.T = p.T;
    a.E = p.E;
    a.G = p.G;
    a.M = p.M;
    a.K = p.K;
    a.softmax = p.softmax;
    a.renorm = p.renorm;
    a.group_max = p.group_max;
    a.scale = p.scale;
    a.logits = p.logits;
    a.ld = p.ld;
    a.vec = rows_of_four(p.logits, p.ld, p.dt == DT_F32 ? 4 : 2);
    return a;
}

}  // namespace

hipError_t launch_gate(const GateProblem &p, const float *bias, float *scores, int32_t *idx, float *w, hipStream_t s) {
    if (p.T <= 0) return hipSuccess;
    GateArgs a = gate_args(p);
    a.bias = bias;
    a.bvec = rows_of_four(bias, 0, 4);
    a.scores = scores;
    a.svec = rows_of_four(scores, p.E, 4);
    a.idx = idx;
    a.w = w;
    return with_width(p.T, p.E, [&](auto lc, auto vc) {
        constexpr int L = decltype(lc)::value, V = decltype(vc)::value, TPB = kGateThreads / L;
        const size_t lds = (size_t)TPB * gate_lds_words(p.E, p.G, bias != nullptr) * 4;
        return in_launches(p.T, TPB, [&](int64_t t, unsigned grid) {
            a.t0 = t;
            if (p.dt == DT_F32) gate_kernel<DT_F32, L, V><<<grid, kGateThreads, lds, s>>>(a);
            else gate_kernel<DT_BF16, L, V><<<grid, kGateThreads, lds, s>>>(a);
        });
    });
}

hipError_t launch_gate_backward(const GateProblem &p, const int32_t *idx, const float *w, const float *dw,
                                const float *ds, void *dlogits, int64_t dld, hipStream_t s) {
    if (p.T <= 0) return hipSuccess;
    GateArgs a = gate_args(p);
    a.cidx = idx;
    a.cw = w;
    a.dw = dw;
    a.ds = ds;
    a.svec = rows_of_four(ds, p.E, 4);
    a.dlogits = dlogits;
    a.dld = dld;
    a.dvec = rows_of_four(dlogits, dld, p.dt == DT_F32 ? 4 : 2);
    return with_width(p.T, p.E, [&](auto lc, auto vc) {
        constexpr int L = decltype(lc)::value, V = decltype(vc)::value, TPB = kGateThreads / L;
        const size_t lds = (size_t)TPB * gate_backward_lds_words(p.E) * 4;
        const bool dense = p.softmax || ds;
        return in_launches(p.T, TPB, [&](int64_t t, unsigned grid) {
            a.t0 = t;
            if (p.dt == DT_F32) {
                if (dense) gate_backward_kernel<DT_F32, L, V, true><<<grid, kGateThreads, lds, s>>>(a);
                else gate_backward_kernel<DT_F32, L, V, false><<<grid, kGateThreads, lds, s>>>(a);
            } else {
                if (dense) gate_backward_kernel<DT_BF16, L, V, true><<<grid, kGateThreads, lds, s>>>(a);
                else gate_backward_kernel<DT_BF16, L, V, false><<<grid, kGateThreads, lds, s>>>(a);
            }
        });
    });
}

}  // namespace moe
