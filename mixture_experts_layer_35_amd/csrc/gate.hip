// gate.hip -- routing from logits: softmax or sigmoid scores, a bias for balance,
// groups, top-K, renormalised weights ("DeepSeek-V3 Technical Report", §2.1.2, for the
// sigmoid form), and the gradient of the weights at the logits.
//
// A token belongs to L lanes of a wave, lane l holding experts l*V .. l*V + V-1 in
// registers, so that lane order is index order and a tie's lower index is the lower lane.
#include <type_traits>

#include "common.h"
#include "internal.h"

// A product and a sum that the definition rounds one after the other stay two roundings.
#pragma clang fp contract(off)

namespace moe {

namespace {

constexpr int kGateThreads = 256;
constexpr int kMaxK = 32;   // slots of a token, at most

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Largest of v over the L lanes of a token, in all of them.  Four steps stay inside a row
// of 16 lanes (DPP); the rest cross rows.
template <int L, class T, class Op>
__device__ __forceinline__ T lanes_reduce(T v, Op op) {
    auto dpp = [](T x, auto ctrl) {
        const int y = __builtin_bit_cast(int, x);
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(y, y, decltype(ctrl)::value, 0xF, 0xF, false));
    };
    v = op(v, dpp(v, std::integral_constant<int, 0xB1>{}));               // lane ^ 1
    v = op(v, dpp(v, std::integral_constant<int, 0x4E>{}));               // lane ^ 2
    if (L >= 8) v = op(v, dpp(v, std::integral_constant<int, 0x141>{}));  // the other quad of 8
    if (L >= 16) v = op(v, dpp(v, std::integral_constant<int, 0x140>{})); // the other half of 16
    if (L >= 32) v = op(v, __shfl_xor(v, 16, 64));
    if (L >= 64) v = op(v, __shfl_xor(v, 32, 64));
    return v;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    return lanes_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
    return lanes_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    return lanes_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
// fp64 sum of one fp32 value a lane.
template <int L>
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
    for (int m = 1; m < L; m <<= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// Order of choice values as unsigned integers; 0 stands below all of them.
__device__ __forceinline__ uint32_t choice_key(float c) {
    const uint32_t b = __float_as_uint(c == 0.0f ? 0.0f : c);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
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

template <int DT>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    return DT == DT_F32 ? ((const float *)p)[i] : bf16_to_f32(((const uint16_t *)p)[i]);
}

// V values of a row from element i0 on; `fill` past element n.
template <int DT, int V>
__device__ __forceinline__ void load_row(const void *row, int i0, int n, bool vec, float fill, float (&v)[V]) {
    if (vec && i0 + V <= n) {
        if (DT == DT_F32) {
#pragma unroll
            for (int r = 0; r < V; r += 4) {
                const f32x4 x = *(const f32x4 *)((const float *)row + i0 + r);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[r + k] = x[k];
            }
        } else {
#pragma unroll
            for (int r = 0; r < V; r += 4) {
                const u32x2 x = *(const u32x2 *)((const uint16_t *)row + i0 + r);
                v[r] = __uint_as_float(x[0] << 16);
                v[r + 1] = __uint_as_float(x[0] & 0xFFFF0000u);
                v[r + 2] = __uint_as_float(x[1] << 16);
                v[r + 3] = __uint_as_float(x[1] & 0xFFFF0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int r = 0; r < V; ++r) v[r] = i0 + r < n ? load1<DT>(row, i0 + r) : fill;
}

template <int DT, int V>
__device__ __forceinline__ void store_row(void *row, int i0, int n, bool vec, const float (&v)[V]) {
    if (vec && i0 + V <= n) {
#pragma unroll
        for (int r = 0; r < V; r += 4) {
            if (DT == DT_F32) *(f32x4 *)((float *)row + i0 + r) = f32x4{v[r], v[r + 1], v[r + 2], v[r + 3]};
            else *(u32x2 *)((uint16_t *)row + i0 + r) = u32x2{pack_bf16x2(v[r], v[r + 1]), pack_bf16x2(v[r + 2], v[r + 3])};
        }
        return;
    }
#pragma unroll
    for (int r = 0; r < V; ++r) {
        if (i0 + r >= n) continue;
        if (DT == DT_F32) ((float *)row)[i0 + r] = v[r];
        else ((uint16_t *)row)[i0 + r] = (uint16_t)pack_bf16x2(v[r], 0.0f);
    }
}

struct GateArgs {
    int64_t T, ld, dld;
    int E, G, M, K;
    bool softmax, renorm, group_max;
    bool vec, svec, dvec;   // rows of the logits, of scores / ds and of dlogits take four-value accesses
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

// Softmax statistics of a token: largest logit in use and 1 / sum of the exponentials (0 where none is in use).
template <int L, int V>
__device__ __forceinline__ void softmax_stats(const float (&z)[V], float &m, float &inv) {
    float t = neg_inf();
#pragma unroll
    for (int r = 0; r < V; ++r) t = fmaxf(t, z[r]);   // fmaxf passes over NaN
    m = lanes_max<L>(t);
    // the sum is held in 64 bits and rounded once, so that no order of the additions can move a choice
    double sum = 0.0;
#pragma unroll
    for (int r = 0; r < V; ++r) sum += softmax_exp(z[r], m);
    const float total = (float)lanes_sum<L>(sum);
    inv = total > 0.0f ? 1.0f / total : 0.0f;
}

__host__ __device__ inline int gate_lds_floats(int E, int G) { return 2 * kMaxK + (G > 1 ? E + G : 0); }
__host__ __device__ inline int gate_backward_lds_floats(int E) { return E + 3; }

template <int DT, int L, int V>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(const GateArgs a) {
    constexpr int TPB = kGateThreads / L;                 // tokens per workgroup
    extern __shared__ float lds[];
    const int sub = threadIdx.x / L, l = threadIdx.x % L;
    const int E = a.E, K = a.K, G = a.G;
    // per token: the slots' keys and indices, then (with groups) the choice values and the groups' keys
    uint32_t *slot_key = (uint32_t *)(lds + sub * gate_lds_floats(E, G));
    int *slot_idx = (int *)(slot_key + kMaxK);
    float *cval = (float *)(slot_idx + kMaxK);
    uint32_t *gkey = (uint32_t *)(cval + E);
    // the wave's tokens past T work on the last one and store nothing
    const int64_t t0 = (int64_t)blockIdx.x * TPB + sub;
    const bool live = t0 < a.T;
    const int64_t t = live ? t0 : a.T - 1;
    const char *row = (const char *)a.logits + t * a.ld * (DT == DT_F32 ? 4 : 2);
    const int i0 = l * V;

    float z[V];
    load_row<DT, V>(row, i0, E, a.vec, neg_inf(), z);
    float m = 0.0f, inv = 0.0f;
    if (a.softmax) softmax_stats<L, V>(z, m, inv);
    auto score = [&](float x) { return a.softmax ? softmax_exp(x, m) * inv : sigmoid_score(x); };
    uint32_t key[V];
    float s[V];
#pragma unroll
    for (int r = 0; r < V; ++r) {
        s[r] = score(z[r]);
        float c = s[r];
        if (a.bias) c += i0 + r < E ? a.bias[i0 + r] : 0.0f;
        if (!in_use(z[r]) || c != c) c = neg_inf();
        key[r] = i0 + r < E ? choice_key(c) : 0u;
    }
    if (a.scores && live) store_row<DT_F32, V>(a.scores + t * E, i0, E, a.svec, s);

    if (G > 1) {
        const int gs = E / G;
#pragma unroll
        for (int r = 0; r < V; ++r)
            if (i0 + r < E) cval[i0 + r] = key_value(key[r]);
        __syncthreads();
        for (int g = l; g < G; g += L) {
            float v1 = neg_inf(), v2 = neg_inf();
            for (int i = 0; i < gs; ++i) {
                const float c = cval[g * gs + i];
                v2 = fmaxf(v2, fminf(v1, c));
                v1 = fmaxf(v1, c);
            }
            gkey[g] = choice_key(a.group_max || v2 == neg_inf() ? v1 : v1 + v2);
        }
        __syncthreads();
        // a group is kept when fewer than M others come before it
        uint32_t lo = 0, hi = 0;
        for (int g = l; g < G; g += L) {
            const uint32_t k = gkey[g];
            int before = 0;
            for (int o = 0; o < G; ++o) before += gkey[o] > k || (gkey[o] == k && o < g) ? 1 : 0;
            if (before < a.M) {
                if (g < 32) lo |= 1u << g;
                else hi |= 1u << (g - 32);
            }
        }
        auto either = [](uint32_t x, uint32_t y) { return x | y; };
        lo = lanes_reduce<L>(lo, either);
        hi = lanes_reduce<L>(hi, either);
        const uint64_t kept = (uint64_t)hi << 32 | lo;
#pragma unroll
        for (int r = 0; r < V; ++r)
            if (key[r] != 0u && !((kept >> ((i0 + r) / gs)) & 1)) key[r] = kKeyNone;
    }

    // K rounds: the lane with the largest key (the lowest of them) gives up its first such expert
    uint32_t best;
    int at;
    auto head = [&]() {
        best = 0;
        at = 0;
#pragma unroll
        for (int r = V - 1; r >= 0; --r) {
            if (key[r] >= best) {
                best = key[r];
                at = r;
            }
        }
    };
    head();
    const int lane = threadIdx.x & 63, base = lane / L * L;
    for (int j = 0; j < K; ++j) {
        const uint32_t top = lanes_max<L>(best);
        const uint64_t who = __ballot(best == top);
        const int winner = base + __builtin_ctzll(who >> base);
        if (lane == winner) {
            slot_key[j] = top;
            slot_idx[j] = i0 + at;
#pragma unroll
            for (int r = 0; r < V; ++r)
                if (r == at) key[r] = 0u;
            head();
        }
    }
    __syncthreads();
    // the slots' weights, and their sum from left to right
    auto slot_score = [&](int j) {
        return slot_key[j] == kKeyNone ? 0.0f : score(load1<DT>(row, slot_idx[j]));
    };
    constexpr int Q = L < kMaxK ? kMaxK / L : 1;          // slots a lane handles, at most
    float mine[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int j = l + q * L;
        mine[q] = j < K ? slot_score(j) : 0.0f;
    }
    if (a.renorm) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (l + q * L < K) slot_key[l + q * L] = __float_as_uint(mine[q]);
        __syncthreads();
        float total = 0.0f;
        for (int j = 0; j < K; ++j) total += __uint_as_float(slot_key[j]);
#pragma unroll
        for (int q = 0; q < Q; ++q) mine[q] = total > 0.0f ? mine[q] / total : 0.0f;
    }
    if (!live) return;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int j = l + q * L;
        if (j < K) {
            a.idx[t * K + j] = slot_idx[j];
            a.w[t * K + j] = mine[q] * a.scale;
        }
    }
}

template <int DT, int L, int V>
__global__ __launch_bounds__(kGateThreads) void gate_backward_kernel(const GateArgs a) {
    constexpr int TPB = kGateThreads / L;
    constexpr int Q = L < kMaxK ? kMaxK / L : 1;          // slots a lane handles, at most
    extern __shared__ float lds[];
    const int sub = threadIdx.x / L, l = threadIdx.x % L;
    const int E = a.E, K = a.K;
    float *dsl = lds + sub * gate_backward_lds_floats(E); // the slots' part of ds
    const int64_t t0 = (int64_t)blockIdx.x * TPB + sub;
    const bool live = t0 < a.T;
    const int64_t t = live ? t0 : a.T - 1;
    const char *row = (const char *)a.logits + t * a.ld * (DT == DT_F32 ? 4 : 2);
    const int i0 = l * V;

    float z[V], m = 0.0f, inv = 0.0f;
    load_row<DT, V>(row, i0, E, a.vec, neg_inf(), z);
    if (a.softmax) softmax_stats<L, V>(z, m, inv);
    auto score = [&](float x) { return a.softmax ? softmax_exp(x, m) * inv : sigmoid_score(x); };
#pragma unroll
    for (int r = 0; r < V; ++r)
        if (i0 + r < E) dsl[i0 + r] = 0.0f;

    // slots: s_j and g_j, zero where the weight is 0.  The weights' sum is fixed under
    // renormalisation, so a common part of the g moves nothing: taking g_0 away first keeps the
    // difference below exact where the g are alike (K = 1 gives 0).
    float sj[Q], gj[Q];
    int ij[Q];
    const float g0 = a.renorm && a.cw[t * K] != 0.0f ? a.dw[t * K] : 0.0f;
    float sum_s = 0.0f, sum_gs = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int j = l + q * L;
        const bool on = j < K && a.cw[t * K + j] != 0.0f;
        ij[q] = on ? a.cidx[t * K + j] : 0;
        const bool ok = on && (unsigned)ij[q] < (unsigned)E;
        if (!ok) ij[q] = -1;
        sj[q] = ok ? score(load1<DT>(row, ij[q])) : 0.0f;
        gj[q] = ok ? a.dw[t * K + j] - g0 : 0.0f;
        sum_s += sj[q];
        sum_gs += gj[q] * sj[q];
    }
    float invd = 1.0f, mean = 0.0f;
    if (a.renorm) {
        const float D = lanes_sum<L>(sum_s);
        invd = D > 0.0f ? 1.0f / D : 0.0f;
        mean = lanes_sum<L>(sum_gs) * invd;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < Q; ++q)
        if (ij[q] >= 0) dsl[ij[q]] = (gj[q] - mean) * invd * a.scale;
    __syncthreads();

    float d[V], s[V];
    if (a.ds) load_row<DT_F32, V>(a.ds + t * E, i0, E, a.svec, 0.0f, d);
    else {
#pragma unroll
        for (int r = 0; r < V; ++r) d[r] = 0.0f;
    }
    float dot = 0.0f;
#pragma unroll
    for (int r = 0; r < V; ++r) {
        s[r] = score(z[r]);
        // an expert out of use takes no gradient, whatever the caller's dscores holds there
        d[r] = in_use(z[r]) ? d[r] + (i0 + r < E ? dsl[i0 + r] : 0.0f) : 0.0f;
        dot += d[r] * s[r];
    }
    if (a.softmax) dot = lanes_sum<L>(dot);
#pragma unroll
    for (int r = 0; r < V; ++r) d[r] = a.softmax ? s[r] * (d[r] - dot) : d[r] * s[r] * (1.0f - s[r]);
    if (live) store_row<DT, V>((char *)a.dlogits + t * a.dld * (DT == DT_F32 ? 4 : 2), i0, E, a.dvec, d);
}

// f(L, V) for the smallest token width that holds E experts: up to 16 values a lane, so that a
// wave serves four tokens at 256 experts.
template <class F>
hipError_t with_width(int E, F f) {
    using std::integral_constant;
    if (E <= 32) return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
    if (E <= 64) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    if (E <= 128) return f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
    if (E <= 256) return f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    if (E <= 512) return f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
    return f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
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
    a.scores = scores;
    a.svec = rows_of_four(scores, p.E, 4);
    a.idx = idx;
    a.w = w;
    return with_width(p.E, [&](auto lc, auto vc) {
        constexpr int L = decltype(lc)::value, V = decltype(vc)::value, TPB = kGateThreads / L;
        const unsigned grid = (unsigned)((p.T + TPB - 1) / TPB);
        const size_t lds = (size_t)TPB * gate_lds_floats(p.E, p.G) * 4;
        if (p.dt == DT_F32) gate_kernel<DT_F32, L, V><<<grid, kGateThreads, lds, s>>>(a);
        else gate_kernel<DT_BF16, L, V><<<grid, kGateThreads, lds, s>>>(a);
        return hipGetLastError();
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
    return with_width(p.E, [&](auto lc, auto vc) {
        constexpr int L = decltype(lc)::value, V = decltype(vc)::value, TPB = kGateThreads / L;
        const unsigned grid = (unsigned)((p.T + TPB - 1) / TPB);
        const size_t lds = (size_t)TPB * gate_backward_lds_floats(p.E) * 4;
        if (p.dt == DT_F32) gate_backward_kernel<DT_F32, L, V><<<grid, kGateThreads, lds, s>>>(a);
        else gate_backward_kernel<DT_BF16, L, V><<<grid, kGateThreads, lds, s>>>(a);
        return hipGetLastError();
    });
}

}  // namespace moe
