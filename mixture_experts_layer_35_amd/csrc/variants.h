// variants.h -- which variant of a kernel a call takes, from its sizes alone.  Host code without HIP, so that it
// can be asked about any size without a GPU.
#pragma once

#include <cstdint>

namespace moe {

// ---- gate on logits ----------------------------------------------------------
// A token's lanes and the values each of them holds, lanes * values >= E.  Up to 16 values a lane keep a wave on four
// tokens at 256 experts, which costs the fewest instructions a token; a batch whose waves would leave compute units idle
// takes four values a lane instead, the shortest chain of instructions to its end.  256 experts: 16384 tokens 12.7 us
// with 16 values a lane, 17.2 with four; one token 7.6 us and 5.4.
struct GateWidth {
    int lanes, values;
};

inline GateWidth gate_width(int64_t T, int E, int64_t cus) {
    const bool few = T * ((E + 3) / 4) <= cus * 4 * 64;   // lanes of 4 values fill one wave a SIMD
    if (E <= 32) return {8, 4};
    if (E <= 64) return few ? GateWidth{16, 4} : GateWidth{8, 8};
    if (E <= 128) return few ? GateWidth{32, 4} : GateWidth{16, 8};
    if (E <= 256) return few ? GateWidth{64, 4} : GateWidth{16, 16};
    if (E <= 512) return few ? GateWidth{64, 8} : GateWidth{32, 16};
    return {64, 16};
}

// ---- experts on MX4 ----------------------------------------------------------
enum Mx4Variant {
    kMx4Shared,     // tiles of 64 weight rows by up to 16 tokens, four waves a tile
    kMx4Stream,     // tiles of 64 weight rows by up to 32 tokens, a wave each
    kMx4Tile128,    // tiles of 256 weight rows by up to 128 tokens, a workgroup each
    kMx4Tile160,    // by up to 160 tokens
};

// Tokens of a tile.
constexpr int mx4_tokens(Mx4Variant v) { return v == kMx4Shared ? 16 : v == kMx4Stream ? 32 : v == kMx4Tile128 ? 128 : 160; }

// Runs of 128 values of the reduction, of which two are a segment; ftiles: blocks of 64 weight rows.
inline Mx4Variant mx4_variant(int64_t max_rows, int64_t n_exp, int64_t kruns, int64_t ftiles, int64_t cus) {
    const int64_t experts = max_rows < n_exp ? max_rows : n_exp;
    // row blocks of an expert's tiles, at most
    auto blocks = [&](Mx4Variant v) { return experts + (max_rows - experts) / mx4_tokens(v); };
    // Four waves share a tile where that ends sooner: `rounds` tiles a workgroup, one after the other, each a
    // quarter of the segments and, for adding up, as long as 2.5 more, against all segments by one wave.  With
    // rows of 7168 (28 segments) and 2048 (8), experts of 7168 x 2048: 1 token to 8 experts, gate/up in 2 rounds
    // shared 42 us (the whole call), not shared 50; 32 tokens of one expert, down in 1 round 23 against 26,
    // 48 tokens in 2 rounds 28 against 26.
    const int64_t segs = (kruns + 1) / 2, rounds = (blocks(kMx4Shared) * ftiles + cus - 1) / cus;
    if (rounds * (segs + 10) < 4 * segs) return kMx4Shared;
    // Tiles for a wave by itself as long as there is no more than one for each wave: one expert of 7168 x 2048,
    // 384 tokens, gate/up of 768 tiles 42 us (the whole call) against 52 in the tile kernel, 640 tokens, 1280 tiles
    // 65 against 53; 8 x 512 tokens of 512 x 256, 1024 tiles in either pass 16 against 22.
    if (blocks(kMx4Stream) * ftiles <= cus * 4) return kMx4Stream;
    // Tiles of up to 160 tokens where experts of the average size need fewer of them than of 128 (an eighth is
    // left for experts above the average) and there is one for each workgroup.  256 experts of 7168 x 2048:
    // 90 rows 1290 us either way, 128 rows 1410 us against 1540 with 128 tokens, 219 rows 2430 against 2100,
    // 256 rows 2330 against 2430; 8 experts of 2048 x 1024, 128 rows, 64 tiles: 33 against 30.
    const int64_t n = n_exp;
    const bool fewer = (max_rows + 140 * n - 1) / (140 * n) < (max_rows + 112 * n - 1) / (112 * n);
    return fewer && blocks(kMx4Tile160) * ((ftiles + 3) / 4) >= cus ? kMx4Tile160 : kMx4Tile128;
}

// ---- products of experts -------------------------------------------------------
enum ProductVariant {
    kProductAny,        // operands through registers: where one of them does not lie in pieces of 16 bytes
    kProductStream,     // tiles of 64 features by up to 8 rows, four waves a tile
    kProduct160,        // tiles of 256 features by up to 160 rows, three stages of LDS
    kProduct256,        // by up to 256 rows, two stages
};

// Rows of a tile.
constexpr int product_rows(ProductVariant v) {
    return v == kProductStream ? 8 : v == kProduct160 ? 160 : v == kProduct256 ? 256 : 128;
}

// features: the output's (the inputs of the gradient at x); pieces: whether both operands lie in pieces of 16 bytes.  Where one
// does not, both go through registers, and few rows lose most: one token to 8 experts of 7161 x 2048 246 us, of 7168 x 2048 43;
// 2 tokens to 16 experts of 7168 x 2048 333 us with x's rows 3 values wider, 79 without; 128 tokens, 256 experts 2730 and 1190.
inline ProductVariant product_variant(int64_t max_rows, int64_t n_exp, int64_t features, bool pieces, int64_t cus) {
    if (!pieces) return kProductAny;
    const int64_t experts = max_rows < n_exp ? max_rows : n_exp;
    // Small tiles as long as there are no more than two for each compute unit.  Small tiles and tiles of 160 rows, experts of one
    // row each, in microseconds: 7168 to 2048, 8 experts (256 small tiles) 35 and 69, 16 (512) 79 and 96, 24 (768) 117 and 118;
    // 512 to 512, 64 experts (512) 7.5 and 9.1, 96 (768) 11.1 and 10.5; the gradient at x of 2048 to 7168, 12 experts (384) 76
    // and 85, 16 (512) 90 and 89, 24 (768) 133 and 115; 8 bits, 7168 to 2048, 12 experts 34 and 39, 16 40 and 39, 24 66 and 61.
    const int64_t small = (experts + (max_rows - experts) / product_rows(kProductStream)) * ((features + 63) / 64);
    if (small <= 2 * cus) return kProductStream;
    // Tiles of 160 rows, which leave room for a stage more, where experts of the average size need one of them.  7168 to 2048, 32
    // experts of as many rows each, tiles of 160 and of 256: 128 rows 181 and 205 us, 160 rows 200 and 215, 170 rows 277 and 220,
    // 256 rows 287 and 259, 320 rows 342 and 347, 512 rows 522 and 466.  The host does not know how rows are spread: 150 on
    // average and 183 at most takes tiles of 160, 313 us against 214; 200 on average and 1539 at most tiles of 256, 394 against
    // 295.  Nor does the rule look at how many tiles there are: 8 experts of 256 rows, 2048 to 2048, take 54 us in 64 tiles of
    // 256 and would take 37 in 128 of 160.  256 experts of 128 rows: 1560 us with 160, 1686 with 128, which half of the experts
    // need two of.
    return max_rows > 160 * n_exp ? kProduct256 : kProduct160;
}

// ---- orthogonalised updates ----------------------------------------------------
enum OrthVariant { kOrth256x256, kOrth256x128, kOrth128x128, kOrth64x64 };   // a tile's sides along a and b

// The tiles that end soonest: rounds of tiles over the workgroups, each as long as one tile takes.  A tile of 256 x 256 takes
// 2.2 to 3.1 times as long as one of 128 x 128, one of 256 x 128 1.4 to 1.7 times.  Microseconds with 256 x 256, 256 x 128 and
// 128 x 128: 8 matrices of 2048 x 7168, X X^T 907, 818, 887, P X 1178, 1349, 1621; one of them 381, 236, 169 and 150, 178,
// 225; 32 of 512 x 1024, X X^T 70, 45, 57.  Whole calls of five steps with one product's tile changed, 256 x 256, 256 x 128,
// 128 x 128 and 64 x 64, X X^T and S S / P X: one matrix of 256 x 512 387, 258, 201, 138 / 277, 207, 168, 137; 8 of 300 x 700
// 502, 346, 279, 201 / 321, 244, 203, 201; 8 of 512 x 1024 724, 493, 381, 389 / 544, 443, 389, 470; 100 of 200 x 200 397, 309,
// 350, 339 / 368, 308, 324, 381; 24 of 360 x 1000 791, 612, 504, 506 / 506, 535, 517, 605.  The rule took the least or one
// within 3 % of it at 15 sizes.
inline OrthVariant orth_variant(int64_t n, int64_t A, int64_t B, bool symmetric, int64_t workgroups) {
    auto time = [&](int64_t ta, int64_t tb, int64_t tile) {
        const int64_t at = (A + ta - 1) / ta, bt = (B + tb - 1) / tb;
        int64_t tiles = at * bt;
        if (symmetric) {
            tiles = 0;
            for (int64_t i = 0; i < at; ++i) {
                const int64_t above = i * ta / tb;
                tiles += bt - (above < bt ? above : bt);
            }
        }
        return (n * tiles + workgroups - 1) / workgroups * tile;
    };
    const int64_t big = time(256, 256, 26), mid = time(256, 128, 16), small = time(128, 128, 10);
    const int64_t least = time(64, 64, 4);
    if (big <= mid && big <= small && big <= least) return kOrth256x256;
    if (mid <= small && mid <= least) return kOrth256x128;
    return small <= least ? kOrth128x128 : kOrth64x64;
}

}  // namespace moe
