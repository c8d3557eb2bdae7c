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

}  // namespace moe
