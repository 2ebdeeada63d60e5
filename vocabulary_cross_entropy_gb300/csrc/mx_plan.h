// How mx_linear divides a product into tiles, and whether pairs of CTAs or single ones take
// them.  Host code only.
#pragma once

#include <stdint.h>

namespace vce {
namespace mx {

constexpr int kLinearTokens = 128;  // tokens per tile of a CTA (a pair: twice as many)
constexpr int kLinearRows = 256;    // classifier rows per tile; the last tiles may have half

struct LinearPlan {
    int64_t tiles_n, tiles_v;  // tiles of tokens and of classifier rows
    int64_t whole_v;           // the first so many tiles of rows have 256, the others 128
    double single, paired;     // rounds of single CTAs' tiles that either way takes
    bool pairs;
};

// Tiles go to the SMs in rounds, tile t to CTA t % sms.  What the last, partial round would
// hold is cut into tiles of half the rows where those still fit one round: half a round
// instead of one.
//
// Pairs of CTAs where they need less time: a round of theirs takes 0.93 of a round of single
// CTAs, their start as long as five stages more; but they have tiles of 256 tokens and no
// half tiles.  BF16 logits, single / pairs in us (cold L2): 4096 x 128256, 256 tokens 105 / 95, 384
// 146 / 179, 512 189 / 179, 640 234 / 259, 1024 359 / 337, 2048 672 / 642; 4096 x 32000, 1536
// tokens 128 / 117, 2048 189 / 188; 1792 x 4096 x 50304 242 / 232; 2048 x 1024 x 128256 216 / 218.
// (Pairs address scale tiles by 32-bit rows.)
inline LinearPlan plan_linear(int64_t n, int64_t v, int k_tiles, int sms) {
    LinearPlan p{};
    p.tiles_n = (n + kLinearTokens - 1) / kLinearTokens;
    const int64_t all = (v + kLinearRows - 1) / kLinearRows;
    const int64_t whole = all * p.tiles_n / sms * sms / p.tiles_n;  // tiles of rows in full rounds
    const int64_t halves = (v - whole * kLinearRows + 127) / 128;
    const bool cut = whole < all && halves * p.tiles_n <= sms;
    const int64_t full = (cut ? whole : all) * p.tiles_n, rounds = (full + sms - 1) / sms;
    // half tiles beyond what the last round of whole ones leaves free
    p.single = double(rounds) + (cut && halves * p.tiles_n > rounds * sms - full ? 0.5 : 0.0);
    p.whole_v = cut ? whole : all;
    p.tiles_v = cut ? whole + halves : all;

    const int64_t pair_n = (n + 2 * kLinearTokens - 1) / (2 * kLinearTokens), pair_tiles = pair_n * all, pairs = sms / 2;
    p.paired = 0.93 * double((pair_tiles + pairs - 1) / pairs) + 5.0 / k_tiles;
    const int64_t scale_rows = 2 * int64_t(k_tiles) * ((n > v ? n : v) / 128 + 4);
    p.pairs = n > kLinearTokens && p.paired < p.single && pair_tiles < 0x7fffffff && scale_rows < 0x7fffffff;
    if (p.pairs) {
        p.tiles_n = pair_n;
        p.tiles_v = p.whole_v = all;
    }
    return p;
}

}  // namespace mx
}  // namespace vce
