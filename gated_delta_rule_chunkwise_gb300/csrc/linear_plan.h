// How a product of the linear operators is cut: columns of a tile and blocks that share its k blocks.
// Host code alone, so that the plans are checked without a GPU.
#pragma once
#include <algorithm>

namespace ldn {
namespace linear {

struct Plan { int bn, split; };

// The cheapest of the cuts by a model of one block's time in cycles, fitted to both sides of each choice
// over 12 sizes from 1 x 4096 x 4096 to 2048 x 2048 x 2048: a k block costs its products (2 a column) and
// 100, and 290 at least (its loads); a tile its pipeline's filling and 12 a column of epilogue that no
// other tile's products cover; the exchange of a split 4500.
inline Plan plan_for(long long ni, long long nj, int kblocks, int npairs, int narrowest, int sms)
{
    Plan best{0, 1};
    double least = 1e300;
    for (int bn = narrowest; bn <= 256; bn *= 2) {
        if (best.bn && bn / 2 >= nj) break;   // half as wide would already hold all columns
        const long long tiles = ((ni + 127) / 128) * ((nj + bn - 1) / bn);
        for (int split = 1; split <= 8; split *= 2) {
            if (split > 1 && (tiles * split > sms || split > kblocks)) break;
            const long long waves = split > 1 ? 1 : (tiles + sms - 1) / sms;
            const int blocks = (kblocks + split - 1) / split * npairs;
            const double each = std::max(2.0 * bn + 100, 290.0);
            const double cost = waves * (blocks * each + 200) + 12.0 * bn / split + (split > 1 ? 4500 : 0);
            if (cost < least) {
                least = cost;
                best = {bn, split};
            }
        }
    }
    return best;
}

}  // namespace linear
}  // namespace ldn
