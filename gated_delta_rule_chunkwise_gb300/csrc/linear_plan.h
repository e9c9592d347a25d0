// How a product of the linear operators is cut: columns of a tile, blocks that share its k blocks, and
// whether two blocks take a tile of twice the lanes.  Host code alone, so that the plans are checked
// without a GPU.
#pragma once
#include <algorithm>

namespace ldn {
namespace linear {

struct Plan {
    int bn, split;
    bool pair;
};

// The cheapest of the cuts by a model of one block's time in cycles, fitted to both sides of each choice
// over 12 sizes from 1 x 4096 x 4096 to 2048 x 2048 x 2048: a k block costs its products (2 a column) and
// 100 (a pair 20, having half as much to load), and 290 at least; a tile its pipeline's filling and 12 a
// column of epilogue that no other tile's products cover; the exchange of a split 3500 and 16 a column.
// promote: sums in registers.  b_mn: the columns lie along memory, are loaded 64 at a time, and both operands come at 56 bytes a cycle.
inline Plan plan_for(long long ni, long long nj, int kblocks, int npairs, bool b_mn, bool promote, int sms)
{
    const int widths[] = {16, 32, 64, 96, 128, 160, 192, 224, 256};
    Plan best{0, 1, false};
    double least = 1e300;
    for (const int bn : widths) {
        if (b_mn && bn % 64) continue;
        if (best.bn && best.bn >= nj) break;   // narrower tiles already hold all columns
        for (int blocks = 1; blocks <= 8; blocks *= 2)
            for (int pair = 0; pair <= (blocks == 2 && bn % (b_mn ? 128 : 32) == 0); ++pair) {
                const int split = pair ? 1 : blocks, lanes = pair ? 256 : 128;
                if (promote && !pair && bn > 128) continue;   // the sums of half a tile stay in registers
                const long long tiles = ((ni + lanes - 1) / lanes) * ((nj + bn - 1) / bn);
                if (split > 1 && (tiles * split > sms || split > kblocks || bn > 128 || bn % (2 * split))) continue;
                const long long waves = (tiles * blocks + sms - 1) / sms;
                const double loads = b_mn ? (128 + (pair ? bn / 2 : bn)) * 128 / 56.0 : 290.0;
                const double each = std::max(2.0 * bn + (pair ? 20 : 100), loads);
                const double cost = waves * ((kblocks + split - 1) / split * npairs * each + 200) +
                                    12.0 * bn / split + (split > 1 ? 3500 + 16 * bn : 0) + (pair ? 500 : 0);
                if (cost < least) {
                    least = cost;
                    best = {bn, split, pair != 0};
                }
            }
    }
    return best;
}

}  // namespace linear
}  // namespace ldn
