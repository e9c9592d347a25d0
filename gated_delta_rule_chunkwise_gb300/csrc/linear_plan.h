// How a product of the linear operators is cut: columns of a tile, blocks that share its k blocks, and
// whether two blocks take a tile of twice the lanes; and where the accumulators are read.  Host code alone, so
// that both are checked without a GPU.
#pragma once
#include <algorithm>

namespace ldn {
namespace linear {

struct Plan {
    int bn, split;
    bool pair;
};

// Columns of a tile whose sums the first half of the epilogue's warps takes; the other takes the rest.
constexpr int half_columns(int bn) { return (bn / 2 + 15) & ~15; }

// Columns of tensor memory that a block allocates: two accumulators, of bn columns or, promoted, of what is
// read.  That is 32 columns at a time from each half's first on, so with 16 columns of a half (bn = 16, 32)
// 16 more, which hold no sum and are allocated all the same.
constexpr int tensor_columns(int bn, bool promote)
{
    const int first = half_columns(bn), reads = first + (bn - first + 31) / 32 * 32;
    const int each = !promote || bn > 32 ? bn : bn - first ? reads : 32;
    return each <= 16 ? 32 : each <= 32 ? 64 : each <= 64 ? 128 : each <= 128 ? 256 : 512;
}

// The cheapest of the cuts by a model of one block's time in cycles, fitted to both sides of each choice
// over 17 sizes from 1 x 4096 x 4096 to 8192 x 4096 x 4096:
// - a k block costs its products (2 a column) and 100 (a pair 20, having half as much to load), and 290 at
//   least: the 128 lanes of A are read in 70 cycles for each of four steps, however few the columns;
// - b_mn, columns that lie along memory: both operands come at 56 bytes a cycle and SM, 64 columns a load;
// - what every cut reads of HBM comes at 3250 bytes a cycle;
// - a tile's end that no other tile's products cover takes 12 a column, and a split one's exchange 190 a
//   column of a block's share and 250 a block (256 x 4096 to 4096: 64 columns 15.2 us, 128 in two halves
//   16.7; 64 x 4096 to 4096: 64 columns in quarters 10.9, in halves 11.6, whole 13.6);
// - eight blocks of a cluster find room for 13 clusters at once (fp32 64 x 1024 to 1024 in 16 of them 18.5 us,
//   in 8 of twice the columns 12.1).
// promote: sums stay in registers, of 128 columns where no pair shares them.
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
                if (promote && !pair && bn > 128) continue;
                const long long tiles = ((ni + lanes - 1) / lanes) * ((nj + bn - 1) / bn);
                if (split > 1 && (tiles * split > (split == 8 ? sms * 2 / 3 : sms) || split > kblocks || bn > 128 ||
                                  bn % (2 * split)))
                    continue;
                const double waves = (double)((tiles * blocks + sms - 1) / sms);
                const double loads = b_mn ? (128 + (pair ? bn / 2 : bn)) * 128 / 56.0 : 290.0;
                const double each = std::max(2.0 * bn + (pair ? 20 : 100), loads);
                const double products = waves * ((kblocks + split - 1) / split * npairs * each + 200);
                const double stream = ((double)ni + nj) * kblocks * 128 / 3250;
                const double cost = std::max(products, stream) + (split > 1 ? 190.0 * bn / split + 250 * split : 12.0 * bn) +
                                    (pair ? 500 : 0);
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
