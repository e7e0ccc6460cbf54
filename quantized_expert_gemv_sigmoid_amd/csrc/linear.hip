// moe_linear's choice of kernel (linear_dev.h), and its workspace.
#include <algorithm>
#include <cmath>

#include "common.h"

namespace moe {

namespace {

constexpr int kCus = 256;
constexpr size_t kPartBytes = (size_t)64 << 20;  // partial sums of a call stay below this
constexpr int kMaxSplit = 8;                    // parts of K, of four stages at least

bool aligned16(const void *q) { return ((uintptr_t)q & 15) == 0; }

// rows of x and w start at multiples of 16 bytes and hold whole 16-byte pieces
bool pieces(const LinearParams &p)
{
    return p.K % 8 == 0 && p.ldx % 8 == 0 && p.ldw % 8 == 0 && aligned16(p.x) && aligned16(p.w) && aligned16(p.w_up);
}

// four outputs at a time: their rows' places are aligned for it
bool fours(const LinearParams &p)
{
    const bool res = !p.res || (p.ldr % 4 == 0 && ((uintptr_t)p.res & (p.res_f32 ? 15 : 7)) == 0);
    return p.N % 4 == 0 && p.ldo % 4 == 0 && ((uintptr_t)p.out_half & 7) == 0 && aligned16(p.out_f32) && res;
}

size_t part_bytes(const LinearParams &p, int ksplit)
{
    return (size_t)ksplit * (p.w_up ? 2 : 1) * p.M * ((p.N + 3) & ~3) * 4;
}

// A kernel's tile (weight rows, of both matrices where gated, by tokens); the
// time in ns of a stage of 64 of K, base_ns + each_ns per block and CU: their
// average where several blocks share a CU, otherwise the busiest CU's, which
// takes them one after the other; and the rate at which it streams weights
// (bytes per ns).
struct Kind {
    int kind, rows, tokens, base_ns, each_ns;
    bool shared, split, any;
    double rate;
};
constexpr Kind kKinds[] = {
    {kFew1, 16, 8, 0, 55, true, false, false, 5300.0},
    {kFew2, 16, 16, 0, 58, true, false, false, 5200.0},
    {kFew4, 16, 32, 0, 80, true, false, false, 4600.0},
    {kTile64x32, 64, 32, 30, 145, true, true, false, 5500.0},
    {kTile64x64, 64, 64, 20, 195, true, true, false, 5500.0},
    {kTile128x64, 128, 64, 0, 320, false, true, false, 5500.0},
    {kTile128x128, 128, 128, 0, 470, false, true, false, 5500.0},
    {kBig, 256, 256, 0, 1270, false, true, false, 5500.0},
    {kAny64x32, 64, 32, 170, 345, true, true, true, 5500.0},
    {kAny64x64, 64, 64, 200, 400, true, true, true, 5500.0},
    {kAny128x128, 128, 128, 0, 890, false, true, true, 5500.0},
};

// The kernel and split of K of the least estimated time: a launch, the
// stages of a CU or the weights' way from memory, and with a split the partial
// sums' way to the join and its launch.  The constants of kKinds are fits to
// the kernels' measured times with inputs that the caches hold.  Over 128
// calls of M = 1 .. 4096 at ten (K, N) from 515 x 333 to 7168 x 3584, plain
// and gated, timed with every kernel and split, the choice is 2.5% behind the
// best one on average.  It is furthest behind where the shared kinds' blocks
// just exceed the CUs, since their average misses the CUs that hold two: 266
// blocks of 64 x 64 for 1200 x 7168 x 896 take 42 us (128 x 128 in two parts
// 30), 336 for 333 x 7168 x 3584 42 us (128 x 128 in two parts 30).
// Both sides of some others: 24 x 1117 x 2049 64 x 32 in four parts 10.0 us, whole
// 10.2; 200 x 3584 x 7168 128 x 64 19.5, 64 x 64 21.4, 128 x 128 23.9; 800 x
// 1117 x 2049 64 x 64 19.1, 128 x 128 19.9; 333 x 3585 x 3587 128 x 128 in two
// parts 30.8, 64 x 64 in two 38.5; 4096 x 3584 x 7168 256 x 256 165, 128 x 128
// 246; 9 x 3584 x 7168 16 x 16 10.4, 64 x 32 11.3.
LinearPlan plan(const LinearParams &p, bool any)
{
    const int m = p.w_up ? 2 : 1, stages = (p.K + 63) / 64;
    const double weights = 2.0 * m * p.N * p.K;
    LinearPlan best = {any ? kAny64x64 : kTile64x64, 1};
    double least = 1e30;
    for (const Kind &k : kKinds) {
        if (k.any != any) continue;
        const double tiles = (double)((p.N * (int64_t)m + k.rows - 1) / k.rows) * ((p.M + k.tokens - 1) / k.tokens);
        for (int ks = 1; ks <= (k.split ? kMaxSplit : 1); ks *= 2) {
            if (ks > 1 && (stages < 4 * ks || tiles * ks > 4 * kCus || part_bytes(p, ks) > kPartBytes)) break;
            const double full = tiles * ks / kCus, each = k.shared ? std::max(1.0, full) : std::ceil(full);
            const double work = (k.base_ns + each * k.each_ns) * ((stages + ks - 1) / ks);
            // (a tenth of the work: between two that wait for memory, the one with less of it)
            double ns = 3500.0 + std::max(work, weights / k.rate) + 0.1 * work;
            if (ks > 1) ns += 6000.0 + part_bytes(p, ks) / 3000.0;
            if (ns < least) {
                least = ns;
                best = {k.kind, ks};
            }
        }
    }
    return best;
}

}  // namespace

// (a bound that grows with the tokens: a call of fewer may split K where one
// of more does not)
size_t linear_workspace(const LinearParams &p)
{
    int ks = kMaxSplit;
    while (ks > 1 && (p.K + 63) / 64 < 4 * ks) ks /= 2;
    return ks > 1 ? std::max<size_t>(256, std::min(kPartBytes, part_bytes(p, ks))) : 256;
}

LinearPlan linear_plan(const LinearParams &p) { return plan(p, !pieces(p)); }

hipError_t launch_linear(const LinearParams &params, bool f16, hipStream_t st)
{
    LinearParams p = params;
    p.vec = fours(p);
    const LinearPlan c = linear_plan(p);
    if (f16) launch_linear_f16(p, c, st);
    else launch_linear_bf16(p, c, st);
    return hipGetLastError();
}

}  // namespace moe
