// The choice of kernel (linear_dev.h) of moe_linear, moe_mx_linear and
// moe_grouped_linear, and their workspaces.
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
    {kTile256x128, 256, 128, 0, 800, true, true, false, 5500.0},
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
LinearPlan plan(const LinearParams &p, bool any, bool mx = false)
{
    const int m = p.w_up ? 2 : 1, stages = (p.K + 63) / 64;
    const double weights = 2.0 * m * p.N * p.K;
    LinearPlan best = {any ? kAny64x64 : kTile64x64, 1};
    double least = 1e30;
    for (const Kind &k : kKinds) {
        if (k.any != any || (k.kind == kTile256x128 && !mx)) continue;
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

// ------------------------------------------------------------ MXFP4 operands

namespace {

int scale_pitch(const LinearParams &p) { return (p.K + 63) / 64 * 8; }  // 8 scales a stage
// the kernels copy scales as dwords
bool dwords(const LinearParams &p, const uint8_t *a, const uint8_t *b, int64_t ld, int rows)
{
    return p.K % 32 == 0 && (((uintptr_t)a | (uintptr_t)b) & 3) == 0 && (rows == 1 || ld % 4 == 0);
}
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
// rows of weight scales that the workspace has a copy of, and room for x's
size_t weight_scales(const MxParams &p)
{
    return dwords(p, p.ws, p.us, p.ldws, p.N) ? 0 : up256((size_t)(p.us ? 2 : 1) * p.N * scale_pitch(p));
}
size_t x_scales(const MxParams &p) { return up256((size_t)p.M * scale_pitch(p)); }

}  // namespace

size_t mx_linear_workspace(const MxParams &p) { return up256(linear_workspace(p)) + weight_scales(p) + x_scales(p); }

// A stage of 256 codes takes the bytes, reads and cycles of a 16-bit one of 64,
// so the estimate serves (all of it: it is the order that counts).  Measured with
// every kernel and split at 26 sizes of T = 1 .. 4096, the choice is 2% behind the
// best on average; furthest where K is one stage (4096 x 256 x 4096: 256 x 256
// 17.5 us, 256 x 128 14.3).  Both sides of some: 1 x 7168 x 3584 16 x 8 7.0 us
// (from Python), 64 x 32 9.7; 512 x 3584 x 7168 128 x 128 14.2, 256 x 128 23.1;
// 1024 x 7168 x 7168 256 x 128 40.0, 128 x 128 46.4, 256 x 256 50.2; 2048 x 3584 x
// 2 x 6144 256 x 128 55.6, 128 x 128 75, 256 x 256 67.7; 4096 x 7168 x 7168 256 x
// 256 112, 256 x 128 127.
LinearPlan mx_linear_plan(const MxParams &p) { return plan(p, false, true); }

hipError_t launch_mx_linear(const MxParams &params, bool f16, hipStream_t st)
{
    MxParams p = params;
    p.vec = fours(p);
    const bool wd = dwords(p, p.ws, p.us, p.ldws, p.N), xd = dwords(p, p.xs, nullptr, p.ldxs, p.M);
    if (!wd || !xd) {
        const int pitch = scale_pitch(p);
        uint8_t *at = reinterpret_cast<uint8_t *>(p.part) + up256(linear_workspace(p));
        const size_t wrows = wd ? 0 : (size_t)(p.us ? 2 : 1) * p.N;
        const hipError_t e = launch_mx_scale_rows(p.ws, wd ? nullptr : p.us, p.ldws, wd ? 0 : p.N, p.xs, p.ldxs, xd ? 0 : p.M, p.K / 8,
                                                  pitch, at, st);
        if (e != hipSuccess) return e;
        if (!wd) {
            p.ws = at;
            if (p.us) p.us = at + (size_t)p.N * pitch;
            p.ldws = pitch;
        }
        if (!xd) {
            p.xs = at + wrows * pitch;
            p.ldxs = pitch;
        }
    }
    const LinearPlan c = mx_linear_plan(p);
    if (f16) launch_mx_f16(p, c, st);
    else launch_mx_bf16(p, c, st);
    return hipGetLastError();
}

// -------------------------------------------------------------------- groups

namespace {

// A kernel's tile, and the time in ns of a stage of 64 of K (256 of codes) and
// of a block's start and end, per block and CU.
struct GroupedKind {
    int kind, rows, tokens, threads, each_ns, ends_ns;
    bool any;
};
constexpr GroupedKind kGroupedKinds[] = {
    {kTile64x32, 64, 32, 256, 130, 2350, false},    {kTile64x64, 64, 64, 256, 180, 2750, false},
    {kTile128x64, 128, 64, 512, 310, 4500, false},  {kTile128x128, 128, 128, 512, 500, 6000, false},
    {kTile256x128, 256, 128, 256, 950, 5000, false}, {kAny64x32, 64, 32, 256, 290, 1900, true},
    {kAny64x64, 64, 64, 256, 400, 3000, true},      {kAny128x128, 128, 128, 512, 950, 6500, true},
};

}  // namespace

// plan()'s estimate where the rows of each group are not known: as if the M
// rows fell on the groups at random, which leaves some of them empty where
// there are few rows, and a tile of each other group half full on average; and
// with the ends of a block, since a group's product is often a short one.
// Measured with every kernel at 36 sizes of 8 to 32768 rows in ragged groups, ten
// of them not used in the fit: the choice is 2% behind the best on average for
// 16-bit rows, 4% for MXFP4 ones, 5% for unaligned ones.  Furthest: MXFP4 1200 rows
// of 16 x 640 x 2 x 512, 256 x 128 12.6 us, 64 x 64 7.9 (below one block per CU only
// a part of a block's ends counts, which favours large tiles); MXFP4 128 rows of 8 x
// 4096 x 4096, 64 x 32 20.6, 64 x 64 16.1; 1024 of the same in 16 bits, 128 x 128
// 88.8, 256 x 128 70.9; unaligned 4000 of 8 x 2049 x 1025, 128 x 128 82, 64 x 64 66.
// Both sides of some others: 512 rows of 64 x 2048 x 3584 64 x 32 146 us, 256 x 128
// 163; 4096 of 64 x 2048 x 2 x 1408 256 x 128 158, 128 x 128 174, 64 x 32 213; 1000 of
// 1 x 2048 x 2048 128 x 64 15.8, 64 x 64 18.6, 128 x 128 19.2; 16 of 896 x 1024 x 2 x
// 512 64 x 32 8.5, 64 x 64 9.1.  The kernels of 16 rows lost at every size (16 of
// 896: 13 us).  Kind -1: too large for any.
LinearPlan grouped_plan(const GroupedParams &p, bool mx)
{
    const bool any = !mx && !(pieces(p) && p.wstride % 8 == 0);
    const int m = p.w_up ? 2 : 1, stages = (p.K + 63) / 64;
    const double active = p.groups * (1.0 - std::exp(-(double)p.M / p.groups));
    const double weights = 2.0 * m * active * p.N * p.K;
    LinearPlan best = {-1, 1};
    double least = 1e30;
    for (const GroupedKind &k : kGroupedKinds) {
        if (k.any != any) continue;
        const double columns = std::ceil((double)p.N * m / k.rows);
        // (a launch holds fewer than 2^32 threads)
        if (columns * ((double)p.M / k.tokens + std::min(p.groups, p.M)) * k.threads > 4.2e9) continue;
        const double full = columns * std::max(active, (double)p.M / k.tokens + 0.5 * active) / kCus;
        const double work = std::max(1.0, full) * k.each_ns * stages + full * k.ends_ns;
        const double ns = std::max(work, weights / 5600.0) + 0.1 * work;
        if (ns < least) {
            least = ns;
            best = {k.kind, 1};
        }
    }
    return best;
}

hipError_t launch_grouped(const GroupedParams &params, const LinearPlan &c, bool f16, hipStream_t st)
{
    GroupedParams p = params;
    p.vec = fours(p);
    if (f16) launch_grouped_f16(p, c, st);
    else launch_grouped_bf16(p, c, st);
    return hipGetLastError();
}

hipError_t launch_grouped_mx(const GroupedMxParams &params, const LinearPlan &c, bool f16, hipStream_t st)
{
    GroupedMxParams p = params;
    p.vec = fours(p);
    if (f16) launch_grouped_mx_f16(p, c, st);
    else launch_grouped_mx_bf16(p, c, st);
    return hipGetLastError();
}

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
