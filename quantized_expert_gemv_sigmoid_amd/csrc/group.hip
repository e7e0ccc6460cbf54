// The choices of tokens sorted by expert (moe_group), and the experts' rows
// added up again (moe_combine).
#include <algorithm>
#include <type_traits>

#include "../../include/moe.h"
#include "common.h"

namespace moe {

namespace {

// A counting sort that keeps the order of the choices inside an expert, so the
// same call always gives the same places.  Each wave owns a run of choices and
// goes through it 64 at a time; a choice's rank among the wave's is what the
// wave has counted of its expert so far plus the lower lanes that chose it too.
// Up to 1024 choices in one launch (16 of 896 experts 3.4 us, a chain of loads
// and barriers; 16 waves for them took 6.9), more in two: 32768 of 64 experts 5
// and 6-7 us, 32 blocks of 1024 (8 of 4096: 6.5 and 13).  The bytes are nothing
// (0.5 MB); each launch is such a chain, the second one's with the counts of all
// blocks in it.
constexpr int kGroupWaves = 16;
constexpr int kGroupThreads = kGroupWaves * 64;

// lanes whose id equals this lane's, for ids below 2^10, kNone among them
__device__ __forceinline__ uint64_t same_lanes(int id, bool on)
{
    uint64_t m = __ballot(on);
#pragma unroll
    for (int b = 0; b < 10; b++) {
        const uint64_t v = __ballot((id >> b) & 1);
        m &= (id >> b) & 1 ? v : ~v;
    }
    return m;
}

// choices per wave of n (whole steps of 64, so that few choices take few
// waves), and the waves that have any
__device__ __forceinline__ int wave_run(int n) { return ((n + kGroupWaves - 1) / kGroupWaves + 63) & ~63; }
__device__ __forceinline__ int waves_of(int n) { return n > 0 ? (n + wave_run(n) - 1) / wave_run(n) : 0; }

// counts[w][e] of the block's waves, over choices [a, b) of the block
__device__ __forceinline__ void count_choices(const int32_t *ids, int a, int b, int E, int *counts)
{
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int per = wave_run(b - a), a0 = a + wv * per, b0 = min(b, a0 + per);
    int *mine = counts + wv * E;
    for (int i = a0; i < b0; i += 64) {
        const int id = i + lane < b0 ? ids[i + lane] : -1;
        const bool on = (uint32_t)id < (uint32_t)E;
        const uint64_t same = same_lanes(id, on);
        if (on && (same & ((1ull << lane) - 1)) == 0) mine[id] += __popcll(same);  // (one lane per expert)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// Grid: blocks of `per` choices each.  One block does all; of several, a first
// launch writes their counts to hist [blocks][E].
__global__ __launch_bounds__(kGroupThreads) void k_group_count(const int32_t *ids, int R, int per, int E, int32_t *hist)
{
    __shared__ int lds_i[kGroupWaves * kMaxExperts];
    const int a = (int)blockIdx.x * per, b = min(R, a + per);
    const int waves = waves_of(b - a);
    for (int i = threadIdx.x; i < waves * E; i += kGroupThreads) lds_i[i] = 0;
    __syncthreads();
    count_choices(ids, a, b, E, lds_i);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kGroupThreads) {
        int s = 0;
        for (int w = 0; w < waves; w++) s += lds_i[w * E + e];
        hist[blockIdx.x * E + e] = s;
    }
}

__global__ __launch_bounds__(kGroupThreads) void k_group_place(const int32_t *ids, int R, int per, int k, int E,
                                                               const int32_t *hist, int32_t *offsets, int32_t *tokens,
                                                               int32_t *places)
{
    __shared__ int lds_i[kGroupWaves * kMaxExperts], sums[kGroupWaves];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int a = (int)blockIdx.x * per, b = min(R, a + per);
    const int waves = waves_of(b - a);
    for (int i = threadIdx.x; i < waves * E; i += kGroupThreads) lds_i[i] = 0;
    __syncthreads();
    count_choices(ids, a, b, E, lds_i);
    __syncthreads();
    // thread e: the choices of expert e in the blocks before this one, in all,
    // and before each of its waves
    const int e = threadIdx.x;
    int before = 0, total = 0;
    if (e < E) {
        for (int w = 0; w < waves; w++) {
            const int c = lds_i[w * E + e];
            lds_i[w * E + e] = total;
            total += c;
        }
        if (gridDim.x > 1) {
            total = 0;
            for (int g0 = 0; g0 < (int)gridDim.x; g0 += 16) {  // (16 loads on the way at once)
                int c[16];
#pragma unroll
                for (int i = 0; i < 16; i++) c[i] = hist[min(g0 + i, (int)gridDim.x - 1) * E + e];
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    if (g0 + i < (int)blockIdx.x) before += c[i];
                    if (g0 + i < (int)gridDim.x) total += c[i];
                }
            }
        }
    }
    int scan = total;  // over the experts
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(scan, d, 64);
        if (lane >= d) scan += v;
    }
    if (lane == 63) sums[wv] = scan;
    __syncthreads();
    int base = scan - total;
    for (int w = 0; w < wv; w++) base += sums[w];
    if (e < E) {
        for (int w = 0; w < waves; w++) lds_i[w * E + e] += base + before;
        if (blockIdx.x == 0) {
            offsets[e] = base;
            if (e == E - 1) offsets[E] = base + total;
        }
    }
    __syncthreads();
    const int run = wave_run(b - a), a0 = a + wv * run, b0 = min(b, a0 + run);
    int *mine = lds_i + wv * E;
    for (int i = a0; i < b0; i += 64) {
        const int c = i + lane;
        const int id = c < b0 ? ids[c] : -1;
        const bool on = (uint32_t)id < (uint32_t)E;
        const uint64_t same = same_lanes(id, on), lower = same & ((1ull << lane) - 1);
        // (all lanes read before one of them writes, for the next 64 to read)
        const int first = on ? mine[id] : 0, place = on ? first + __popcll(lower) : -1;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (on && lower == 0) mine[id] = first + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (on) tokens[place] = (int)((uint32_t)c / (uint32_t)k);
        if (c < b0) places[c] = place;
    }
}

// --------------------------------------------------------------- combination

// eight values of a row as they are in memory (n of them), and in fp32
struct Raw8 {
    uint4 q[2];
};
__device__ __forceinline__ Raw8 load8_raw(const void *p, int type, int64_t at, int n)
{
    Raw8 r = {{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}};
    if (type == MOE_F32) {
        const float *f = reinterpret_cast<const float *>(p) + at;
        if (n >= 8) {
            __builtin_memcpy(&r, f, 32);
        } else {
            float v[8] = {};
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (j < n) v[j] = f[j];
            __builtin_memcpy(&r, v, 32);
        }
        return r;
    }
    const uint16_t *h = reinterpret_cast<const uint16_t *>(p) + at;
    if (n >= 8) {
        __builtin_memcpy(&r, h, 16);
    } else {
        uint16_t v[8] = {};
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (j < n) v[j] = h[j];
        __builtin_memcpy(&r, v, 16);
    }
    return r;
}
__device__ __forceinline__ void to_f32(const Raw8 &r, int type, float (&v)[8])
{
    if (type == MOE_F32) {
        __builtin_memcpy(v, &r, 32);
        return;
    }
    uint16_t q[8];
    __builtin_memcpy(q, &r, 16);
#pragma unroll
    for (int j = 0; j < 8; j++)
        v[j] = type == MOE_F16 ? (float)__builtin_bit_cast(_Float16, q[j]) : __uint_as_float((uint32_t)q[j] << 16);
}

// A thread adds eight columns of a token's rows, in the order of its choices,
// fp32 throughout; YT: the rows' type.  B rows are on the way at once; a choice
// without a row reads one that is there and adds nothing.  Bound by memory: 4096
// tokens of 8 rows of 2048 bf16 with a residual, rows in any order, 31-33 us (5350-
// 5100 GB/s; four rows on the way and a branch for each 45), of fp32 rows 54-57
// (5600-5300); one token of 16 5 us, a chain of three loads (place, its weight, its
// row) in one block.
template <int YT, int B>
__global__ __launch_bounds__(256) void k_group_combine(CombineParams p)
{
    const int t = blockIdx.y + p.t0, n0 = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (n0 >= p.n) return;
    const int n = min(8, p.n - n0);
    const int32_t *pl = p.places + (int64_t)t * p.k;
    const float *wt = p.weights ? p.weights + (int64_t)t * p.k : nullptr;
    float s[8] = {};
    Raw8 res = {};
    if (p.res) res = load8_raw(p.res, p.res_type, (int64_t)t * p.ldr + n0, n);
    for (int j0 = 0; j0 < (p.rows > 0 ? p.k : 0); j0 += B) {
        Raw8 v[B];
        float w[B];
        bool on[B];
        int64_t at[B];
#pragma unroll
        for (int j = 0; j < B; j++) {
            const int place = j0 + j < p.k ? pl[j0 + j] : -1;
            on[j] = (uint32_t)place < (uint32_t)p.rows;
            w[j] = on[j] ? (wt ? wt[j0 + j] : 1.0f) : 0.0f;
            at[j] = (int64_t)(on[j] ? place : 0) * p.ldy + n0;
        }
#pragma unroll
        for (int j = 0; j < B; j++)
            if (j0 + j < p.k) v[j] = load8_raw(p.y, YT, at[j], n);
#pragma unroll
        for (int j = 0; j < B; j++) {
            if (!on[j]) continue;
            float f[8];
            to_f32(v[j], YT, f);
#pragma unroll
            for (int i = 0; i < 8; i++) s[i] = fmaf(w[j], f[i], s[i]);
        }
    }
    if (p.res) {
        float r[8];
        to_f32(res, p.res_type, r);
#pragma unroll
        for (int i = 0; i < 8; i++) s[i] += r[i];
    }
    const int64_t at = (int64_t)t * p.ldo + n0;
    if (p.out_type == MOE_F32) {
        float *o = reinterpret_cast<float *>(p.out) + at;
        if (n == 8) {
            __builtin_memcpy(o, s, 32);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (i < n) o[i] = s[i];
        }
        return;
    }
    uint16_t h[8], *o = reinterpret_cast<uint16_t *>(p.out) + at;
#pragma unroll
    for (int i = 0; i < 8; i++)
        h[i] = p.out_type == MOE_F16 ? __builtin_bit_cast(uint16_t, (_Float16)s[i]) : f32_to_bf16_rne(s[i]);
    if (n == 8) {
        __builtin_memcpy(o, h, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) o[i] = h[i];
    }
}

// choices of a block and the blocks of a call
int64_t group_per(int64_t R) { return std::max<int64_t>(1024, (R + 63) / 64); }

}  // namespace

// (at least what a call of fewer choices takes)
size_t group_workspace(int64_t R, int E)
{
    const int64_t blocks = (R + group_per(R) - 1) / group_per(R);
    return blocks > 1 ? std::max<size_t>(256, (size_t)blocks * E * 4) : 256;
}

// (R: 2^26 at most)
hipError_t launch_group(const int32_t *ids, int64_t R, int k, int E, int32_t *offsets, int32_t *tokens, int32_t *places,
                        void *ws, hipStream_t st)
{
    const int per = (int)group_per(R), blocks = (int)std::max<int64_t>(1, (R + per - 1) / per);
    int32_t *hist = reinterpret_cast<int32_t *>(ws);
    if (blocks > 1) k_group_count<<<blocks, kGroupThreads, 0, st>>>(ids, (int)R, per, E, hist);
    k_group_place<<<blocks, kGroupThreads, 0, st>>>(ids, (int)R, per, k, E, hist, offsets, tokens, places);
    return hipGetLastError();
}

hipError_t launch_group_combine(const CombineParams &params, int y_type, hipStream_t st)
{
    CombineParams p = params;
    const int total = p.T;
    for (p.t0 = 0; p.t0 < total; p.t0 += 65535) {
        const dim3 grid((p.n + 2047) / 2048, std::min(65535, total - p.t0));
        auto go = [&](auto type) {
            constexpr int YT = decltype(type)::value;
            if (p.k <= 8) k_group_combine<YT, 8><<<grid, 256, 0, st>>>(p);
            else k_group_combine<YT, 16><<<grid, 256, 0, st>>>(p);
        };
        if (y_type == MOE_F32) go(std::integral_constant<int, MOE_F32>{});
        else if (y_type == MOE_F16) go(std::integral_constant<int, MOE_F16>{});
        else go(std::integral_constant<int, MOE_BF16>{});
    }
    return hipGetLastError();
}

}  // namespace moe
