// Routing from given logits: softmax or sigmoid scores, selection bias,
// groups, top-k, renormalised weights (moe_gate).
//
// One wave per token: lane l holds experts l, l + 64, ...  Selection values
// are compared as doubles, so that experts whose fp32 values would round
// together keep their order; but only for the few experts that can be among
// the best k:
//
//   - every expert gets an fp32 value a in the order of the selection values
//     up to a margin d: the logit itself where there is no bias (both scores
//     grow with it), else the score in fp32 plus the bias;
//   - t, at most the k-th largest of the lanes' maxima, is a lower bound of
//     the k-th largest a, so the best k are among the experts with
//     a >= t - 2 d (about 20 of 896 for k = 16), which are put one to a lane;
//   - these get their scores as doubles, and their ranks by counting.
//
// Where more than 64 experts stay (equal logits), or two groups' values are
// too close to tell apart in fp32, the token takes `whole`: all values as
// doubles, k rounds of a wave-wide maximum.  A value of -inf marks an expert
// that takes no part, and a NaN one ranks as +inf.
//
// What bounds it: 16384 tokens of 896 fp32 logits, k = 16, sigmoid with a
// bias: 24.4 us with the counts, of which reading the logits is 11.9 at the
// card's copy rate.  The rest is vector instructions, about 500 per token
// (two transcendental ones per expert, the candidates' doubles), at the four
// waves per SIMD that 128 registers allow: five waves with 96 cost more in
// spills than they hide (28.4 us).  All values as doubles and k rounds of a
// maximum took 175 us.  Up to a few hundred tokens it is the launches.
#include <math.h>

#include "common.h"

namespace moe {

namespace {

constexpr int kGateWaves = 8;

template <typename L>
__device__ __forceinline__ float logit_f32(L v);
template <>
__device__ __forceinline__ float logit_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float logit_f32<_Float16>(_Float16 v) { return (float)v; }
template <>
__device__ __forceinline__ float logit_f32<uint16_t>(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// exp(x) to about 2^-52: 2^n e^r with r = x - n ln 2 (ln 2 in two parts),
// |r| <= ln(2) / 2, and e^r by its Taylor series to r^13 (the next term is
// below 2^-57); past the doubles' range inf and 0
__device__ __forceinline__ double exp64(double v)
{
    const double x = fmin(fmax(v, -1100.0), 1100.0);
    const double n = rint(x * 1.4426950408889634);
    double r = fma(n, -0.6931471803691238, x);
    r = fma(n, -1.9082149292705877e-10, r);
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return v != v ? v : ldexp(p, (int)n);
}

template <int CTRL>
__device__ __forceinline__ float dpp_f(float old, float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float wave_max(float v)
{
    v = fmaxf(v, dpp_f<0xB1>(v, v));   // quad_perm [1,0,3,2]
    v = fmaxf(v, dpp_f<0x4E>(v, v));   // quad_perm [2,3,0,1]
    v = fmaxf(v, dpp_f<0x141>(v, v));  // row_half_mirror
    v = fmaxf(v, dpp_f<0x140>(v, v));  // row_mirror
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)u, CTRL, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum64(double v)
{
    v += dpp_d<0xB1>(v);
    v += dpp_d<0x4E>(v);
    v += dpp_d<0x141>(v);
    v += dpp_d<0x140>(v);
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}
__device__ __forceinline__ double wave_max64(double v)
{
    v = fmax(v, dpp_d<0xB1>(v));
    v = fmax(v, dpp_d<0x4E>(v));
    v = fmax(v, dpp_d<0x141>(v));
    v = fmax(v, dpp_d<0x140>(v));
    v = fmax(v, __shfl_xor(v, 16, 64));
    return fmax(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ int wave_min(int v)
{
    v = min(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true));
    v = min(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true));
    v = min(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true));
    v = min(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true));
    v = min(v, __shfl_xor(v, 16, 64));
    return min(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ int below(uint64_t mask)  // set bits below this lane
{
    return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

struct Pick {  // lane j < k: the j-th choice, id -1 where there is none
    int id;
    double s;
};

// the score of a logit: softmax with maximum m (of the experts that take
// part) and the sum of exp(l - m)
template <bool SOFT>
__device__ __forceinline__ double score_of(float l, float m, double sum)
{
    // (+inf - +inf: the limit, 0)
    if (SOFT) return exp64(l == m ? 0.0 : (double)l - (double)m) / sum;
    return 1.0 / (1.0 + exp64(-(double)l));
}

__device__ __forceinline__ int group_of(const GateParams &p, int e) { return (int)((uint32_t)e * p.group_inv >> 20); }

// LDS of a wave: every expert's value (in `choose` the groups' part, as
// floats; in `whole`), or the candidates
struct GateCands {
    int id[64];
    double c[64];  // selection values
    double s[64];  // scores and ids by rank
    int by[64];
};
template <int EPL>
union GateLds {
    double v[64 * EPL];
    GateCands n;
};

// Lane g < groups: whether group g stays, of the values v[E] in LDS.  P lanes
// to a group: each takes every P-th of its experts, then their two largest
// join.  `mine`: lane g's group value; `terms`: the magnitudes of what it is
// the sum of, 0 for an infinite one (those are exact).
template <typename T>
__device__ __forceinline__ bool group_stays(const GateParams &p, const T *v, T &mine, T &terms)
{
    const T ninf = -INFINITY;
    const int lane = threadIdx.x & 63, size = p.E / p.groups, P = 1 << (31 - __builtin_clz(64 / p.groups));
    const int g = lane / P;
    T v1 = ninf, v2 = ninf;
    if (g < p.groups) {
        for (int j = lane % P; j < size; j += P) {
            const T x = v[g * size + j];
            v2 = fmax(v2, fmin(v1, x));
            v1 = fmax(v1, x);
        }
    }
    for (int d = 1; d < P; d <<= 1) {
        const T o1 = __shfl_xor(v1, d, 64), o2 = __shfl_xor(v2, d, 64);
        v2 = fmax(fmax(v2, o2), fmin(v1, o1));
        v1 = fmax(v1, o1);
    }
    v2 = p.top2 && v2 != ninf ? v2 : (T)0;
    mine = __shfl(v1 + v2, min(lane * P, 63), 64);
    terms = __shfl(fabs(v1) == -ninf ? (T)0 : fabs(v1) + fabs(v2), min(lane * P, 63), 64);
    int rank = 0;
    for (int i = 0; i < p.groups; i++) {
        const T o = __shfl(mine, i, 64);
        rank += o > mine || (o == mine && i < lane) ? 1 : 0;
    }
    return lane < p.groups && rank < p.top_groups;
}

// everything as doubles in LDS, k rounds of a maximum
template <bool SOFT, typename L>
__device__ __forceinline__ Pick whole(const GateParams &p, const L *row, const float *biases, double *v, float m, double sum)
{
    const int lane = threadIdx.x & 63;
    const double ninf = -INFINITY;
#pragma unroll 1
    for (int e0 = lane; e0 < p.E; e0 += 256) {  // (four logits on the way at a time)
        float l4[4];
#pragma unroll
        for (int i = 0; i < 4; i++) l4[i] = logit_f32<L>(row[min(e0 + 64 * i, p.E - 1)]);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int e = e0 + 64 * i;
            if (e >= p.E) break;
            const float l = l4[i], b = biases[e];
            const double x = score_of<SOFT>(l, m, sum) + b;
            v[e] = l != -INFINITY && b != -INFINITY ? (x != x ? (double)INFINITY : x) : ninf;
        }
    }
    __builtin_amdgcn_wave_barrier();
    uint64_t kept = ~0ull;
    if (p.groups > 1) {
        double value, terms;
        kept = __builtin_amdgcn_ballot_w64(group_stays<double>(p, v, value, terms));
    }
    Pick mine = {-1, 0.0};
    double best = ninf;  // the lane's largest, and whose it is
    int id = 0;
    bool look = true;
#pragma unroll 1
    for (int j = 0; j < p.k; j++) {
        if (look) {
            best = ninf;
#pragma unroll 4
            for (int e = lane; e < p.E; e += 64) {
                const double x = v[e];
                const bool more = x > best && (p.groups == 1 || ((kept >> group_of(p, e)) & 1));  // (strict: the lower id of a tie)
                best = more ? x : best;
                id = more ? e : id;
            }
        }
        const double top = wave_max64(best);
        if (top == ninf) break;
        const int first = wave_min(best == top ? id : 1 << 30);
        if (lane == j) mine.id = first;
        look = id == first && best == top;
        if (look) v[first] = ninf;
        __builtin_amdgcn_wave_barrier();
    }
    if (mine.id >= 0) mine.s = score_of<SOFT>(logit_f32<L>(row[mine.id]), m, sum);
    return mine;
}

// a value near t may be off by this much, and so may the order of two
__device__ __forceinline__ float margin(bool by_logit, float t)
{
    // By logit: two logits closer than this may have equal scores as doubles.
    // Else: the fp32 score is off by less than 2^-21 (exp_hw(x) is within
    // (1 + 1.45 |x|) 2^-23 of itself, which s (1 - s), or e^x for the
    // softmax, takes below 2^-22; and a few roundings), the sum with the bias
    // by its rounding.
    return by_logit ? 4.8e-7f * fabsf(t) + 1e-9f : 4.8e-7f + 2.4e-7f * fabsf(t);
}

// the logits of a row of E that lane l holds: experts l, l + 64, ...; past
// the end 0 (a buffer's bounds: one address for all of them)
template <int EPL, typename L>
__device__ __forceinline__ void load_row(const L *row, int E, float (&l)[EPL])
{
    const __amdgpu_buffer_rsrc_t r = grsrc(row, (uint32_t)(E * sizeof(L)));
    const int at = (threadIdx.x & 63) * (int)sizeof(L);
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        if constexpr (sizeof(L) == 4)
            l[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, at + i * 256, 0, 0));
        else
            l[i] = logit_f32<L>(__builtin_bit_cast(L, __builtin_amdgcn_raw_buffer_load_b16(r, at + i * 128, 0, 0)));
    }
}

// the same lane number, but not known to be: what follows from it is computed
// where it is used instead of being kept in registers over the token loop
__device__ __forceinline__ int lane_here()
{
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// The choices of one token from its logits l and the biases in LDS (-inf: no
// expert, or one switched off; 0 without a bias).  l is free, and filled with
// the logits of the row `next`, once the experts' values are known.
template <int EPL, bool SOFT, bool by_logit, typename L>
__device__ __forceinline__ Pick choose(const GateParams &p, const L *row, const L *next, float (&l)[EPL],
                                       const float *biases, GateLds<EPL> &lds)
{
    const int lane = lane_here();
    const float ninf = -INFINITY;
    GateCands &w = lds.n;
    float a[EPL], bias[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) bias[i] = biases[lane + 64 * i];
    float m = ninf;
    double sum = 1.0;
    if (SOFT) {
#pragma unroll
        for (int i = 0; i < EPL; i++) m = fmaxf(m, bias[i] != ninf ? l[i] : ninf);
        m = wave_max(m);
        if (!by_logit || !p.renorm) {  // (renormalised weights do not need it)
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; i++) {
                const double e = exp64(l[i] == m ? 0.0 : (double)l[i] - (double)m);
                sum += l[i] != ninf && bias[i] != ninf ? e : 0.0;
                __builtin_amdgcn_sched_barrier(0);  // (one after the other: few registers)
            }
            sum = wave_sum64(sum);
        }
    }
    const float inv = (float)(1.0 / sum);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        float v = l[i];
        if (!by_logit) v = SOFT ? exp_hw(v == m ? 0.0f : v - m) * inv : sigmoid_hw(v);
        a[i] = l[i] != ninf ? v + bias[i] : ninf;  // (-inf: takes no part; without a bias + 0)
        nan |= a[i] != a[i];
    }
    if (__builtin_amdgcn_ballot_w64(nan)) {
        bool hit = false;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            a[i] = a[i] != a[i] ? (bias[i] != ninf ? (float)INFINITY : ninf) : a[i];
            hit |= l[i] != l[i] && bias[i] != ninf;
        }
        if (SOFT && by_logit && __builtin_amdgcn_ballot_w64(hit)) {  // every score is NaN
            sum = NAN;
#pragma unroll
            for (int i = 0; i < EPL; i++) a[i] = a[i] != ninf ? (float)INFINITY : ninf;
        }
    }
    load_row<EPL, L>(next, p.E, l);
    // logits between which every two have different scores as doubles (the
    // sigmoid's reach 1, and both scores 0, further out)
    const float high = !by_logit || SOFT ? (float)INFINITY : 20.0f;
    const float low = !by_logit ? ninf : SOFT ? m - 700.0f : -700.0f;

    bool slow = false;
    if (p.groups > 1) {
        float *v = reinterpret_cast<float *>(lds.v);
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (lane + 64 * i < p.E) v[lane + 64 * i] = a[i];
        __builtin_amdgcn_wave_barrier();
        float mine, terms;
        const bool keep = group_stays<float>(p, v, mine, terms), drop = lane < p.groups && !keep;
        const uint64_t kept = __builtin_amdgcn_ballot_w64(keep);
        // Every group's value within its bounds: the margins of its one or two
        // terms, whose own sizes count (two that cancel leave a sum near 0).
        // Of a term's 2.4e-7 |v| its rounding takes 0.6e-7, the sum's as much,
        // the bound's as much; a finite sum past fp32 may be anything.
        const float err = by_logit ? 2.0f * margin(true, terms) : margin(false, terms) + (p.top2 ? 4.8e-7f : 0.0f);
        const bool known = terms < INFINITY;
        const float least = known ? mine - err : ninf, most = known ? mine + err : INFINITY;
        const float in = -wave_max(keep ? -least : ninf), out = wave_max(drop ? most : ninf);  // the last kept, the first not
        slow = out != ninf && (!(in > out) || out > high || in < low);
#pragma unroll
        for (int i = 0; i < EPL; i++) a[i] = (kept >> (group_of(p, lane + 64 * i) & 63)) & 1 ? a[i] : ninf;
        __builtin_amdgcn_wave_barrier();
    }

    // t: a value that at least k lanes' maxima reach (or the lowest one), by
    // halving the range of those maxima
    const float lowest = -3.4028234e38f;
    float t = lowest;
    if (EPL > 1) {
        float top = ninf;
#pragma unroll
        for (int i = 0; i < EPL; i++) top = fmaxf(top, a[i]);
        float hi = wave_max(top), lo = -wave_max(top == ninf ? ninf : -top);
        if (__builtin_popcountll(__builtin_amdgcn_ballot_w64(top != ninf)) >= p.k) {
            t = lo;
#pragma unroll 1
            for (int i = 0; i < 12; i++) {
                const float mid = 0.5f * lo + 0.5f * hi;
                const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(top >= mid));
                if (n >= p.k) lo = t = mid;
                else hi = mid;
                if (n == p.k) break;
            }
            t = fminf(t, high);
            if (t < INFINITY) t -= 2.0f * margin(by_logit, t);
            t = t < low ? lowest : fmaxf(t, lowest);
        }
    }
    // the lane's candidates as a set of its slots (the first slot the highest
    // bit), then one of each lane's at a time into the list
    uint32_t set = 0;
#pragma unroll
    for (int i = 0; i < EPL; i++) set = set + set + (a[i] >= t ? 1u : 0u);
    int n = 0;
#pragma unroll 1
    for (uint64_t mask; (mask = __builtin_amdgcn_ballot_w64(set != 0)) != 0;) {
        const int top = 31 - __builtin_clz(set | 1u), at = n + below(mask);
        if (set && at < 64) w.id[at] = lane + 64 * (EPL - 1 - top);
        set &= ~(1u << top);
        n += __builtin_popcountll(mask);
    }
    if (slow || n > 64) return whole<SOFT, L>(p, row, biases, lds.v, m, sum);
    // (one wave: its LDS accesses are performed in issue order)
    __builtin_amdgcn_wave_barrier();
    // candidate `lane`, its score and selection value
    const bool there = lane < n;
    const int id = there ? w.id[lane] : 0;
    const double s = score_of<SOFT>(logit_f32<L>(row[id]), m, sum);
    double c = s + (double)biases[id];
    c = there ? (c != c ? (double)INFINITY : c) : -(double)INFINITY;
    w.c[lane] = c;
    __builtin_amdgcn_wave_barrier();
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; j++) rank += w.c[j] > c ? 1 : 0;
    // (distinct values have the ranks 0 .. n - 1, equal ones share the least of theirs)
    if (wave_sum(there ? (float)rank : 0.0f) != (float)(n * (n - 1) / 2)) {
#pragma unroll 1
        for (int j = 0; j < n; j++) rank += w.c[j] == c && w.id[j] < id ? 1 : 0;
    }
    if (there) {  // (distinct ranks 0 .. n - 1)
        w.s[rank] = s;
        w.by[rank] = id;
    }
    __builtin_amdgcn_wave_barrier();
    Pick out = {-1, 0.0};
    if (lane < min(n, p.k)) out = {w.by[lane], w.s[lane]};
    __builtin_amdgcn_wave_barrier();
    return out;
}

// Tokens of a block's waves in turn.  ALONE: the one block counts the choices
// in LDS and writes the counts; else it clears them for k_gate_count.
template <int EPL, bool SOFT, bool BY_LOGIT, typename L, bool ALONE>
__global__ __launch_bounds__(kGateWaves * 64) __attribute__((amdgpu_waves_per_eu(4))) void k_gate(GateParams p)
{
    __shared__ GateLds<EPL> lds[kGateWaves];
    __shared__ int hist[ALONE ? 64 * EPL : 1];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // (tokens in scalars)
    if (ALONE) {
        for (int e = threadIdx.x; e < p.E; e += kGateWaves * 64) hist[e] = 0;
        __syncthreads();
    } else if (p.counts && blockIdx.x == 0) {
        for (int e = threadIdx.x; e < p.E; e += kGateWaves * 64) p.counts[e] = 0;
    }
    __shared__ float bias[64 * EPL];  // (-inf past the end)
    for (int e = threadIdx.x; e < 64 * EPL; e += kGateWaves * 64) bias[e] = e < p.E ? (p.bias ? p.bias[e] : 0.0f) : -INFINITY;
    __syncthreads();
    const L *logits = reinterpret_cast<const L *>(p.logits);
    float l[EPL];
    int t = blockIdx.x * kGateWaves + wv;
    load_row<EPL, L>(logits + (size_t)min(t, p.T - 1) * p.ld, p.E, l);
    for (; t < p.T; t += gridDim.x * kGateWaves) {
        const L *row = logits + (size_t)t * p.ld;
        const L *next = logits + (size_t)min(t + (int)gridDim.x * kGateWaves, p.T - 1) * p.ld;
        const Pick c = choose<EPL, SOFT, BY_LOGIT, L>(p, row, next, l, bias, lds[wv]);
        double w = c.s;
        if (p.renorm) {
            const double total = wave_sum64(lane < p.k ? c.s : 0.0);
            w = total != 0.0 ? w / total : w;
        }
        if (c.id < 0) w = 0.0;  // (a place left: also where the sum is NaN)
        if (lane < p.k) {
            p.ids[(size_t)t * p.k + lane] = c.id;
            p.weights[(size_t)t * p.k + lane] = (float)(w * (double)p.scale);
            if (ALONE && c.id >= 0) atomicAdd(&hist[c.id], 1);
        }
    }
    if (ALONE) {
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += kGateWaves * 64) p.counts[e] = hist[e];
    }
}

// the choices counted: a part of them per block in LDS, then one addition per
// block and expert (one block alone writes its counts)
__global__ __launch_bounds__(1024) void k_gate_count(GateParams p)
{
    __shared__ int hist[kMaxExperts];
    for (int e = threadIdx.x; e < p.E; e += 1024) hist[e] = 0;
    __syncthreads();
    const int64_t n = (int64_t)p.T * p.k, step = (int64_t)gridDim.x * 1024;
    for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < n; i += 4 * step) {
        int id[4];
#pragma unroll
        for (int j = 0; j < 4; j++) id[j] = i + j * step < n ? p.ids[i + j * step] : -1;
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (id[j] >= 0) atomicAdd(&hist[id[j]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += 1024) {
        if (gridDim.x == 1) p.counts[e] = hist[e];
        else if (hist[e]) atomicAdd(p.counts + e, hist[e]);
    }
}

// blocks at most, two per CU; more tokens take turns, a row's logits loaded
// while the one before is chosen from (16384x896: 24.4 us, with 1024 blocks
// 25.6, with 2048 28.2)
constexpr int kGateBlocks = 512;
constexpr int kCountPart = 4096;   // choices that a counting block takes

template <int EPL, bool SOFT, bool BY_LOGIT, typename L>
void launch_epl(const GateParams &p, hipStream_t st)
{
    // (a token to each wave of one block: the counts in the same launch)
    if (p.T <= kGateWaves && p.counts) {
        k_gate<EPL, SOFT, BY_LOGIT, L, true><<<1, kGateWaves * 64, 0, st>>>(p);
        return;
    }
    const int blocks = (p.T + kGateWaves - 1) / kGateWaves;
    k_gate<EPL, SOFT, BY_LOGIT, L, false><<<blocks < kGateBlocks ? blocks : kGateBlocks, kGateWaves * 64, 0, st>>>(p);
    if (p.counts) {
        const int64_t parts = ((int64_t)p.T * p.k + kCountPart - 1) / kCountPart;
        k_gate_count<<<(int)(parts < 64 ? parts : 64), 1024, 0, st>>>(p);
    }
}

template <bool SOFT, bool BY_LOGIT, typename L>
void launch_score(const GateParams &p, hipStream_t st)
{
    const int epl = (p.E + 63) / 64;
    if (epl <= 1) launch_epl<1, SOFT, BY_LOGIT, L>(p, st);
    else if (epl <= 2) launch_epl<2, SOFT, BY_LOGIT, L>(p, st);
    else if (epl <= 4) launch_epl<4, SOFT, BY_LOGIT, L>(p, st);
    else if (epl <= 8) launch_epl<8, SOFT, BY_LOGIT, L>(p, st);
    else if (epl <= 14) launch_epl<14, SOFT, BY_LOGIT, L>(p, st);
    else launch_epl<16, SOFT, BY_LOGIT, L>(p, st);
}

template <typename L>
void launch_typed(const GateParams &p, hipStream_t st)
{
    const bool by_logit = !p.bias && !(p.groups > 1 && p.top2);
    if (p.softmax && by_logit) launch_score<true, true, L>(p, st);
    else if (p.softmax) launch_score<true, false, L>(p, st);
    else if (by_logit) launch_score<false, true, L>(p, st);
    else launch_score<false, false, L>(p, st);
}

}  // namespace

hipError_t launch_gate(const GateParams &p, int logits_type, hipStream_t st)
{
    if (logits_type == 2) launch_typed<float>(p, st);
    else if (logits_type == 1) launch_typed<_Float16>(p, st);
    else launch_typed<uint16_t>(p, st);
    return hipGetLastError();
}

}  // namespace moe
