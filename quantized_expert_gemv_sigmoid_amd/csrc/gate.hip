// Routing from given logits: softmax or sigmoid scores, selection bias,
// groups, top-k, renormalised weights (moe_gate).
//
// One wave per token: lane l holds experts l, l + 64, ...  Scores and
// selection values are doubles, so that experts whose fp32 values would round
// together keep their order; a value of -inf marks an expert that takes no
// part, and a NaN one ranks as +inf.  The k picks are k rounds of a wave-wide
// maximum.
#include <math.h>

#include "common.h"

namespace moe {

namespace {

template <typename L>
__device__ __forceinline__ float logit_f32(L v);
template <>
__device__ __forceinline__ float logit_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float logit_f32<_Float16>(_Float16 v) { return (float)v; }
template <>
__device__ __forceinline__ float logit_f32<uint16_t>(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__device__ __forceinline__ double wave_max(double v)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = fmax(v, __shfl_xor(v, m, 64));
    return v;
}
__device__ __forceinline__ double wave_sum64(double v)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}
__device__ __forceinline__ int wave_min(int v)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = min(v, __shfl_xor(v, m, 64));
    return v;
}

template <int EPL, typename L>
__global__ __launch_bounds__(256) void k_gate(GateParams p)
{
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= p.T) return;
    const L *row = reinterpret_cast<const L *>(p.logits) + (size_t)t * p.ld;
    const double ninf = -INFINITY;
    double s[EPL], c[EPL];
    bool on[EPL];
    float l[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = lane + 64 * i, ec = min(e, p.E - 1);
        l[i] = logit_f32<L>(row[ec]);
        const float b = p.bias ? p.bias[ec] : 0.0f;
        on[i] = e < p.E && l[i] != -INFINITY && b != -INFINITY;
        c[i] = b;
    }
    if (p.softmax) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; i++) m = on[i] ? fmaxf(m, l[i]) : m;
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            // (+inf - +inf: the limit, 0)
            s[i] = on[i] ? exp(l[i] == m ? 0.0 : (double)l[i] - (double)m) : 0.0;
            sum += s[i];
        }
        sum = wave_sum64(sum);
#pragma unroll
        for (int i = 0; i < EPL; i++) s[i] = s[i] / sum;
    } else {
#pragma unroll
        for (int i = 0; i < EPL; i++) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    }
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const double v = s[i] + c[i];
        c[i] = on[i] ? (v != v ? (double)INFINITY : v) : ninf;
    }
    if (p.groups > 1) {
        double mine = ninf;  // lane g: the value of group g
        for (int g = 0; g < p.groups; g++) {
            double a = ninf, b = ninf;  // the lane's two largest
#pragma unroll
            for (int i = 0; i < EPL; i++) {
                const double v = ((lane + 64 * i) * p.group_inv) >> 20 == g ? c[i] : ninf;
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
            const double top = wave_max(a);
            double value = top;
            if (p.top2) {
                // the second: the others' largest, and the second of the one
                // lane that gave the first
                const uint64_t who = __builtin_amdgcn_ballot_w64(a == top);
                const bool first = lane == (int)__builtin_ctzll(who);
                const double second = wave_max(first ? b : a);
                value = top + (second == ninf ? 0.0 : second);
            }
            mine = lane == g ? value : mine;
        }
        int rank = 0;
        for (int g = 0; g < p.groups; g++) {
            const double o = __shfl(mine, g, 64);
            rank += o > mine || (o == mine && g < lane) ? 1 : 0;
        }
        const uint64_t kept = __builtin_amdgcn_ballot_w64(lane < p.groups && rank < p.top_groups);
#pragma unroll
        for (int i = 0; i < EPL; i++)
            c[i] = (kept >> (((lane + 64 * i) * p.group_inv) >> 20)) & 1 ? c[i] : ninf;
    }
    int my_id = -1;
    double my_s = 0.0, total = 0.0;
    for (int j = 0; j < p.k; j++) {
        double best = ninf, bs = 0.0;
        int bi = 0;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const bool more = c[i] > best;  // (strict: the lower id of a tie)
            best = more ? c[i] : best;
            bs = more ? s[i] : bs;
            bi = more ? i : bi;
        }
        const double top = wave_max(best);
        if (top == ninf) break;
        const int id = wave_min(best == top ? lane + 64 * bi : 1 << 30);
        const double sv = __shfl(bs, id & 63, 64);
        total += sv;
        my_id = lane == j ? id : my_id;
        my_s = lane == j ? sv : my_s;
#pragma unroll
        for (int i = 0; i < EPL; i++) c[i] = lane + 64 * i == id ? ninf : c[i];
    }
    if (lane < p.k) {
        double w = my_s;
        if (p.renorm && total != 0.0) w = w / total;
        p.ids[(size_t)t * p.k + lane] = my_id;
        p.weights[(size_t)t * p.k + lane] = (float)(w * (double)p.scale);
        if (p.counts && my_id >= 0) atomicAdd(p.counts + my_id, 1);
    }
}

__global__ __launch_bounds__(256) void k_gate_zero(int E, int32_t *counts)
{
    const int e = blockIdx.x * 256 + threadIdx.x;
    if (e < E) counts[e] = 0;
}

template <typename L>
void launch_typed(const GateParams &p, hipStream_t st)
{
    const int epl = (p.E + 63) / 64, grid = (p.T + 3) / 4;
    if (epl <= 1) k_gate<1, L><<<grid, 256, 0, st>>>(p);
    else if (epl <= 2) k_gate<2, L><<<grid, 256, 0, st>>>(p);
    else if (epl <= 4) k_gate<4, L><<<grid, 256, 0, st>>>(p);
    else if (epl <= 8) k_gate<8, L><<<grid, 256, 0, st>>>(p);
    else k_gate<16, L><<<grid, 256, 0, st>>>(p);
}

}  // namespace

hipError_t launch_gate(const GateParams &p, int logits_type, hipStream_t st)
{
    if (p.counts) k_gate_zero<<<(p.E + 255) / 256, 256, 0, st>>>(p.E, p.counts);
    if (logits_type == 2) launch_typed<float>(p, st);
    else if (logits_type == 1) launch_typed<_Float16>(p, st);
    else launch_typed<uint16_t>(p, st);
    return hipGetLastError();
}

}  // namespace moe
