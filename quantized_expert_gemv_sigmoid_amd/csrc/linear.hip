// Dense product with its epilogue (moe_linear):
//   out[t][n] = act(sum_k x[t][k] w[n][k] + bias[n]) + residual[t][n],
// or act of two such sums (w and w_up) for the gated activations.
//
// Every kernel multiplies D[n][t] = w x^T on the matrix cores with fp32 sums:
// the weights are the A operand, so a lane ends with four consecutive n of
// one token.
#include <math.h>

#include "../../include/moe.h"
#include "common.h"

namespace moe {

namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16_t mfma32(bf16x8_t a, bf16x8_t b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mfma32(f16x8_t a, f16x8_t b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// ---------------------------------------------------------------- epilogue

template <bool F16>
__device__ __forceinline__ float half_f32(uint16_t v)
{
    return F16 ? (float)__builtin_bit_cast(_Float16, v) : __uint_as_float((uint32_t)v << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t f32_half(float v)
{
    return F16 ? __builtin_bit_cast(uint16_t, (_Float16)v) : f32_to_bf16_rne(v);
}

// the activations; 1 / b of the SiTU betas is shared by the calls of a kernel
__device__ __forceinline__ float activate(float a, float u, int act, float b1, float b2)
{
    switch (act) {
    case MOE_LINEAR_RELU: return a > 0.0f ? a : (a != a ? a : 0.0f);
    case MOE_LINEAR_SILU: return a * sigmoid_hw(a);
    case MOE_LINEAR_GELU: return 0.5f * a * erfcf(a * -0.707106781186547524f);
    case MOE_LINEAR_GELU_TANH: return a * sigmoid_hw(1.5957691216057308f * (a + 0.044715f * a * a * a));
    case MOE_LINEAR_SITU_GLU: return gated_act(a, u, 0, b1, b2);
    case MOE_LINEAR_SWIGLU: return gated_act(a, u, 1, b1, b2);
    default: return a;
    }
}

template <bool F16>
__device__ __forceinline__ float bias_at(const void *b, int f32, int n)
{
    if (!b) return 0.0f;
    return f32 ? reinterpret_cast<const float *>(b)[n] : half_f32<F16>(reinterpret_cast<const uint16_t *>(b)[n]);
}

// one output from its sums
template <bool F16>
__device__ __forceinline__ void finish(const LinearParams &p, int t, int n, float a, float u)
{
    a += bias_at<F16>(p.bias, p.bias_f32, n);
    u += bias_at<F16>(p.bias_up, p.bias_f32, n);
    float v = activate(a, u, p.act, p.b1, p.b2);
    if (p.res) {
        const size_t at = (size_t)t * p.ldr + n;
        v += p.res_f32 ? reinterpret_cast<const float *>(p.res)[at]
                       : half_f32<F16>(reinterpret_cast<const uint16_t *>(p.res)[at]);
    }
    const size_t at = (size_t)t * p.ldo + n;
    if (p.out_half) reinterpret_cast<uint16_t *>(p.out_half)[at] = f32_half<F16>(v);
    if (p.out_f32) p.out_f32[at] = v;
}

// ------------------------------------------------- any alignment, any size

// 8 consecutive values of a row, zeros from k = K on
__device__ __forceinline__ uint4 load8(const uint16_t *row, int k, int K)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k + 8 <= K) {
        __builtin_memcpy(&v, row + k, 16);
    } else {
        uint16_t h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (k + i < K) h[i] = row[k + i];
        __builtin_memcpy(&v, h, 16);
    }
    return v;
}

constexpr int kAnyTile = 64, kAnyK = 32, kAnyRow = kAnyK * 2 + 16;  // (16: rows on different banks)

// 64 n x 64 tokens per block of four waves, each 32 x 32
template <bool F16, bool GATED>
__global__ __launch_bounds__(256) void k_linear_any(LinearParams p)
{
    using V = typename std::conditional<F16, f16x8_t, bf16x8_t>::type;
    __shared__ __align__(16) uint8_t sw[(GATED ? 2 : 1) * kAnyTile * kAnyRow], sx[kAnyTile * kAnyRow];
    const int n0 = blockIdx.x * kAnyTile, t0 = blockIdx.y * kAnyTile;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int r = threadIdx.x / 4, q = threadIdx.x % 4;  // the row and 16-byte piece this thread stages
    const bool nok = n0 + r < p.N, tok = t0 + r < p.M;
    const uint16_t *wr = reinterpret_cast<const uint16_t *>(p.w) + (nok ? (size_t)(n0 + r) * p.ldw : 0);
    const uint16_t *ur = reinterpret_cast<const uint16_t *>(p.w_up) + (nok ? (size_t)(n0 + r) * p.ldw : 0);
    const uint16_t *xr = reinterpret_cast<const uint16_t *>(p.x) + (tok ? (size_t)(t0 + r) * p.ldx : 0);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int nw = (wv & 1) * 32, tw = (wv >> 1) * 32;
    f32x16_t acc = {}, acu = {};
    for (int k0 = 0; k0 < p.K; k0 += kAnyK) {
        const int k = k0 + 8 * q;
        const uint4 a = nok ? load8(wr, k, p.K) : zero, x = tok ? load8(xr, k, p.K) : zero;
        const uint4 u = GATED && nok ? load8(ur, k, p.K) : zero;
        __syncthreads();
        *reinterpret_cast<uint4 *>(sw + r * kAnyRow + q * 16) = a;
        if (GATED) *reinterpret_cast<uint4 *>(sw + (kAnyTile + r) * kAnyRow + q * 16) = u;
        *reinterpret_cast<uint4 *>(sx + r * kAnyRow + q * 16) = x;
        __syncthreads();
#pragma unroll
        for (int st = 0; st < kAnyK / 16; st++) {
            const int at = (lane & 31) * kAnyRow + (2 * st + (lane >> 5)) * 16;
            const V b = *reinterpret_cast<const V *>(sx + tw * kAnyRow + at);
            acc = mfma32(*reinterpret_cast<const V *>(sw + nw * kAnyRow + at), b, acc);
            if (GATED) acu = mfma32(*reinterpret_cast<const V *>(sw + (kAnyTile + nw) * kAnyRow + at), b, acu);
        }
    }
    const int t = t0 + tw + (lane & 31);
    if (t >= p.M) return;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int n = n0 + nw + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
        if (n < p.N) finish<F16>(p, t, n, acc[i], GATED ? acu[i] : 0.0f);
    }
}

template <bool F16>
void launch_any(const LinearParams &p, hipStream_t st)
{
    const dim3 grid((p.N + kAnyTile - 1) / kAnyTile, (p.M + kAnyTile - 1) / kAnyTile);
    if (p.w_up) k_linear_any<F16, true><<<grid, 256, 0, st>>>(p);
    else k_linear_any<F16, false><<<grid, 256, 0, st>>>(p);
}

}  // namespace

size_t linear_workspace(const LinearParams &) { return 256; }

hipError_t launch_linear(const LinearParams &p, bool f16, hipStream_t st)
{
    if (f16) launch_any<true>(p, st);
    else launch_any<false>(p, st);
    return hipGetLastError();
}

}  // namespace moe
