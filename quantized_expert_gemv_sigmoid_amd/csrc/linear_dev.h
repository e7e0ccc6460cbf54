// Dense product with its epilogue (moe_linear):
//   out[t][n] = act(sum_k x[t][k] w[n][k] + bias[n]) + residual[t][n],
// or act of two such sums (w and w_up) for the gated activations.
//
// Every kernel multiplies D[n][t] = w x^T on the matrix cores with fp32 sums:
// the weights are the A operand, so a lane ends with four consecutive n of
// one token.  K comes in stages of 64 into LDS rows of 128 bytes, their
// 16-byte pieces permuted (piece ^ row / 2) so that fragment reads touch every
// bank alike.  Four kernels, by what bounds them (which call takes which:
// linear.hip):
//   k_linear_big   the matrix cores: 256 x 256 tiles
//   k_linear_tile  LDS reads and latency: 64 x 32 to 128 x 128 tiles
//   k_linear_few   the weights' way from memory, each row read once: 16 rows
//                  x 8 to 32 tokens
//   k_linear_join  sums of a K split over blocks
#pragma once

#include <math.h>
#include <type_traits>

#include "../../include/moe.h"
#include "common.h"

namespace moe {

namespace {

// c += a b, 16 x 16 x 32, c in accumulation registers for good: written out,
// since the compiler moves such small accumulators between registers around
// a loop that holds 64 of them
__device__ __forceinline__ void mfma16(bf16x8_t a, bf16x8_t b, f32x4_t &c)
{
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void mfma16(f16x8_t a, f16x8_t b, f32x4_t &c)
{
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
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

// tanh(x) = n / d for x >= 0, e = exp(-2 x): (1 - e) / (1 + e), and below
// 1/16, where 1 - e cancels, the odd Taylor polynomial to x^7 (the next term
// is below 3e-13 of it)
__device__ __forceinline__ void tanh_parts(float x, float e, float &n, float &d)
{
    const float x2 = x * x;
    const float small = x * (1.0f + x2 * (-1.0f / 3.0f + x2 * (2.0f / 15.0f + x2 * (-17.0f / 315.0f))));
    n = x < 0.0625f ? small : 1.0f - e;
    d = x < 0.0625f ? 1.0f : 1.0f + e;
}

// SiTU-GLU b1 tanh(g / b1) sigmoid(g) b2 tanh(u / b2) with one reciprocal for
// the three quotients (r1 = 1 / b1, r2 = 1 / b2; each beta goes to its own
// tanh, since b1 b2 may be past fp32's range)
__device__ __forceinline__ float situ_glu(float g, float u, float b1, float b2, float r1, float r2)
{
    const float x = fabsf(g) * r1, y = fabsf(u) * r2;
    float n1, d1, n2, d2;
    tanh_parts(x, exp_hw(-2.0f * x), n1, d1);
    tanh_parts(y, exp_hw(-2.0f * y), n2, d2);
    const float h = (b1 * n1) * (b2 * n2) * rcp_hw(d1 * d2 * (1.0f + exp_hw(-g)));
    return __uint_as_float(__float_as_uint(h) ^ ((__float_as_uint(g) ^ __float_as_uint(u)) & 0x80000000u));
}

// a[i] = act(a[i], u[i]): one branch for all NV values
template <bool GATED, int NV>
__device__ __forceinline__ void activate(float (&a)[NV], const float (&u)[NV], int act, float b1, float b2)
{
    if (GATED) {
        if (act == MOE_LINEAR_SITU_GLU) {
#pragma unroll
            for (int i = 0; i < NV; i++) a[i] = situ_glu(a[i], u[i], b1, b2, 1.0f / b1, 1.0f / b2);
        } else {
#pragma unroll
            for (int i = 0; i < NV; i++) a[i] = gated_act(a[i], u[i], 1, b1, b2);
        }
        return;
    }
    switch (act) {
    case MOE_LINEAR_RELU:
#pragma unroll
        for (int i = 0; i < NV; i++) a[i] = a[i] < 0.0f ? 0.0f : a[i];
        break;
    case MOE_LINEAR_SILU:
#pragma unroll
        for (int i = 0; i < NV; i++) a[i] *= sigmoid_hw(a[i]);
        break;
    case MOE_LINEAR_GELU:
#pragma unroll
        for (int i = 0; i < NV; i++) a[i] = 0.5f * a[i] * erfcf(a[i] * -0.707106781186547524f);
        break;
    case MOE_LINEAR_GELU_TANH:  // (1 + tanh z) / 2 = sigmoid(2 z)
#pragma unroll
        for (int i = 0; i < NV; i++)
            a[i] *= sigmoid_hw(1.5957691216057308f * (a[i] + 0.044715f * a[i] * a[i] * a[i]));
        break;
    default: break;
    }
}

template <bool F16>
__device__ __forceinline__ float bias_at(const void *b, int f32, int n)
{
    if (!b) return 0.0f;
    return f32 ? reinterpret_cast<const float *>(b)[n] : half_f32<F16>(reinterpret_cast<const uint16_t *>(b)[n]);
}

// four values in the 16-bit type, round to nearest even
template <bool F16>
__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d)
{
    if (F16) {
        const f16x2v_t x = {(_Float16)a, (_Float16)b}, y = {(_Float16)c, (_Float16)d};
        return make_uint2(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y));
    }
    const bf16x2v_t x = {(__bf16)a, (__bf16)b}, y = {(__bf16)c, (__bf16)d};
    return make_uint2(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y));
}

// The residual's four values at n .. n + 3 of R tokens t[i] (none where
// t[i] < 0), as they are in memory; where all four exist.  (Rows may start
// anywhere: a wide access needs no alignment here, and an aligned one costs
// the same.  2048x1117x2049: stores one by one 44.8 us, by four 38.2.)
template <int R>
__device__ __forceinline__ void load_res(const LinearParams &p, const int (&t)[R], int n, uint4 (&r)[R])
{
    if (!p.res || n + 4 > p.N) return;
    if (p.res_f32) {
#pragma unroll
        for (int i = 0; i < R; i++)
            if (t[i] >= 0)
                __builtin_memcpy(&r[i], reinterpret_cast<const float *>(p.res) + (size_t)t[i] * p.ldr + n, 16);
    } else {
#pragma unroll
        for (int i = 0; i < R; i++)
            if (t[i] >= 0)
                __builtin_memcpy(&r[i], reinterpret_cast<const uint16_t *>(p.res) + (size_t)t[i] * p.ldr + n, 8);
    }
}

// R rows of four outputs each, n .. n + 3 of tokens t[i], from their
// activated sums a and load_res's values; rows with t[i] < 0 are not there.
template <bool F16, int R>
__device__ __forceinline__ void write_rows(const LinearParams &p, const int (&t)[R], int n, float (&a)[4 * R], const uint4 (&r)[R])
{
    uint16_t *oh = reinterpret_cast<uint16_t *>(p.out_half);
    if (n + 4 <= p.N) {
        if (p.res && p.res_f32) {
#pragma unroll
            for (int i = 0; i < R; i++) {
                a[4 * i] += __uint_as_float(r[i].x);
                a[4 * i + 1] += __uint_as_float(r[i].y);
                a[4 * i + 2] += __uint_as_float(r[i].z);
                a[4 * i + 3] += __uint_as_float(r[i].w);
            }
        } else if (p.res) {
#pragma unroll
            for (int i = 0; i < R; i++) {
                a[4 * i] += half_f32<F16>((uint16_t)r[i].x);
                a[4 * i + 1] += half_f32<F16>((uint16_t)(r[i].x >> 16));
                a[4 * i + 2] += half_f32<F16>((uint16_t)r[i].y);
                a[4 * i + 3] += half_f32<F16>((uint16_t)(r[i].y >> 16));
            }
        }
        if (oh) {
#pragma unroll
            for (int i = 0; i < R; i++)
                if (t[i] >= 0) {
                    const uint2 v = pack4<F16>(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
                    __builtin_memcpy(oh + (size_t)t[i] * p.ldo + n, &v, 8);
                }
        }
        if (p.out_f32) {
#pragma unroll
            for (int i = 0; i < R; i++)
                if (t[i] >= 0) __builtin_memcpy(p.out_f32 + (size_t)t[i] * p.ldo + n, &a[4 * i], 16);
        }
        return;
    }
    const float *rf = reinterpret_cast<const float *>(p.res);
    const uint16_t *rh = reinterpret_cast<const uint16_t *>(p.res);
#pragma unroll
    for (int i = 0; i < R; i++) {
        if (t[i] < 0) continue;
        const size_t ra = (size_t)t[i] * p.ldr + n, at = (size_t)t[i] * p.ldo + n;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (n + j >= p.N) continue;
            float v = a[4 * i + j];
            if (p.res) v += p.res_f32 ? rf[ra + j] : half_f32<F16>(rh[ra + j]);
            if (oh) oh[at + j] = f32_half<F16>(v);
            if (p.out_f32) p.out_f32[at + j] = v;
        }
    }
}

// one row of sums (biases included), its residual loaded here
template <bool F16, bool GATED>
__device__ __forceinline__ void finish_row(const LinearParams &p, int t, int n, float (&a)[4], const float (&u)[4])
{
    const int tt[1] = {t};
    uint4 r[1] = {};
    load_res<1>(p, tt, n, r);
    activate<GATED>(a, u, p.act, p.b1, p.b2);
    write_rows<F16, 1>(p, tt, n, a, r);
}

// the biases of outputs n .. n + 3
template <bool F16>
__device__ __forceinline__ void bias4(const void *b, int f32, int n, int N, float (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = n + i < N ? bias_at<F16>(b, f32, n + i) : 0.0f;
}

// Partial sums of K part ks: rows of a multiple of four values, the parts one
// after the other, gated ones as the sums of w and then of w_up.
__device__ __forceinline__ size_t part_pitch(const LinearParams &p) { return (size_t)((p.N + 3) & ~3); }
template <bool GATED>
__device__ __forceinline__ void store_part(const LinearParams &p, int ks, int t, int n, f32x4_t a, f32x4_t u)
{
    const size_t plane = (size_t)p.M * part_pitch(p);
    float *o = p.part + (size_t)ks * (GATED ? 2 : 1) * plane + (size_t)t * part_pitch(p) + n;
    *reinterpret_cast<f32x4_t *>(o) = a;
    if (GATED) *reinterpret_cast<f32x4_t *>(o + plane) = u;
}

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

// -------------------------------------------------- whole prompts: 256 x 256

// wait until at most N of the wave's copies and L of its LDS reads are in flight
template <int N, int L = 0>
__device__ __forceinline__ void wait_copies()
{
    static_assert(N >= 0 && N < 64 && L >= 0 && L < 16, "vmcnt, lgkmcnt fields");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (L << 8));
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

template <bool F16>
struct Frag {
    using V = typename std::conditional<F16, f16x8_t, bf16x8_t>::type;
};

// Output tile number of a block: the blocks of one XCD (block % 8) take a run
// of tiles, four token tiles by eight weight tiles at a time, so that the 32
// blocks its CUs hold share their rows in its L2.
__device__ __forceinline__ void tile_of(int block, int tn, int tt, int &n, int &t)
{
    const int total = tn * tt, q = total >> 3, r = total & 7, x = block & 7;
    const int l = x * q + min(x, r) + (block >> 3);
    const int g = l / (4 * tn), in = l - g * 4 * tn, h = min(4, tt - 4 * g);
    t = 4 * g + in % h;
    n = in / h;
}

// rows [0, rows) of a matrix from `base`, as far as its last row's K values
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const uint16_t *base, int rows, int64_t ld, int K)
{
    const uint32_t bytes = rows > 0 ? (uint32_t)(((int64_t)(rows - 1) * ld + K) * 2) : 0u;
    return grsrc(base, bytes);
}

// 16 bytes per lane at voff of r to LDS at dst + 16 lane (dst wave-uniform).
// The caller orders the copies with waits and barriers.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t r, uint32_t dst, uint32_t voff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(voff), "s"(r)
                 : "memory", "m0");
}

constexpr int kUnit = 128 * 128;            // bytes of 128 rows x 64 k
constexpr int kBigRing = 8 * kUnit;         // two stages of A0 A1 B0 B1
constexpr int kBigRow = 64 * 4 + 16;        // a row of the epilogue's buffer
constexpr int kBigWave = 128 * kBigRow;  // a wave's part of it
constexpr int kBigLds = 4 * kBigWave > kBigRing ? 4 * kBigWave : kBigRing;

// 256 x 256 outputs (gated: 128 of each matrix) per block and CU, four waves
// of 128 x 128, one to a SIMD, whose 256 sums per lane fill the accumulation
// registers: 64 products of 16 x 16 x 32 per 32 fragment reads of 16 bytes,
// so LDS supplies half of what it could, and the matrix cores are the bound.
// 16 x 16 x 32 and not 32 x 32 x 16: on registers alone the whole chip does
// 2050 TFLOP/s with the former and 1660-1850 with the latter, which draws
// more power (4096 x 7168 x 7168: 372 us with the latter, 325 with the former).
// Measured: 4096 x 7168 x 7168 296-309 us by the box (1422-1360 TFLOP/s, the
// library's product 285-293), with bias and a 16-bit residual 315-318; 4096 x
// 3584 x 2 x 6144 SwiGLU 251-262 (library 245), SiTU-GLU 273-286.  Matrix
// cores busy for 76% of the kernel; 8192^3 reaches 1491 TFLOP/s, where clocks
// give way to power.  The rest is the last
// turn of tiles (448 on 256 CUs) and the epilogue, which nothing overlaps as
// a CU holds one block.
template <bool F16, bool GATED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_linear_big(LinearParams p, int tn,
                                                                                               int tt, int ksplit)
{
    using V = typename Frag<F16>::V;
    __shared__ __align__(1024) uint8_t lds_blk[kBigLds];
    LDS uint8_t *lds = (LDS uint8_t *)lds_blk;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ti, ni;
    tile_of(blockIdx.x % (tn * tt), tn, tt, ni, ti);
    const int t0 = ti * 256, n0 = ni * (GATED ? 128 : 256);
    // the block's part of K
    const int ks = blockIdx.x / (tn * tt), SA = (p.K + 63) / 64;
    const int kb = (int)((int64_t)SA * ks / ksplit) * 64, K = min(p.K, (int)((int64_t)SA * (ks + 1) / ksplit) * 64) - kb;
    const uint16_t *W = reinterpret_cast<const uint16_t *>(p.w) + kb, *U = reinterpret_cast<const uint16_t *>(p.w_up) + kb;
    const uint16_t *X = reinterpret_cast<const uint16_t *>(p.x) + kb + (size_t)t0 * p.ldx;
    const int na1 = n0 + 128;
    const __amdgpu_buffer_rsrc_t rA0 = rows_rsrc(W + (size_t)n0 * p.ldw, min(128, p.N - n0), p.ldw, K);
    const __amdgpu_buffer_rsrc_t rA1 =
        GATED ? rows_rsrc(U + (size_t)n0 * p.ldw, min(128, p.N - n0), p.ldw, K)
              : rows_rsrc(na1 < p.N ? W + (size_t)na1 * p.ldw : W, min(128, p.N - na1), p.ldw, K);
    const __amdgpu_buffer_rsrc_t rB0 = rows_rsrc(X, min(128, p.M - t0), p.ldx, K);
    const __amdgpu_buffer_rsrc_t rB1 =
        rows_rsrc(t0 + 128 < p.M ? X + (size_t)128 * p.ldx : X, min(128, p.M - t0 - 128), p.ldx, K);

    // copies: the wave's 32 rows of a unit in four pieces of 8, this lane's 16 bytes of each
    const int l8 = lane >> 3, piece = (lane & 7) ^ (l8 >> 1);
    uint32_t va[4], vb[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t row = 32 * wv + 8 * j + l8, col = (piece ^ (j & 1 ? 4 : 0)) * 16;
        va[j] = (uint32_t)(row * p.ldw * 2) + col;
        vb[j] = (uint32_t)(row * p.ldx * 2) + col;
    }
    int kc0 = piece * 8, kc1 = (piece ^ 4) * 8;
    const uint32_t m0w = (uint32_t)(uintptr_t)lds + wv * 4096;
    // unit positions in a stage's buffer
    constexpr int A0 = 0, A1 = kUnit, B0 = 2 * kUnit, B1 = 3 * kUnit, BUF = 4 * kUnit;
    // piece j of the wave's part of a unit, D stages on (checked where that stage may end past K)
    auto copy = [&](auto check, auto d, __amdgpu_buffer_rsrc_t r, int at, bool b, int j) {
        constexpr int D = decltype(d)::value;
        uint32_t v = (b ? vb[j] : va[j]) + D * 128;
        if (decltype(check)::value) v = (j & 1 ? kc1 : kc0) + D * 64 < K ? v : 0x80000000u;
        copy16(r, m0w + at + j * 1024, v);
    };

    // fragment reads: lane l holds row l % 16 of a 16-row tile, the k pieces l / 16 and 4 + l / 16 of a stage
    const int r16 = lane & 15, q4 = lane >> 4;
    const int wn = wv >> 1, wt = wv & 1;
    const LDS uint8_t *fa[2], *fb[2];  // in the buffer that is read next
#pragma unroll
    for (int st = 0; st < 2; st++) {
        const int o = r16 * 128 + (((st * 4 + q4) ^ (r16 >> 1)) << 4);
        fa[st] = lds + wn * 64 * 128 + o;
        fb[st] = lds + wt * 64 * 128 + o;
    }
    V a0[2][4], a1[2][4], b0[2][4], b1[2][4];
    auto readA = [&](V(&a)[2][4], int at, int i) { a[i >> 2][i & 3] = __builtin_bit_cast(V, lds_ld16(fa[i >> 2] + at + (i & 3) * 2048)); };
    auto readB = [&](V(&b)[2][4], int at, int i) { b[i >> 2][i & 3] = __builtin_bit_cast(V, lds_ld16(fb[i >> 2] + at + (i & 3) * 2048)); };
    auto turn = [&](const LDS uint8_t *(&q)[2], int d) { q[0] += d; q[1] += d; };
    f32x4_t acc[2][2][4][4] = {};  // [A half][B half][16 n][16 tokens]

    using Yes = std::true_type;
    using No = std::false_type;
    using D0 = std::integral_constant<int, 0>;
    using D1 = std::integral_constant<int, 1>;
    using D2 = std::integral_constant<int, 2>;
    using D3 = std::integral_constant<int, 3>;
    auto unit = [&](auto d, __amdgpu_buffer_rsrc_t r, int at, bool b) {
#pragma unroll
        for (int j = 0; j < 4; j++) copy(Yes{}, d, r, at, b, j);
    };
    unit(D0{}, rA0, A0, false);
    unit(D0{}, rB0, B0, true);
    unit(D0{}, rB1, B1, true);
    unit(D0{}, rA1, A1, false);
    unit(D1{}, rA0, BUF + A0, false);
    unit(D1{}, rB1, BUF + B1, true);
    unit(D1{}, rB0, BUF + B0, true);
    unit(D1{}, rA1, BUF + A1, false);
    wait_copies<24>();
    barrier();
#pragma unroll
    for (int i = 0; i < 8; i++) {
        readA(a0, A0, i);
        readB(b0, B0, i);
    }
    wait_copies<24>();  // (these reads too: the first two phases fill the units anew)

    // A phase multiplies one A half with one B half (64 n x 64 tokens x 64 k
    // per wave: 32 products).  Spread between them go the reads of the half
    // the next phase needs, and the copies, two stages on, of the unit whose
    // last reads were issued two phases before: every unit is filled six
    // phases before it is read.
    auto phase = [&](auto check, auto d, __amdgpu_buffer_rsrc_t r, int at, bool b, f32x4_t(&c)[4][4], const V(&x)[2][4],
                     const V(&y)[2][4], auto read) {
        __builtin_amdgcn_sched_barrier(0);
        wait_copies<20, 8>();
        barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 32; i++) {
            const int st = i >> 4, f = (i >> 2) & 3, g = f & 1 ? 3 - (i & 3) : i & 3;
            mfma16(x[st][f], y[st][g], c[f][g]);
            if (i % 4 == 0) read(i >> 2);
            if (i % 8 == 2) copy(check, d, r, at, b, i >> 3);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto two_stages = [&](auto check) {
        // stage s: B0 first
        phase(check, D2{}, rA0, A0, false, acc[0][0], a0, b0, [&](int i) { readB(b1, B1, i); });
        phase(check, D2{}, rB0, B0, true, acc[0][1], a0, b1, [&](int i) { readA(a1, A1, i); });
        turn(fa, BUF);
        phase(check, D2{}, rB1, B1, true, acc[1][1], a1, b1, [&](int i) { readA(a0, A0, i); });
        turn(fb, BUF);
        phase(check, D2{}, rA1, A1, false, acc[1][0], a1, b0, [&](int i) { readB(b1, B1, i); });
        // stage s + 1: B1 first
        phase(check, D3{}, rA0, BUF + A0, false, acc[0][1], a0, b1, [&](int i) { readB(b0, B0, i); });
        phase(check, D3{}, rB1, BUF + B1, true, acc[0][0], a0, b0, [&](int i) { readA(a1, A1, i); });
        turn(fa, -BUF);
        phase(check, D3{}, rB0, BUF + B0, true, acc[1][0], a1, b0, [&](int i) { readA(a0, A0, i); });
        turn(fb, -BUF);
        phase(check, D3{}, rA1, BUF + A1, false, acc[1][1], a1, b1, [&](int i) { readB(b0, B0, i); });
#pragma unroll
        for (int j = 0; j < 4; j++) va[j] += 256, vb[j] += 256;
        kc0 += 128;
        kc1 += 128;
    };
    // (the copies of stages up to s + 3 stay inside K while 64 (s + 4) <= K)
    const int S = (K + 63) / 64;
    int s = 0;
    for (; 64 * (s + 4) <= K; s += 2) two_stages(No{});
    for (; s < S; s += 2) two_stages(Yes{});
    __builtin_amdgcn_sched_barrier(0);
    // The last products' results: nobody else waits for written-out products,
    // so every sum goes through a statement behind the wait.
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int i = 0; i < 4; i++) {
        f32x4_t(&c)[4][4] = acc[i >> 1][i & 1];
        asm volatile(""
                     : "+a"(c[0][0]), "+a"(c[0][1]), "+a"(c[0][2]), "+a"(c[0][3]), "+a"(c[1][0]), "+a"(c[1][1]), "+a"(c[1][2]),
                       "+a"(c[1][3]), "+a"(c[2][0]), "+a"(c[2][1]), "+a"(c[2][2]), "+a"(c[2][3]), "+a"(c[3][0]), "+a"(c[3][1]),
                       "+a"(c[3][2]), "+a"(c[3][3]));
    }
    wait_copies<0>();
    barrier();

    // epilogue: 64 n x 128 tokens of sums (gated: 64 tokens of both matrices)
    // at a time through the wave's own LDS, so that a row's 64 outputs leave
    // as 16 lanes x 4
    LDS uint8_t *buf = lds + wv * kBigWave;
    const int c4 = (lane & 15) * 4;
    const int row_l = r16 * kBigRow + q4 * 16;
    constexpr int ROWS = GATED ? 64 : 128, R = 4, BATCHES = ROWS / (4 * R);
#pragma unroll 1
    for (int round = 0; round < 2; round++) {
        const int n = n0 + (GATED ? 0 : round * 128) + wn * 64 + c4;
        auto token = [&](int r) {
            const int t = t0 + (GATED ? round * 128 + r : (r >> 6) * 128 + (r & 63)) + wt * 64;
            return t < p.M && n < p.N ? t : -1;
        };
        auto sums = [&](int r) { return reinterpret_cast<LDS f32x4_t *>(buf + r * kBigRow + c4 * 4); };
        // Whole tiles with aligned rows: rows 4 k of the lane's at scalar
        // distances from its first.  Their residual goes to registers at once,
        // before any store: a load waits for the stores before it to reach
        // memory, so batches that load and store in turn took 22 us more per
        // 256 tiles of 16-bit residuals.
        const bool direct = ksplit == 1 && p.vec && t0 + 256 <= p.M && n0 + (GATED ? 128 : 256) <= p.N;
        const int tr = t0 + (GATED ? round * 128 : 0) + wt * 64, nr = n0 + (GATED ? 0 : round * 128) + wn * 64;
        auto rows_of = [&](const void *base, int64_t ld, int sz) {
            return grsrc(reinterpret_cast<const char *>(base) + ((size_t)tr * ld + nr) * sz, 0xfffffffcu);
        };
        auto row_at = [&](int k, int64_t ld, int sz) { return (int)((uint32_t)((4 * k >> 6) * 128 + (4 * k & 63)) * (uint32_t)(ld * sz)); };
        auto lane_at = [&](int64_t ld, int sz) { return (int)(q4 * (uint32_t)(ld * sz) + c4 * sz); };
        const __amdgpu_buffer_rsrc_t rr = rows_of(p.res, p.ldr, p.res_f32 ? 4 : 2), rh = rows_of(p.out_half, p.ldo, 2),
                                     rf = rows_of(p.out_f32, p.ldo, 4);
        const int vr = lane_at(p.ldr, p.res_f32 ? 4 : 2), vh = lane_at(p.ldo, 2), vf = lane_at(p.ldo, 4);
        uint2 early[ROWS / 4] = {};
        if (direct && p.res && !p.res_f32) {
#pragma unroll
            for (int k = 0; k < ROWS / 4; k++)
                early[k] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rr, vr, row_at(k, p.ldr, 2), 0));
        }
        auto put = [&](int row, const f32x4_t(&c)[4][4]) {
#pragma unroll
            for (int f = 0; f < 4; f++)
#pragma unroll
                for (int g = 0; g < 4; g++)
                    *reinterpret_cast<LDS f32x4_t *>(buf + row_l + (row + g * 16) * kBigRow + f * 64) = c[f][g];
        };
        if (round == 0) {
            put(0, acc[0][0]);
            put(64, GATED ? acc[1][0] : acc[0][1]);
        } else {
            put(0, GATED ? acc[0][1] : acc[1][0]);
            put(64, acc[1][1]);
        }
        if (ksplit > 1) {
            for (int r = q4; r < ROWS; r += 4)
                if (const int t = token(r); t >= 0) store_part<GATED>(p, ks, t, n, *sums(r), *sums((GATED ? 64 : 0) + r));
            continue;
        }
        float ba[4], bu[4] = {};
        bias4<F16>(p.bias, p.bias_f32, n, p.N, ba);
        if (GATED) bias4<F16>(p.bias_up, p.bias_f32, n, p.N, bu);
        auto activated = [&](int r0, float(&a)[4 * R]) {  // rows r0 + 4 i
            float u[4 * R];
#pragma unroll
            for (int i = 0; i < R; i++) {
                const f32x4_t c = *sums(r0 + 4 * i);
                f32x4_t d = {};
                if (GATED) d = *sums(64 + r0 + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    a[4 * i + j] = c[j] + ba[j];
                    u[4 * i + j] = GATED ? d[j] + bu[j] : 0.0f;
                }
            }
            activate<GATED>(a, u, p.act, p.b1, p.b2);
        };
        if (!direct) {
#pragma unroll 1
            for (int r0 = q4; r0 < ROWS; r0 += 4 * R) {
                int t[R];
                float a[4 * R];
                uint4 res[R] = {};
#pragma unroll
                for (int i = 0; i < R; i++) t[i] = token(r0 + 4 * i);
                load_res<R>(p, t, n, res);
                activated(r0, a);
                write_rows<F16, R>(p, t, n, a, res);
            }
            continue;
        }
        auto store = [&](int k, const f32x4_t &v) {
            if (p.out_half)
                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, pack4<F16>(v[0], v[1], v[2], v[3])), rh, vh,
                                                      row_at(k, p.ldo, 2), 0);
            if (p.out_f32)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rf, vf, row_at(k, p.ldo, 4), 0);
        };
        // the activation in a loop, so that its code is there once; back to
        // LDS where the residual, in registers, waits for it
        if (GATED || p.act != MOE_LINEAR_NONE) {
#pragma unroll 1
            for (int k = 0; k < ROWS / 4; k += R) {
                float a[4 * R];
                activated(q4 + 4 * k, a);
#pragma unroll
                for (int i = 0; i < R; i++) {
                    const f32x4_t v = {a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]};
                    if (p.res) *sums(q4 + 4 * (k + i)) = v;
                    else store(k + i, v);
                }
            }
            if (!p.res) continue;
#pragma unroll
            for (int j = 0; j < 4; j++) ba[j] = 0.0f;
        }
        auto write = [&](int k, float4 r) {
            const f32x4_t c = *sums(q4 + 4 * k);
            store(k, f32x4_t{c[0] + ba[0] + r.x, c[1] + ba[1] + r.y, c[2] + ba[2] + r.z, c[3] + ba[3] + r.w});
        };
        if (!p.res) {
#pragma unroll
            for (int k = 0; k < ROWS / 4; k++) write(k, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        } else if (!p.res_f32) {
#pragma unroll
            for (int k = 0; k < ROWS / 4; k++)
                write(k, make_float4(half_f32<F16>((uint16_t)early[k].x), half_f32<F16>((uint16_t)(early[k].x >> 16)),
                                     half_f32<F16>((uint16_t)early[k].y), half_f32<F16>((uint16_t)(early[k].y >> 16))));
        } else {
            constexpr int PART = ROWS / 16;  // (fp32: a quarter of the rows at a time)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                float4 res[PART];
#pragma unroll
                for (int k = 0; k < PART; k++)
                    res[k] = __builtin_bit_cast(
                        float4, __builtin_amdgcn_raw_buffer_load_b128(rr, vr, row_at(q * PART + k, p.ldr, 4), 0));
#pragma unroll
                for (int k = 0; k < PART; k++) write(q * PART + k, res[k]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
}

// ------------------------------------------------------- a few hundred tokens

__device__ __forceinline__ f32x4_t mfma16v(bf16x8_t a, bf16x8_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma16v(f16x8_t a, f16x8_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// TN weight rows (gated: TN / 2 of each matrix) x TM tokens per block, K in a
// ring of NST stages of 64; WN x WT waves.  Each wave holds fragments a step
// ahead of its products.  The 128-row tiles are bound by LDS at 128 bytes a
// clock: a stage of the 128 x 128 tile reads 96 KB of fragments (12 KB by each
// of eight waves) and receives 32, 1024 clocks (0.47 us) against about 512 of
// products, the 128 x 64 tile 64 and 24 KB, 704 clocks (0.32 us) against 256.
// The small ones are bound by a stage's latency (the ring's length beyond
// three stages changes nothing: 24 x 3584 x 6144 12.4 us with three and six).
// Measured with inputs in the caches and from memory (in brackets the
// library's product): 200 x 3584 x 7168 (128 x 64) 19.8 and 26.6 us (23, 26),
// 4096 x 7168 x 896 to fp32 (128 x 128) 52 and 70 (56, 66), 24 x 3584 x 2 x
// 6144 (64 x 32) 15.6 and 19.5 (21, 22), which is 4500 GB/s of weights.  Rows
// that are not 16-byte aligned (ANY) go through registers, for both operands:
// 333 x 1117 x 2049 12.8 and 13.9 us (21, 21), 2048 x 1117 x 2049 38 and 41
// (27, 27), 2048 x 3585 x 3587 86 and 116 (74, 89).
template <int TN, int TM, int WN, int WT, int NST>
struct Tile {
    static constexpr int NW = WN * WT, THREADS = NW * 64;
    static constexpr int STAGE = (TN + TM) * 128;
    static constexpr int CW = STAGE / 1024 / NW;     // copies per wave and stage
    static constexpr int FN = TN / 2 / WN / 16;      // 16-row tiles per wave and half
    static constexpr int FT = TM / WT / 16;
    static constexpr int EN = TN / 2 / WN;           // epilogue: outputs per row of a wave's half
    static constexpr int EROW = EN * 4 + 16;
    static constexpr int EWAVE = 2 * (TM / WT) * EROW;
    static constexpr int LDSB = NST * STAGE > NW * EWAVE ? NST * STAGE : NW * EWAVE;
    static_assert(TN / 16 % NW == 0 && TM / 8 % NW == 0 && FN >= 1 && FT >= 1 && EN % 16 == 0 && NST >= 3, "tile");
};

template <bool F16, bool GATED, bool ANY, int TN, int TM, int WN, int WT, int NST>
__global__ __launch_bounds__(WN * WT * 64) void k_linear_tile(LinearParams p, int tn, int tt, int ksplit)
{
    using G = Tile<TN, TM, WN, WT, NST>;
    using V = typename Frag<F16>::V;
    __shared__ __align__(1024) uint8_t lds_blk[G::LDSB];
    LDS uint8_t *lds = (LDS uint8_t *)lds_blk;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ti, ni;
    tile_of(blockIdx.x % (tn * tt), tn, tt, ni, ti);
    const int ks = blockIdx.x / (tn * tt);
    const int t0 = ti * TM, n0 = ni * (GATED ? TN / 2 : TN);
    const int SA = (p.K + 63) / 64, s0 = (int)((int64_t)SA * ks / ksplit), s1 = (int)((int64_t)SA * (ks + 1) / ksplit);

    // rows of the two weight halves and of the tokens
    const uint16_t *W = reinterpret_cast<const uint16_t *>(p.w), *U = reinterpret_cast<const uint16_t *>(p.w_up);
    const int n1 = GATED ? n0 : n0 + TN / 2;
    const __amdgpu_buffer_rsrc_t r0 = rows_rsrc(W + (size_t)n0 * p.ldw, min(TN / 2, p.N - n0), p.ldw, p.K);
    const __amdgpu_buffer_rsrc_t r1 =
        rows_rsrc(n1 < p.N ? (GATED ? U : W) + (size_t)n1 * p.ldw : W, min(TN / 2, p.N - n1), p.ldw, p.K);
    const __amdgpu_buffer_rsrc_t rx =
        rows_rsrc(reinterpret_cast<const uint16_t *>(p.x) + (size_t)t0 * p.ldx, min(TM, p.M - t0), p.ldx, p.K);
    // copies: pieces of 8 rows; the wave takes pieces wv + NW j of the
    // stage's, so that copy j is of the same rows' matrix for every wave
    const int l8 = lane >> 3;
    const uint32_t lbase = (uint32_t)(uintptr_t)lds + wv * 1024;
    uint32_t cv[G::CW];
    const int kc = ((lane & 7) ^ ((4 * wv + (l8 >> 1)) & 7)) * 8;  // this lane's k in them
#pragma unroll
    for (int j = 0; j < G::CW; j++) {
        const int pc = wv + G::NW * j;
        const bool isx = G::NW * j >= TN / 8;
        const int row = (isx ? pc - TN / 8 : pc % (TN / 16)) * 8 + l8;
        cv[j] = (uint32_t)(row * (isx ? p.ldx : p.ldw) * 2) + (kc + s0 * 64) * 2;
    }
    // copy j of a stage (the next one in turn for that j) into a slot; checked where the stage may end past K or s1
    auto copy = [&](auto check, int stage, int slot, int j) {
        const uint32_t at = lbase + slot * G::STAGE + G::NW * j * 1024;
        uint32_t v = cv[j];
        if (decltype(check)::value) v = stage * 64 + kc < p.K && stage < s1 ? v : 0x80000000u;
        cv[j] += 128;
        if (G::NW * j >= TN / 8) copy16(rx, at, v);
        else if (G::NW * j < TN / 16) copy16(r0, at, v);
        else copy16(r1, at, v);
    };
    // ANY: rows that direct copies cannot take (they want 16-byte pieces) go
    // through registers, loaded two stages before they are stored; rows past
    // the end repeat the last one, and their sums are not written
    const uint16_t *rp[G::CW];
    uint4 held[2][G::CW];
#pragma unroll
    for (int j = 0; ANY && j < G::CW; j++) {
        const int pc = wv + G::NW * j, half = G::NW * j >= TN / 16;
        if (G::NW * j >= TN / 8)
            rp[j] = reinterpret_cast<const uint16_t *>(p.x) + (size_t)min(t0 + (pc - TN / 8) * 8 + l8, p.M - 1) * p.ldx;
        else
            rp[j] = (GATED && half ? U : W) + (size_t)min((half ? n1 : n0) + pc % (TN / 16) * 8 + l8, p.N - 1) * p.ldw;
    }
    auto load = [&](auto check, uint4(&h)[G::CW], int stage, int j) {
        const int k = stage * 64 + kc;
        if (!decltype(check)::value) {
            __builtin_memcpy(&h[j], rp[j] + k, 16);
        } else {
            h[j] = make_uint4(0, 0, 0, 0);
            if (stage < s1) h[j] = load8(rp[j], k, p.K);
        }
    };
    auto store = [&](const uint4(&h)[G::CW], int slot, int j) {
        *reinterpret_cast<LDS u32x4_t *>(lds + wv * 1024 + slot * G::STAGE + G::NW * j * 1024 + lane * 16) =
            __builtin_bit_cast(u32x4_t, h[j]);
    };
    const int r16 = lane & 15, q4 = lane >> 4;
    const int wn = wv / WT, wt = wv % WT;
    int fa[2], fb[2];
#pragma unroll
    for (int st = 0; st < 2; st++) {
        const int o = r16 * 128 + (((st * 4 + q4) ^ (r16 >> 1)) << 4);
        fa[st] = wn * (TN / 2 / WN) * 128 + o;
        fb[st] = TN * 128 + wt * (TM / WT) * 128 + o;
    }
    constexpr int FA = 2 * G::FN, FT = G::FT, NM = FA * FT, NR = FA + FT;
    f32x4_t acc[FA][FT] = {};  // rows of half 0, then of half 1
    V a[2][FA], b[2][FT];
    // read i (the token fragments first) of step st of a slot
    auto read = [&](int slot, int st, int i) {
        const LDS uint8_t *base = lds + slot * G::STAGE;
        if (i < FT) {
            b[st][i] = __builtin_bit_cast(V, lds_ld16(base + fb[st] + i * 2048));
        } else {
            const int f = i - FT;
            a[st][f] = __builtin_bit_cast(V, lds_ld16(base + fa[st] + (f / G::FN) * (TN / 2) * 128 + (f % G::FN) * 2048));
        }
    };
    // the products of step st, and spread between them the reads of the next
    // step and (at the second step) the copies of the stage NST - 1 on
    auto part = [&](auto check, int st, int slot, int stage, int into) {
#pragma unroll
        for (int i = 0; i < NM; i++) {
            const int f = i / FT, g = f & 1 ? FT - 1 - i % FT : i % FT;
            acc[f][g] = mfma16v(a[st][f], b[st][g], acc[f][g]);
#pragma unroll
            for (int j = i * NR / NM; j < (i + 1) * NR / NM; j++) read(slot, 1 - st, j);
            if (!ANY && st == 1) {
#pragma unroll
                for (int j = i * G::CW / NM; j < (i + 1) * G::CW / NM; j++) copy(check, stage, into, j);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (ANY) {
        // stage s + 2 is stored in the middle of stage s, stage s + 4 loaded then
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < G::CW; j++) load(std::true_type{}, held[i], s0 + i, j);
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < G::CW; j++) {
                store(held[i], i, j);
                load(std::true_type{}, held[i], s0 + 2 + i, j);
            }
        lds_barrier();
    } else {
#pragma unroll
        for (int i = 0; i < NST - 1; i++)
#pragma unroll
            for (int j = 0; j < G::CW; j++) copy(std::true_type{}, s0 + i, i, j);
        wait_copies<(NST - 2) * G::CW>();
        barrier();
    }
#pragma unroll
    for (int i = 0; i < NR; i++) read(0, 0, i);
    int slot = 0;
    auto one_stage = [&](auto check, int s, uint4(&h)[G::CW]) {
        const int next = slot + 1 == NST ? 0 : slot + 1, last = slot == 0 ? NST - 1 : slot - 1;
        __builtin_amdgcn_sched_barrier(0);
        part(check, 0, slot, 0, 0);
        // (every wave has read the last stage's slot by now: it is filled anew below)
        if (ANY) lds_barrier();  // (loads into registers stay in flight across it)
        else wait_copies<(NST - 3) * G::CW, 15>(), barrier();
        __builtin_amdgcn_sched_barrier(0);
        part(check, 1, next, s + NST - 1, last);
        if (ANY) {
#pragma unroll
            for (int j = 0; j < G::CW; j++) {
                store(h, last, j);
                load(check, h, s + 4, j);
            }
        }
        slot = next;
    };
    int s = s0;
    if (ANY) {
        const int whole = min(s1, p.K / 64) - 5;  // two stages from this one on still load whole stages
        for (; s <= whole - 1; s += 2) {
            one_stage(std::false_type{}, s, held[0]);
            one_stage(std::false_type{}, s + 1, held[1]);
        }
        for (; s + 1 < s1; s += 2) {
            one_stage(std::true_type{}, s, held[0]);
            one_stage(std::true_type{}, s + 1, held[1]);
        }
        if (s < s1) one_stage(std::true_type{}, s, held[0]);
    } else {
        const int whole = min(s1, p.K / 64) - (NST - 1);  // stages before this one copy whole stages of the block's
        for (; s < whole; s++) one_stage(std::false_type{}, s, held[0]);
        for (; s < s1; s++) one_stage(std::true_type{}, s, held[0]);
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_copies<0>();
    barrier();

    // epilogue through the wave's own LDS: rows of tokens, EN sums of each
    // half; a lane has four outputs of R rows of a half.  Every residual is
    // loaded before the first store (a load waits for the stores before it).
    LDS uint8_t *buf = lds + wv * G::EWAVE;
    constexpr int TR = TM / WT, LPR = G::EN / 4, RPI = 64 / LPR, R = TR / RPI, HALVES = GATED ? 1 : 2;
    static_assert(TR % RPI == 0, "rows");
    const int c4 = (lane % LPR) * 4, row0 = lane / LPR;
    int t[HALVES][R];
    uint4 res[HALVES][R] = {};
#pragma unroll
    for (int h = 0; h < HALVES; h++) {
        const int n = (h ? n1 : n0) + wn * G::EN + c4;
#pragma unroll
        for (int i = 0; i < R; i++) {
            t[h][i] = t0 + wt * TR + row0 + i * RPI;
            t[h][i] = t[h][i] < p.M && n < p.N ? t[h][i] : -1;
        }
        if (ksplit == 1) load_res<R>(p, t[h], n, res[h]);
    }
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
        for (int f = 0; f < G::FN; f++)
#pragma unroll
            for (int g = 0; g < G::FT; g++)
                *reinterpret_cast<LDS f32x4_t *>(buf + (h * TR + g * 16 + r16) * G::EROW + f * 64 + q4 * 16) = acc[h * G::FN + f][g];
    auto sums = [&](int h, int i) {
        return *reinterpret_cast<const LDS f32x4_t *>(buf + (h * TR + row0 + i * RPI) * G::EROW + c4 * 4);
    };
#pragma unroll
    for (int h = 0; h < HALVES; h++) {
        const int n = (h ? n1 : n0) + wn * G::EN + c4;
        if (ksplit > 1) {
#pragma unroll
            for (int i = 0; i < R; i++)
                if (t[h][i] >= 0) store_part<GATED>(p, ks, t[h][i], n, sums(h, i), sums(GATED ? 1 : h, i));
            continue;
        }
        float a[4 * R], u[4 * R], ba[4], bu[4] = {};
        bias4<F16>(p.bias, p.bias_f32, n, p.N, ba);
        if (GATED) bias4<F16>(p.bias_up, p.bias_f32, n, p.N, bu);
#pragma unroll
        for (int i = 0; i < R; i++) {
            const f32x4_t c = sums(h, i), d = sums(GATED ? 1 : h, i);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                a[4 * i + j] = c[j] + ba[j];
                u[4 * i + j] = GATED ? d[j] + bu[j] : 0.0f;
            }
        }
        activate<GATED>(a, u, p.act, p.b1, p.b2);
        write_rows<F16, R>(p, t[h], n, a, res[h]);
    }
}

// sums of the K parts, in their order, and the epilogue: a thread per four
// outputs.  A launch of its own (about 2 us) and not the last block's work:
// the sums keep their order, and no counter has to be cleared.
template <bool F16, bool GATED, int KS>
__global__ __launch_bounds__(256) void k_linear_join(LinearParams p)
{
    const int nq = (p.N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int t[1] = {(int)(i / nq)}, n = (int)(i % nq) * 4;
    if (t[0] >= p.M) return;
    const size_t plane = (size_t)p.M * part_pitch(p);
    const float *o = p.part + (size_t)t[0] * part_pitch(p) + n;
    constexpr int PL = GATED ? 2 : 1;
    f32x4_t v[KS * PL];
#pragma unroll
    for (int k = 0; k < KS * PL; k++) v[k] = *reinterpret_cast<const f32x4_t *>(o + k * plane);
    float a[4], u[4] = {}, ba[4], bu[4] = {};
    bias4<F16>(p.bias, p.bias_f32, n, p.N, ba);
    if (GATED) bias4<F16>(p.bias_up, p.bias_f32, n, p.N, bu);
#pragma unroll
    for (int k = 1; k < KS; k++) {
        v[0] += v[k * PL];
        if (GATED) v[1] += v[k * PL + 1];
    }
#pragma unroll
    for (int j = 0; j < 4; j++) {
        a[j] = v[0][j] + ba[j];
        u[j] = GATED ? v[PL - 1][j] + bu[j] : 0.0f;
    }
    finish_row<F16, GATED>(p, t[0], n, a, u);
}

// ------------------------------------------------------------ served batches

// A block multiplies 16 weight rows (gated: 16 of each matrix) with 8 XP
// tokens; each of its eight waves takes an eighth of K through a ring of NST
// stages of 64 in LDS of its own, filled by direct copies, so no wave waits
// for another until the sums join.  Tokens past the end are zeros.  Bound by
// the weights' way: 1 x 7168 x 3584 10.0 us, 5140 GB/s, where the caches hold
// them, 11.5 us, 4470 GB/s, from memory (the first kernel, a wave per row
// without LDS, took 91).
// One stage more in the ring takes the same time.
constexpr int kFewWaves = 8;

template <bool GATED, int XP, int NST>
struct Few {
    static constexpr int NR = GATED ? 2 : 1, MT = (XP + 1) / 2;
    static constexpr int CW = 2 * NR + XP, STAGE = CW * 1024;
    static constexpr int RING = kFewWaves * NST * STAGE, JOIN = kFewWaves * NR * MT * 1024;
    static constexpr int LDSB = RING > JOIN ? RING : JOIN;
};

template <bool F16, bool GATED, int XP, int NST>
__global__ __launch_bounds__(kFewWaves * 64) void k_linear_few(LinearParams p)
{
    using G = Few<GATED, XP, NST>;
    using V = typename Frag<F16>::V;
    __shared__ __align__(1024) uint8_t lds_blk[G::LDSB];
    LDS uint8_t *lds = (LDS uint8_t *)lds_blk;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, q4 = lane >> 4, l8 = lane >> 3;
    const int n0 = blockIdx.x * 16, t0 = blockIdx.y * 8 * XP;
    const int SA = (p.K + 63) / 64, s0 = (int)((int64_t)SA * wv / kFewWaves), s1 = (int)((int64_t)SA * (wv + 1) / kFewWaves);
    const uint16_t *W = reinterpret_cast<const uint16_t *>(p.w), *U = reinterpret_cast<const uint16_t *>(p.w_up);
    const __amdgpu_buffer_rsrc_t rw = rows_rsrc(W + (size_t)n0 * p.ldw, min(16, p.N - n0), p.ldw, p.K);
    const __amdgpu_buffer_rsrc_t ru = GATED ? rows_rsrc(U + (size_t)n0 * p.ldw, min(16, p.N - n0), p.ldw, p.K) : rw;
    const __amdgpu_buffer_rsrc_t rx =
        rows_rsrc(reinterpret_cast<const uint16_t *>(p.x) + (size_t)t0 * p.ldx, min(8 * XP, p.M - t0), p.ldx, p.K);
    uint32_t cw[2], cx[XP];
    const int piece = (lane & 7) ^ (l8 >> 1);
    const int kc[2] = {piece * 8, (piece ^ 4) * 8};
#pragma unroll
    for (int j = 0; j < 2; j++) cw[j] = (uint32_t)((8 * j + l8) * p.ldw * 2) + (kc[j] + s0 * 64) * 2;
#pragma unroll
    for (int j = 0; j < XP; j++) cx[j] = (uint32_t)((8 * j + l8) * p.ldx * 2) + (kc[j & 1] + s0 * 64) * 2;
    LDS uint8_t *ring = lds + wv * NST * G::STAGE;
    const uint32_t mring = (uint32_t)(uintptr_t)ring;
    auto copies = [&](int stage, int slot) {  // the next stage in turn
        const uint32_t at = mring + slot * G::STAGE;
        const bool in = stage < s1;
        const bool ok[2] = {in && stage * 64 + kc[0] < p.K, in && stage * 64 + kc[1] < p.K};
#pragma unroll
        for (int j = 0; j < 2; j++) {
            copy16(rw, at + j * 1024, ok[j] ? cw[j] : 0x80000000u);
            if (GATED) copy16(ru, at + (2 + j) * 1024, ok[j] ? cw[j] : 0x80000000u);
            cw[j] += 128;
        }
#pragma unroll
        for (int j = 0; j < XP; j++) {
            copy16(rx, at + (2 * G::NR + j) * 1024, ok[j & 1] ? cx[j] : 0x80000000u);
            cx[j] += 128;
        }
    };
    int fo[2];
#pragma unroll
    for (int st = 0; st < 2; st++) fo[st] = r16 * 128 + (((st * 4 + q4) ^ (r16 >> 1)) << 4);
    // (eight tokens: the other half of the tile repeats them)
    const int fx = XP == 1 ? fo[0] & 1023 : fo[0], fx1 = XP == 1 ? fo[1] & 1023 : fo[1];
    f32x4_t acc[G::NR][G::MT] = {};
#pragma unroll
    for (int i = 0; i < NST; i++) copies(s0 + i, i);
    int slot = 0;
    for (int s = s0; s < s1; s++) {
        wait_copies<(NST - 1) * G::CW>();
        const LDS uint8_t *base = ring + slot * G::STAGE;
        V a[2][G::NR], b[2][G::MT];
#pragma unroll
        for (int st = 0; st < 2; st++) {
#pragma unroll
            for (int i = 0; i < G::NR; i++) a[st][i] = __builtin_bit_cast(V, lds_ld16(base + fo[st] + i * 2048));
#pragma unroll
            for (int m = 0; m < G::MT; m++)
                b[st][m] = __builtin_bit_cast(V, lds_ld16(base + 2 * G::NR * 1024 + (st ? fx1 : fx) + m * 2048));
        }
        wait_copies<63>();  // (the reads are done: the slot may be filled again)
        copies(s + NST, slot);
#pragma unroll
        for (int st = 0; st < 2; st++)
#pragma unroll
            for (int i = 0; i < G::NR; i++)
#pragma unroll
                for (int m = 0; m < G::MT; m++) acc[i][m] = mfma16v(a[st][i], b[st][m], acc[i][m]);
        slot = slot + 1 == NST ? 0 : slot + 1;
    }
    wait_copies<0>();
    barrier();
    LDS f32x4_t *part = (LDS f32x4_t *)lds_blk;
#pragma unroll
    for (int i = 0; i < G::NR; i++)
#pragma unroll
        for (int m = 0; m < G::MT; m++) part[((i * G::MT + m) * kFewWaves + wv) * 64 + lane] = acc[i][m];
    __syncthreads();
    for (int m = wv; m < G::MT; m += kFewWaves) {
        const int n = n0 + q4 * 4;
        const int t[1] = {t0 + m * 16 + r16};
        if (t[0] >= min(p.M, t0 + 8 * XP) || n >= p.N) continue;
        float a[4], u[4] = {}, ba[4], bu[4] = {};
        bias4<F16>(p.bias, p.bias_f32, n, p.N, ba);
        if (GATED) bias4<F16>(p.bias_up, p.bias_f32, n, p.N, bu);
        f32x4_t ca = {}, cu = {};
#pragma unroll
        for (int w = 0; w < kFewWaves; w++) {
            ca += part[(m * kFewWaves + w) * 64 + lane];
            if (GATED) cu += part[((G::MT + m) * kFewWaves + w) * 64 + lane];
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
            a[e] = ca[e] + ba[e];
            u[e] = cu[e] + bu[e];
        }
        finish_row<F16, GATED>(p, t[0], n, a, u);
    }
}

// ----------------------------------------------------------------- launching

template <bool F16, bool GATED>
void launch_join(const LinearParams &p, int ksplit, hipStream_t st)
{
    const int grid = (int)(((int64_t)p.M * ((p.N + 3) / 4) + 255) / 256);
    if (ksplit == 2) k_linear_join<F16, GATED, 2><<<grid, 256, 0, st>>>(p);
    else if (ksplit == 4) k_linear_join<F16, GATED, 4><<<grid, 256, 0, st>>>(p);
    else if (ksplit == 8) k_linear_join<F16, GATED, 8><<<grid, 256, 0, st>>>(p);
}

template <bool F16, bool GATED, int XP, int NST>
void launch_few(const LinearParams &p, hipStream_t st)
{
    const dim3 grid((p.N + 15) / 16, (p.M + 8 * XP - 1) / (8 * XP));
    k_linear_few<F16, GATED, XP, NST><<<grid, kFewWaves * 64, 0, st>>>(p);
}

template <bool F16, bool GATED, bool ANY, int TN, int TM, int WN, int WT, int NST>
void launch_tile(const LinearParams &p, int ksplit, hipStream_t st)
{
    constexpr int NB = GATED ? TN / 2 : TN;
    const int tt = (p.M + TM - 1) / TM, tn = (p.N + NB - 1) / NB;
    k_linear_tile<F16, GATED, ANY, TN, TM, WN, WT, NST><<<tn * tt * ksplit, WN * WT * 64, 0, st>>>(p, tn, tt, ksplit);
    launch_join<F16, GATED>(p, ksplit, st);
}

template <bool F16, bool GATED>
void launch_big(const LinearParams &p, int ksplit, hipStream_t st)
{
    constexpr int NB = GATED ? 128 : 256;
    const int tt = (p.M + 255) / 256, tn = (p.N + NB - 1) / NB;
    k_linear_big<F16, GATED><<<tn * tt * ksplit, 256, 0, st>>>(p, tn, tt, ksplit);
    launch_join<F16, GATED>(p, ksplit, st);
}

template <bool F16, bool GATED>
void launch_gated(const LinearParams &p, const LinearPlan &c, hipStream_t st)
{
    switch (c.kind) {
    case kFew1: return launch_few<F16, GATED, 1, GATED ? 2 : 3>(p, st);
    case kFew2: return launch_few<F16, GATED, 2, 2>(p, st);
    case kFew4: return launch_few<F16, GATED, 4, 2>(p, st);
    case kTile64x32: return launch_tile<F16, GATED, false, 64, 32, 2, 2, 6>(p, c.ksplit, st);
    case kTile64x64: return launch_tile<F16, GATED, false, 64, 64, 2, 2, 5>(p, c.ksplit, st);
    case kTile128x64: return launch_tile<F16, GATED, false, 128, 64, 4, 2, 6>(p, c.ksplit, st);
    case kTile128x128: return launch_tile<F16, GATED, false, 128, 128, 2, 4, 4>(p, c.ksplit, st);
    case kAny64x32: return launch_tile<F16, GATED, true, 64, 32, 2, 2, 3>(p, c.ksplit, st);
    case kAny64x64: return launch_tile<F16, GATED, true, 64, 64, 2, 2, 3>(p, c.ksplit, st);
    case kAny128x128: return launch_tile<F16, GATED, true, 128, 128, 2, 4, 3>(p, c.ksplit, st);
    case kBig: return launch_big<F16, GATED>(p, c.ksplit, st);
    }
}

template <bool F16>
void launch_typed(const LinearParams &p, const LinearPlan &c, hipStream_t st)
{
    if (p.w_up) launch_gated<F16, true>(p, c, st);
    else launch_gated<F16, false>(p, c, st);
}

}  // namespace
}  // namespace moe
