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

// a[i] = act(a[i], u[i]): one branch for all NV values
template <bool GATED, int NV>
__device__ __forceinline__ void activate(float (&a)[NV], const float (&u)[NV], int act, float b1, float b2)
{
    if (GATED) {
        if (act == MOE_LINEAR_SITU_GLU) {
#pragma unroll
            for (int i = 0; i < NV; i++) a[i] = gated_act(a[i], u[i], 0, b1, b2);
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

// R rows of four outputs each, n .. n + 3 of tokens t[i], from their sums a
// and u (biases included); rows with t[i] < 0 are not there.  p.vec: all four
// outputs exist and every row of the residual and the outputs is aligned for
// them.
template <bool F16, bool GATED, int R>
__device__ __forceinline__ void finish_rows(const LinearParams &p, const int (&t)[R], int n, float (&a)[4 * R],
                                            const float (&u)[4 * R])
{
    activate<GATED>(a, u, p.act, p.b1, p.b2);
    const float *rf = reinterpret_cast<const float *>(p.res);
    const uint16_t *rh = reinterpret_cast<const uint16_t *>(p.res);
    uint16_t *oh = reinterpret_cast<uint16_t *>(p.out_half);
    if (p.vec) {
        if (p.res && p.res_f32) {
            float4 v[R];
#pragma unroll
            for (int i = 0; i < R; i++)
                if (t[i] >= 0) v[i] = *reinterpret_cast<const float4 *>(rf + (size_t)t[i] * p.ldr + n);
#pragma unroll
            for (int i = 0; i < R; i++) {
                a[4 * i] += v[i].x;
                a[4 * i + 1] += v[i].y;
                a[4 * i + 2] += v[i].z;
                a[4 * i + 3] += v[i].w;
            }
        } else if (p.res) {
            ushort4 v[R];
#pragma unroll
            for (int i = 0; i < R; i++)
                if (t[i] >= 0) v[i] = *reinterpret_cast<const ushort4 *>(rh + (size_t)t[i] * p.ldr + n);
#pragma unroll
            for (int i = 0; i < R; i++) {
                a[4 * i] += half_f32<F16>(v[i].x);
                a[4 * i + 1] += half_f32<F16>(v[i].y);
                a[4 * i + 2] += half_f32<F16>(v[i].z);
                a[4 * i + 3] += half_f32<F16>(v[i].w);
            }
        }
        if (oh) {
#pragma unroll
            for (int i = 0; i < R; i++)
                if (t[i] >= 0)
                    *reinterpret_cast<uint2 *>(oh + (size_t)t[i] * p.ldo + n) =
                        pack4<F16>(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
        }
        if (p.out_f32) {
#pragma unroll
            for (int i = 0; i < R; i++)
                if (t[i] >= 0)
                    *reinterpret_cast<float4 *>(p.out_f32 + (size_t)t[i] * p.ldo + n) =
                        make_float4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
        }
        return;
    }
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

// the biases of outputs n .. n + 3
template <bool F16>
__device__ __forceinline__ void bias4(const void *b, int f32, int n, int N, float (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = n + i < N ? bias_at<F16>(b, f32, n + i) : 0.0f;
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
    const int t[1] = {t0 + tw + (lane & 31) < p.M ? t0 + tw + (lane & 31) : -1};
#pragma unroll
    for (int g = 0; g < 4; g++) {
        const int n = n0 + nw + 8 * g + 4 * (lane >> 5);
        if (n >= p.N) continue;
        float ba[4], bu[4] = {};
        bias4<F16>(p.bias, p.bias_f32, n, p.N, ba);
        if (GATED) bias4<F16>(p.bias_up, p.bias_f32, n, p.N, bu);
        float a[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            a[i] = acc[4 * g + i] + ba[i];
            u[i] = GATED ? acu[4 * g + i] + bu[i] : 0.0f;
        }
        finish_rows<F16, GATED, 1>(p, t, n, a, u);
    }
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

template <bool F16, bool GATED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_linear_big(LinearParams p, int tn,
                                                                                               int tt)
{
    using V = typename Frag<F16>::V;
    __shared__ __align__(1024) uint8_t lds_blk[kBigLds];
    LDS uint8_t *lds = (LDS uint8_t *)lds_blk;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int ti, ni;
    tile_of(blockIdx.x, tn, tt, ni, ti);
    const int t0 = ti * 256, n0 = ni * (GATED ? 128 : 256);
    const uint16_t *W = reinterpret_cast<const uint16_t *>(p.w), *U = reinterpret_cast<const uint16_t *>(p.w_up);
    const uint16_t *X = reinterpret_cast<const uint16_t *>(p.x) + (size_t)t0 * p.ldx;
    const int na1 = n0 + 128;
    const __amdgpu_buffer_rsrc_t rA0 = rows_rsrc(W + (size_t)n0 * p.ldw, min(128, p.N - n0), p.ldw, p.K);
    const __amdgpu_buffer_rsrc_t rA1 =
        GATED ? rows_rsrc(U + (size_t)n0 * p.ldw, min(128, p.N - n0), p.ldw, p.K)
              : rows_rsrc(na1 < p.N ? W + (size_t)na1 * p.ldw : W, min(128, p.N - na1), p.ldw, p.K);
    const __amdgpu_buffer_rsrc_t rB0 = rows_rsrc(X, min(128, p.M - t0), p.ldx, p.K);
    const __amdgpu_buffer_rsrc_t rB1 =
        rows_rsrc(t0 + 128 < p.M ? X + (size_t)128 * p.ldx : X, min(128, p.M - t0 - 128), p.ldx, p.K);

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
        if (decltype(check)::value) v = (j & 1 ? kc1 : kc0) + D * 64 < p.K ? v : 0x80000000u;
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
    const int S = (p.K + 63) / 64;
    int s = 0;
    for (; 64 * (s + 4) <= p.K; s += 2) two_stages(No{});
    for (; s < S; s += 2) two_stages(Yes{});
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");  // the last products' results (written-out products: the compiler does not wait)
    wait_copies<0>();
    barrier();

    // epilogue: 64 n x 128 tokens of sums (gated: 64 tokens of both matrices)
    // at a time through the wave's own LDS, so that a row's 64 outputs leave
    // as 16 lanes x 4
    LDS uint8_t *buf = lds + wv * kBigWave;
    const int c4 = (lane & 15) * 4;
    const int row_l = r16 * kBigRow + q4 * 16;
    constexpr int R = 4;
#pragma unroll 1
    for (int round = 0; round < 2; round++) {
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
        const int n = n0 + (GATED ? 0 : round * 128) + wn * 64 + c4;
        if (n < p.N) {
            float ba[4], bu[4] = {};
            bias4<F16>(p.bias, p.bias_f32, n, p.N, ba);
            if (GATED) bias4<F16>(p.bias_up, p.bias_f32, n, p.N, bu);
#pragma unroll 1
            for (int r0 = q4; r0 < (GATED ? 64 : 128); r0 += 4 * R) {
                int t[R];
                float a[4 * R], u[4 * R];
#pragma unroll
                for (int i = 0; i < R; i++) {
                    const int r = r0 + 4 * i;
                    t[i] = t0 + (GATED ? round * 128 + r : (r >> 6) * 128 + (r & 63)) + wt * 64;
                    t[i] = t[i] < p.M ? t[i] : -1;
                    const f32x4_t c = *reinterpret_cast<const LDS f32x4_t *>(buf + r * kBigRow + c4 * 4);
                    f32x4_t d = {};
                    if (GATED) d = *reinterpret_cast<const LDS f32x4_t *>(buf + (64 + r) * kBigRow + c4 * 4);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        a[4 * i + j] = c[j] + ba[j];
                        u[4 * i + j] = GATED ? d[j] + bu[j] : 0.0f;
                    }
                }
                finish_rows<F16, GATED, R>(p, t, n, a, u);
            }
        }
    }
}

template <bool F16>
void launch_any(const LinearParams &p, hipStream_t st)
{
    const dim3 grid((p.N + kAnyTile - 1) / kAnyTile, (p.M + kAnyTile - 1) / kAnyTile);
    if (p.w_up) k_linear_any<F16, true><<<grid, 256, 0, st>>>(p);
    else k_linear_any<F16, false><<<grid, 256, 0, st>>>(p);
}

template <bool F16>
void launch_big(const LinearParams &p, hipStream_t st)
{
    const int tt = (p.M + 255) / 256, tn = (p.N + (p.w_up ? 127 : 255)) / (p.w_up ? 128 : 256);
    if (p.w_up) k_linear_big<F16, true><<<tn * tt, 256, 0, st>>>(p, tn, tt);
    else k_linear_big<F16, false><<<tn * tt, 256, 0, st>>>(p, tn, tt);
}

bool aligned16(const void *q) { return ((uintptr_t)q & 15) == 0; }

// 16-byte pieces: rows of x and w start at multiples of 16 bytes and hold whole pieces
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

template <bool F16>
void launch_typed(const LinearParams &p, hipStream_t st)
{
    if (pieces(p) && p.M > 64) launch_big<F16>(p, st);
    else launch_any<F16>(p, st);
}

}  // namespace

size_t linear_workspace(const LinearParams &) { return 256; }

hipError_t launch_linear(const LinearParams &params, bool f16, hipStream_t st)
{
    LinearParams p = params;
    p.vec = fours(p);
    if (f16) launch_typed<true>(p, st);
    else launch_typed<false>(p, st);
    return hipGetLastError();
}

}  // namespace moe
