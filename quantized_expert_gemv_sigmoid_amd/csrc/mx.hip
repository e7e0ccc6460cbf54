// MXFP4 rows made and read back (moe_mx_quantize, moe_mx_dequantize), and the
// scale rows of moe_mx_linear laid out for its kernels.
//
// A block of 32 values shares a scale 2^e: e = floor(log2(largest magnitude))
// - 2, or one more where that magnitude is past 6 * 2^e (MOE_MX_FIT), at least
// -127; its values over 2^e are rounded to E2M1.  The exponent is read off the
// largest magnitude's bits and the quotients are exact, so nothing is rounded
// but the codes.
//
// Both kernels are bound by memory: 28672 x 3584 bf16 quantised 42-53 us (260 MB,
// 6150-4900 GB/s with inputs in turn), read back 42-48; fp32 84 and 84; one row
// of 7168 2.0 and 2.5 (a launch).  Two quarters of blocks per thread on the way
// at once: one is 5% slower to read back (50.2 us), four 5% slower for short rows
// (60000 x 300: 11.3 us, 10.5 with two).
#include <algorithm>
#include <type_traits>

#include "../../include/moe.h"
#include "common.h"

namespace moe {

namespace {

// i / d for i < 2^31, by a product: m = ceil(2^(31 + s) / d), s = ceil(log2 d)
struct Divisor {
    uint32_t d, m;
    int s;
};
Divisor divisor(uint32_t d)
{
    int s = 0;
    while ((1u << s) < d) s++;
    return {d, (uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d), s};
}
__device__ __forceinline__ uint32_t over(uint32_t i, const Divisor &v) { return (uint32_t)(((uint64_t)i * v.m) >> (31 + v.s)); }

// 2^(b - 127), b = 0 .. 254
__device__ __forceinline__ float pow2_of(uint32_t b) { return __uint_as_float(b == 0 ? 0x00400000u : b << 23); }

template <int TYPE>
struct Eight {  // eight values as they are in memory
    uint4 q[TYPE == MOE_F32 ? 2 : 1];
};

// largest magnitude's bits (as fp32 where TYPE is MOE_F32, else as 16 bits)
template <int TYPE>
__device__ __forceinline__ uint32_t top_of(const Eight<TYPE> &v)
{
    if constexpr (TYPE == MOE_F32) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            m = max(m, v.q[i].x & 0x7fffffffu);
            m = max(m, v.q[i].y & 0x7fffffffu);
            m = max(m, v.q[i].z & 0x7fffffffu);
            m = max(m, v.q[i].w & 0x7fffffffu);
        }
        return m;
    } else {
        typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
        u16x2_t m = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; i++)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, u4at(v.q[0], i) & 0x7fff7fffu));
        return max((uint32_t)m.x, (uint32_t)m.y);
    }
}

// The scale byte of a block from its largest magnitude; 255 for infinities
// and NaN.
template <int TYPE>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top, int fit)
{
    uint32_t bits = top;  // as fp32
    if (TYPE == MOE_BF16) bits = top << 16;
    if (TYPE == MOE_F16) bits = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)top));
    if (bits >= 0x7f800000u) return 255;
    int e = (int)(bits >> 23) - 2;  // (subnormal: below the smallest scale)
    if (fit && (bits & 0x7fffffu) > 0x400000u) e++;
    return (uint32_t)max(e, 0);
}

// eight codes, the first value's in the low nibble
template <int TYPE>
__device__ __forceinline__ uint32_t codes_of(const Eight<TYPE> &v, float scale)
{
    uint32_t c = 0;
    if constexpr (TYPE == MOE_F32) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.q[0].x), __uint_as_float(v.q[0].y), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.q[0].z), __uint_as_float(v.q[0].w), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.q[1].x), __uint_as_float(v.q[1].y), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(v.q[1].z), __uint_as_float(v.q[1].w), scale, 3);
    } else if constexpr (TYPE == MOE_BF16) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.q[0].x), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.q[0].y), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.q[0].z), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v.q[0].w), scale, 3);
    } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2v_t, v.q[0].x), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2v_t, v.q[0].y), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2v_t, v.q[0].z), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2v_t, v.q[0].w), scale, 3);
    }
    return c;
}

struct MxRows {
    int64_t ldx, ldc, lds;   // elements; bytes
    int cols;
    uint32_t items;          // rows x eighths of blocks: four to a block
    Divisor per_row;
    int fit;
};

template <int TYPE>
__device__ __forceinline__ void load_eight(Eight<TYPE> &v, const void *x, int64_t at, int n)
{
    constexpr int SZ = TYPE == MOE_F32 ? 4 : 2;
    const char *p = reinterpret_cast<const char *>(x) + at * SZ;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(v.q) / 16); i++) v.q[i] = make_uint4(0, 0, 0, 0);
    if (n >= 8) {
        __builtin_memcpy(&v, p, sizeof(v.q));
    } else {
        using T = typename std::conditional<TYPE == MOE_F32, uint32_t, uint16_t>::type;
        T h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) h[i] = reinterpret_cast<const T *>(p)[i];
        __builtin_memcpy(&v, h, sizeof(v.q));
    }
}

// Eight values per lane and four lanes per block, U blocks' quarters of a
// thread on the way at once.
template <int TYPE, int U>
__global__ __launch_bounds__(256) void k_mx_quantize(const void *x, uint8_t *codes, uint8_t *scales, MxRows p)
{
    const uint32_t i0 = blockIdx.x * (256 * U) + threadIdx.x;
    Eight<TYPE> v[U];
    uint32_t row[U], c8[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const uint32_t i = i0 + u * 256;
        row[u] = over(i, p.per_row);
        c8[u] = i - row[u] * p.per_row.d;
        load_eight<TYPE>(v[u], x, row[u] * p.ldx + 8 * (int64_t)c8[u], i < p.items ? p.cols - 8 * (int)c8[u] : 0);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        // (a block's four lanes are all there or none: items is a multiple of four)
        uint32_t top = top_of<TYPE>(v[u]);
        top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));
        top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));
        if (i0 + u * 256 >= p.items) continue;
        const uint32_t b = scale_byte<TYPE>(top, p.fit);
        const uint32_t c = b == 255 ? 0u : codes_of<TYPE>(v[u], pow2_of(b));
        __builtin_memcpy(codes + row[u] * p.ldc + 4 * (int64_t)c8[u], &c, 4);
        if ((c8[u] & 3) == 0) scales[row[u] * p.lds + (c8[u] >> 2)] = (uint8_t)b;
    }
}

template <int TYPE, int U>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t *codes, const uint8_t *scales, void *out, MxRows p)
{
    const uint32_t i0 = blockIdx.x * (256 * U) + threadIdx.x;
    uint32_t row[U], c8[U], c[U], b[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const uint32_t i = i0 + u * 256;
        row[u] = over(i, p.per_row);
        c8[u] = i - row[u] * p.per_row.d;
        c[u] = b[u] = 0;
        if (i < p.items) {
            __builtin_memcpy(&c[u], codes + row[u] * p.ldc + 4 * (int64_t)c8[u], 4);
            b[u] = scales[row[u] * p.lds + (c8[u] >> 2)];
        }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int n = i0 + u * 256 < p.items ? p.cols - 8 * (int)c8[u] : 0;
        const float s = b[u] == 255 ? __uint_as_float(0x7fc00000u) : pow2_of(b[u]);
        float f[8];
        f32x2_t t;
        t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 0), f[0] = t.x, f[1] = t.y;
        t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 1), f[2] = t.x, f[3] = t.y;
        t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 2), f[4] = t.x, f[5] = t.y;
        t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 3), f[6] = t.x, f[7] = t.y;
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] *= s;
        constexpr int SZ = TYPE == MOE_F32 ? 4 : 2;
        char *o = reinterpret_cast<char *>(out) + (row[u] * p.ldx + 8 * (int64_t)c8[u]) * SZ;
        if constexpr (TYPE == MOE_F32) {
            if (n >= 8) {
                __builtin_memcpy(o, f, 32);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (j < n) reinterpret_cast<float *>(o)[j] = f[j];
            }
        } else {
            uint16_t h[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                h[j] = TYPE == MOE_F16 ? __builtin_bit_cast(uint16_t, (_Float16)f[j]) : f32_to_bf16_rne(f[j]);
            if (n >= 8) {
                __builtin_memcpy(o, h, 16);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (j < n) reinterpret_cast<uint16_t *>(o)[j] = h[j];
            }
        }
    }
}

// Rows of scales to rows of `pitch` bytes, zeros behind the last one: a thread per 8 bytes.
__global__ __launch_bounds__(256) void k_mx_scale_rows(const uint8_t *s0, const uint8_t *s1, const uint8_t *s2, int64_t ld01,
                                                       int64_t ld2, int rows01, int rows2, int n, int pitch, uint8_t *out)
{
    const int per = pitch / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / per;
    const int at = (int)(i - r * per) * 8, m = s1 ? 2 : 1;
    if (r >= (int64_t)m * rows01 + rows2) return;
    const uint8_t *src = r < rows01 ? s0 + r * ld01 : r < (int64_t)m * rows01 ? s1 + (r - rows01) * ld01 : s2 + (r - (int64_t)m * rows01) * ld2;
    uint64_t v = 0;
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (at + j < n) v |= (uint64_t)src[at + j] << (8 * j);
    *reinterpret_cast<uint64_t *>(out + r * pitch + at) = v;
}

// Rows of one launch: items stay below 2^31.
template <class F>
void by_rows(int64_t rows, int cols, F launch)
{
    const int64_t per = (int64_t)((cols + 31) / 32) * 4, most = (((int64_t)1 << 30) / per);
    for (int64_t r = 0; r < rows; r += most) launch(r, (uint32_t)(std::min(most, rows - r) * per), divisor((uint32_t)per));
}

}  // namespace

hipError_t launch_mx_quantize(const void *x, int type, int64_t ldx, int64_t rows, int cols, uint8_t *codes, int64_t ldc,
                              uint8_t *scales, int64_t lds, int fit, hipStream_t st)
{
    by_rows(rows, cols, [&](int64_t r, uint32_t items, const Divisor &d) {
        const MxRows p = {ldx, ldc, lds, cols, items, d, fit};
        const char *xr = reinterpret_cast<const char *>(x) + r * ldx * (type == MOE_F32 ? 4 : 2);
        uint8_t *c = codes + r * ldc, *s = scales + r * lds;
        if (type == MOE_F32) k_mx_quantize<MOE_F32, 2><<<(items + 511) / 512, 256, 0, st>>>(xr, c, s, p);
        else if (type == MOE_F16) k_mx_quantize<MOE_F16, 2><<<(items + 511) / 512, 256, 0, st>>>(xr, c, s, p);
        else k_mx_quantize<MOE_BF16, 2><<<(items + 511) / 512, 256, 0, st>>>(xr, c, s, p);
    });
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t lds, int64_t rows, int cols,
                                void *out, int type, int64_t ldo, hipStream_t st)
{
    by_rows(rows, cols, [&](int64_t r, uint32_t items, const Divisor &d) {
        const MxRows p = {ldo, ldc, lds, cols, items, d, 0};
        char *o = reinterpret_cast<char *>(out) + r * ldo * (type == MOE_F32 ? 4 : 2);
        const uint8_t *c = codes + r * ldc, *s = scales + r * lds;
        if (type == MOE_F32) k_mx_dequantize<MOE_F32, 2><<<(items + 511) / 512, 256, 0, st>>>(c, s, o, p);
        else if (type == MOE_F16) k_mx_dequantize<MOE_F16, 2><<<(items + 511) / 512, 256, 0, st>>>(c, s, o, p);
        else k_mx_dequantize<MOE_BF16, 2><<<(items + 511) / 512, 256, 0, st>>>(c, s, o, p);
    });
    return hipGetLastError();
}

hipError_t launch_mx_scale_rows(const uint8_t *w, const uint8_t *w_up, int64_t ldw, int n, const uint8_t *x, int64_t ldx, int t,
                                int blocks, int pitch, uint8_t *out, hipStream_t st)
{
    const int64_t threads = ((int64_t)(w_up ? 2 : 1) * n + t) * (pitch / 8);
    k_mx_scale_rows<<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(w, w_up, x, ldw, ldx, n, t, blocks, pitch, out);
    return hipGetLastError();
}

}  // namespace moe
