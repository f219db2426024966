// MXFP4 rounding: f32 or bf16 rows to codes and scales and back, the bf16
// parts the products take as operands, and the sum over a token's choices.
// All of these move each byte once and are bound by memory (or, for a few
// rows, by the launch: 1.7 us of the GPU's time for one row).  12288 x 4096 f32:
// codes 54 us (4.3 TB/s), back 35 us (6.5 TB/s); 4093 bf16 rows of 1535 at an odd
// stride 6.6 and 5.4 us; the sum over 8 choices of 8192 x 4096 227 us (5.0 TB/s).
#include "mx.h"

namespace qmoe {

// n / d for n < 2^31 by a multiplication: with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1, n / d = (n + (n m >> 32)) >> l.
struct FastDiv {
    uint32_t d, m, l;
    explicit FastDiv(uint32_t div) : d(div), l(0) {
        while ((1ull << l) < div) l++;
        m = (uint32_t)((((1ull << l) - div) << 32) / div + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (n + __umulhi(n, m)) >> l; }
};

constexpr int64_t MX_MAX_ITEMS = (int64_t)1 << 30;   // items of one launch (FastDiv takes n < 2^31)

// Four lanes per block of 32, eight elements each: the block's largest
// magnitude by two exchanges inside a quad, E = exponent of it - 2 (so that
// element lies in [4, 8)), codes by the rounding conversion (nearest, ties to
// the even code, 6 at most).  The exponent comes from the bits: fields 0 .. 2
// and subnormals take the smallest scale 2^-127.  A NaN or infinity makes the
// whole block NaN (scale byte 255).
template <bool F32>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const void *__restrict__ x, int64_t ld,
                                                          int cols, uint32_t items, FastDiv quads,
                                                          uint8_t *__restrict__ q,
                                                          uint8_t *__restrict__ s) {
    // the lanes of a quad share i / 4 and so one block: all four take part or none
    for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < items; i += gridDim.x * 256u) {
        const uint32_t row = quads.div(i), c = (i - row * quads.d) * 8;
        float v[8];
        mx_load8<F32>(x, (int64_t)row * ld + c, cols - (int)c, v);
        uint32_t m = 0;   // the bits of a magnitude order like the value
#pragma unroll
        for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        m = max(m, dpp_u32<DPP_QUAD_SWAP1>(m));
        m = max(m, dpp_u32<DPP_QUAD_SWAP2>(m));
        const uint32_t field = m >> 23;
        uint32_t code = field > 2 ? field - 2 : 0;
        uint32_t d = 0;
        if (field == 255) {
            code = 255;
        } else {
            const float scale = mx_scale(code);
            d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[0], v[1], scale, 0);
            d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[2], v[3], scale, 1);
            d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[4], v[5], scale, 2);
            d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[6], v[7], scale, 3);
        }
        reinterpret_cast<uint32_t *>(q)[i] = d;
        if ((i & 3) == 0) s[i >> 2] = (uint8_t)code;
    }
}

template <bool F32>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t *__restrict__ q,
                                                            const uint8_t *__restrict__ s,
                                                            uint32_t items, FastDiv quads, int cols,
                                                            void *__restrict__ y, int64_t ld) {
    for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < items; i += gridDim.x * 256u) {
        const uint32_t row = quads.div(i), c = (i - row * quads.d) * 8;
        const uint32_t d = reinterpret_cast<const uint32_t *>(q)[i];
        const float scale = mx_scale(s[i >> 2]);
        const int left = cols - (int)c;
        const int64_t at = (int64_t)row * ld + c;
        if (F32) {
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            union { f32x2 p[4]; f32x4 h[2]; float f[8]; } r;
            r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, scale, 0);
            r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, scale, 1);
            r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, scale, 2);
            r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, scale, 3);
            float *o = static_cast<float *>(y) + at;
            if (left >= 8) {
                __builtin_memcpy(o, &r.h[0], 16);
                __builtin_memcpy(o + 4, &r.h[1], 16);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (j < left) o[j] = r.f[j];
            }
        } else {
            const u32x4 r = mx_decode8(d, scale);
            uint16_t *o = static_cast<uint16_t *>(y) + at;
            if (left >= 8) {
                __builtin_memcpy(o, &r, 16);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (j < left) o[j] = (uint16_t)(r[j / 2] >> (16 * (j & 1)));
            }
        }
    }
}

// bf16 parts of x rows, zero-padded to `width` columns (see MxX).
template <bool F32>
__global__ void __launch_bounds__(256) mx_parts_kernel(const void *__restrict__ x, int64_t ld,
                                                       int cols, uint32_t items, FastDiv octets,
                                                       uint16_t *__restrict__ parts, int width) {
    constexpr int P = F32 ? 3 : 1;
    for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < items; i += gridDim.x * 256u) {
        const uint32_t row = octets.div(i), c = (i - row * octets.d) * 8;
        float v[8];
        mx_load8<F32>(x, (int64_t)row * ld + c, cols - (int)c, v);
        uint16_t o[P][8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (F32) {
                uint16_t p[3];
                mx_split3(v[j], p);
#pragma unroll
                for (int a = 0; a < P; a++) o[a][j] = p[a];
            } else {
                o[0][j] = (uint16_t)(__float_as_uint(v[j]) >> 16);
            }
        }
        uint16_t *dst = parts + (int64_t)row * P * width + c;
#pragma unroll
        for (int a = 0; a < P; a++) __builtin_memcpy(__builtin_assume_aligned(dst + a * width, 16), o[a], 16);
    }
}

// out[t] = sum over the token's choices of its rows of y, in pick order.
template <bool F32>
__global__ void __launch_bounds__(256) mx_combine_kernel(const float *__restrict__ y,
                                                         const int32_t *__restrict__ inv, int k,
                                                         int cols, void *__restrict__ out) {
    const int64_t t = blockIdx.y;
    const int c = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= cols) return;
    const int n = min(4, cols - c);
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < k; j++) {
        const int pos = inv[t * k + j];
        if (pos < 0) continue;
        const float *r = y + (int64_t)pos * cols + c;
        if (n == 4) {
            f32x4 v;
            __builtin_memcpy(&v, r, 16);
#pragma unroll
            for (int i = 0; i < 4; i++) a[i] += v[i];
        } else {
            for (int i = 0; i < n; i++) a[i] += r[i];
        }
    }
    for (int i = 0; i < n; i++) {
        if (F32) static_cast<float *>(out)[t * cols + c + i] = a[i];
        else static_cast<uint16_t *>(out)[t * cols + c + i] = mx_bf16(a[i]);
    }
}

// Calls launch(first row, rows, blocks) over row ranges of at most
// MX_MAX_ITEMS items each.
template <typename Launch>
static hipError_t by_rows(int64_t rows, int64_t per_row, Launch launch) {
    const int64_t step = MX_MAX_ITEMS / per_row > 0 ? MX_MAX_ITEMS / per_row : 1;
    for (int64_t r = 0; r < rows; r += step) {
        const int64_t nr = rows - r < step ? rows - r : step;
        int64_t blocks = (nr * per_row + 255) / 256;
        if (blocks > 16384) blocks = 16384;
        launch(r, (uint32_t)(nr * per_row), (unsigned)blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_mx_quantize(const void *x, bool f32, int64_t rows, int cols, int64_t ld,
                              uint8_t *q, uint8_t *s, hipStream_t st) {
    const int64_t nb = mx_blocks(cols);
    const FastDiv quads((uint32_t)(4 * nb));
    return by_rows(rows, 4 * nb, [&](int64_t r, uint32_t items, unsigned blocks) {
        uint8_t *qr = q + r * nb * 16, *sr = s + r * nb;
        if (f32)
            hipLaunchKernelGGL(mx_quantize_kernel<true>, dim3(blocks), dim3(256), 0, st,
                               static_cast<const float *>(x) + r * ld, ld, cols, items, quads, qr, sr);
        else
            hipLaunchKernelGGL(mx_quantize_kernel<false>, dim3(blocks), dim3(256), 0, st,
                               static_cast<const uint16_t *>(x) + r * ld, ld, cols, items, quads, qr, sr);
    });
}

hipError_t launch_mx_dequantize(const uint8_t *q, const uint8_t *s, int64_t rows, int cols, void *y,
                                bool f32, int64_t ld, hipStream_t st) {
    const int64_t nb = mx_blocks(cols);
    const FastDiv quads((uint32_t)(4 * nb));
    return by_rows(rows, 4 * nb, [&](int64_t r, uint32_t items, unsigned blocks) {
        const uint8_t *qr = q + r * nb * 16, *sr = s + r * nb;
        if (f32)
            hipLaunchKernelGGL(mx_dequantize_kernel<true>, dim3(blocks), dim3(256), 0, st, qr, sr,
                               items, quads, cols, static_cast<float *>(y) + r * ld, ld);
        else
            hipLaunchKernelGGL(mx_dequantize_kernel<false>, dim3(blocks), dim3(256), 0, st, qr, sr,
                               items, quads, cols, static_cast<uint16_t *>(y) + r * ld, ld);
    });
}

hipError_t launch_mx_parts(const void *x, bool f32, int64_t rows, int cols, int64_t ld,
                           uint16_t *parts, int width, hipStream_t st) {
    const FastDiv octets((uint32_t)(width / 8));
    return by_rows(rows, width / 8, [&](int64_t r, uint32_t items, unsigned blocks) {
        if (f32)
            hipLaunchKernelGGL(mx_parts_kernel<true>, dim3(blocks), dim3(256), 0, st,
                               static_cast<const float *>(x) + r * ld, ld, cols, items, octets,
                               parts + r * 3 * width, width);
        else
            hipLaunchKernelGGL(mx_parts_kernel<false>, dim3(blocks), dim3(256), 0, st,
                               static_cast<const uint16_t *>(x) + r * ld, ld, cols, items, octets,
                               parts + r * width, width);
    });
}

hipError_t launch_mx_combine(const float *y, const int32_t *inv, int tokens, int k, int cols,
                             void *out, bool f32, hipStream_t st) {
    const int64_t per = 32768;
    for (int64_t t0 = 0; t0 < tokens; t0 += per) {
        const int64_t nt = tokens - t0 < per ? tokens - t0 : per;
        const dim3 grid((unsigned)((cols + 1023) / 1024), (unsigned)nt);
        if (f32)
            hipLaunchKernelGGL(mx_combine_kernel<true>, grid, dim3(256), 0, st, y, inv + t0 * k, k,
                               cols, static_cast<float *>(out) + t0 * cols);
        else
            hipLaunchKernelGGL(mx_combine_kernel<false>, grid, dim3(256), 0, st, y, inv + t0 * k, k,
                               cols, static_cast<uint16_t *>(out) + t0 * cols);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qmoe
