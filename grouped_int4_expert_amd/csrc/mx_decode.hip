// MXFP4 products of a decode step with a handful of rows: latency counts, so
// the preparation (worklist, bf16 parts of x) and the sum over a token's
// choices run inside the two kernels of a layer call.
//
//  * mx_few_kernel: y = W x, or h = silu(G x) * (U x), for rows that one block
//    can hold.  A block brings its rows of x to LDS as bf16 parts (any type,
//    stride and width; the padding is zero) while its first weights are on
//    their way.  In a layer every (token, choice) pair is a group of its own:
//    an expert that two tokens picked is read twice, the second time mostly
//    from the caches.
//  * mx_few_down_kernel: out[t] = sum_j w_j (D_j h_j) for 16 outputs of a
//    token: each wave takes choices w, w + WV, ... whole, its h parts in LDS of
//    its own, and the waves' sums are added in order (no atomics, no second
//    launch).
// The weights go to the matrix cores as in mx_stream.hip.
//
// One f32 token, 8 of 128 experts 4096 / 1536: gate and up 16 us (53 MB), down 10
// us (27 MB); one row times 4096 x 4096 5 us (8.9 MB).  Calls this short are bound
// by the chain launch, x to LDS, weights, sums, not by the bytes (53 MB at the
// rate of a large copy: 10 us): the scale loads cost 3 us of the 16, the last
// chunks' products and sums 4, and other shapes of the weight loads change nothing.
#include <atomic>

#include "mx.h"

namespace qmoe {

// One chunk (512 inputs) of RT tiles of a wave: codes and scales.
template <int RT>
struct MxfChunk {
    u32x4 q[4][RT];
    uint32_t s[RT];
};

template <int RT>
__device__ __forceinline__ void mxf_load(MxfChunk<RT> &f, const uint8_t *const (&q)[RT],
                                         const uint8_t *const (&s)[RT], int c, int nb) {
    const int quarter = lane_id() >> 4;
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const u32x4 v = mx_scales16(s[i], 16 * c, nb);
#pragma unroll
        for (int t = 0; t < 4; t++) {
            const int b = min(16 * c + 4 * t + quarter, nb - 1);
            f.q[t][i] = *reinterpret_cast<const u32x4 *>(q[i] + (uint32_t)b * 16);
        }
        f.s[i] = mx_pick(v, quarter);
    }
}

// acc[i] += chunk times the x operand whose row starts at `xv` in LDS.
template <int RT>
__device__ __forceinline__ void mxf_mul(f32x4 (&acc)[RT], const MxfChunk<RT> &f, const uint8_t *xv,
                                        int c, int nb) {
    const int quarter = lane_id() >> 4;
#pragma unroll
    for (int t = 0; t < 4; t++) {
        if (16 * c + 4 * t >= nb) break;      // x is zero up to a whole step
        const int b = 16 * c + 4 * t + quarter;
        bf16x8 xf[4];
#pragma unroll
        for (int j = 0; j < 4; j++) xf[j] = *reinterpret_cast<const bf16x8 *>(xv + b * 64 + j * 16);
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const float sc = mx_scale((f.s[i] >> (8 * t)) & 255u);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const bf16x8 wf = __builtin_bit_cast(bf16x8, mx_decode8(f.q[t][i][j], sc));
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[j], acc[i], 0, 0, 0);
            }
        }
    }
}

// Rows of x in LDS: parts behind each other, 16 bytes more than their width
// apart so that the rows of one read fall on different banks.
__host__ __device__ inline int mxf_pitch(int width) { return width * 2 + 16; }

constexpr int MXF_WV = 8;
constexpr int MXF_AHEAD = 3;   // chunks of a row the down kernel has in flight

template <int P, bool PAIR>
__global__ void __launch_bounds__(MXF_WV * 64) mx_few_kernel(MxMat W, MxMat U, MxFew f, MxOut o) {
    constexpr int RT = PAIR ? 2 : 1, RTM = 1, WV = MXF_WV;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    float (*red)[RT][64][4] = reinterpret_cast<float (*)[RT][64][4]>(lds);
    uint8_t *sx = lds + sizeof(float) * WV * RT * 64 * 4;
    const int ncb = ((PAIR ? o.width : W.rows) + 16 * RTM - 1) / (16 * RTM);
    const int item = blockIdx.x / ncb, cb = blockIdx.x - item * ncb;
    int e = 0, row0 = 0, rows = f.rows;
    if (PAIR) {
        e = f.ids[item];
        if (e < 0 || e >= f.experts) return;     // dropped: the down kernel skips it too
        row0 = item / f.k;
        rows = 1;
    }
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int r16 = lane & 15, o0 = cb * 16 * RTM;

    const uint8_t *q[RT], *s[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const MxMat &M = PAIR && i == 1 ? U : W;
        const int row = min(o0 + r16, W.rows - 1);
        q[i] = M.q + (int64_t)e * M.q_stride + (int64_t)row * W.nb * 16;
        s[i] = M.s + (int64_t)e * M.s_stride + (int64_t)row * W.nb;
    }
    const int nb = W.nb, chunks = (nb + 15) / 16;
    MxfChunk<RT> c0;
    if (w < chunks) mxf_load(c0, q, s, w, nb);

    // x rows to LDS, eight values a thread at a time
    const int pitch = mxf_pitch(f.width), octets = f.width / 8;
    for (int i = threadIdx.x; i < rows * octets; i += WV * 64) {
        const int r = i / octets, c = (i - r * octets) * 8;
        float v[8];
        mx_load8<P == 3>(f.x, (int64_t)(row0 + r) * f.ld + c, f.cols - c, v);
        uint16_t p[P][8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if constexpr (P == 3) {
                uint16_t a[3];
                mx_split3(v[j], a);
#pragma unroll
                for (int k = 0; k < 3; k++) p[k][j] = a[k];
            } else {
                p[0][j] = (uint16_t)(__float_as_uint(v[j]) >> 16);
            }
        }
#pragma unroll
        for (int k = 0; k < P; k++)
            __builtin_memcpy(__builtin_assume_aligned(sx + (r * P + k) * pitch + c * 2, 16), p[k], 16);
    }
    __syncthreads();

    const int part = P == 3 ? min(r16 / 5, 2) : 0;
    const int xrow = min(P == 3 ? r16 % 5 : r16, rows - 1);
    const uint8_t *xv = sx + (xrow * P + part) * pitch;
    f32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c = w; c < chunks; c += WV) {
        if (c != w) mxf_load(c0, q, s, c, nb);
        mxf_mul(acc, c0, xv, c, nb);
    }
#pragma unroll
    for (int i = 0; i < RT; i++) *reinterpret_cast<f32x4 *>(red[w][i][lane]) = acc[i];
    __syncthreads();
    for (int idx = threadIdx.x; idx < 16 * RTM * rows; idx += WV * 64) {
        const int r = idx % (16 * RTM), c = idx / (16 * RTM), n = o0 + r;
        const int ln = ((r & 15) >> 2) * 16 + c, v = r & 3;
        float a = 0.f, u = 0.f;
#pragma unroll
        for (int p = 0; p < P; p++)
#pragma unroll
            for (int k = 0; k < WV; k++) {
                a += red[k][r >> 4][ln + 5 * p][v];
                if (PAIR) u += red[k][RT - 1][ln + 5 * p][v];
            }
        if constexpr (PAIR) {
            if (n >= o.width) continue;
            uint16_t *dst = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(o.y) + (int64_t)item * o.ld);
            const float h = n < W.rows ? silu(a) * u : 0.0f;
            if constexpr (P == 3) {
                uint16_t p[3];
                mx_split3(h, p);
#pragma unroll
                for (int k = 0; k < 3; k++) dst[k * o.width + n] = p[k];
            } else {
                dst[n] = mx_bf16(h);
            }
        } else {
            if (n >= W.rows) continue;
            if (o.type == MX_OUT_F32) static_cast<float *>(o.y)[(int64_t)c * o.ld + n] = a;
            else static_cast<uint16_t *>(o.y)[(int64_t)c * o.ld + n] = mx_bf16(a);
        }
    }
}

template <int P>
__global__ void __launch_bounds__(MXF_WV * 64) mx_few_down_kernel(MxMat D, MxFew f,
                                                                  const uint8_t *__restrict__ h,
                                                                  int64_t h_ld, int width,
                                                                  const float *__restrict__ topk_w,
                                                                  void *__restrict__ out) {
    constexpr int WV = MXF_WV;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    float (*red)[64][4] = reinterpret_cast<float (*)[64][4]>(lds);
    const int ncb = (D.rows + 15) / 16;
    const int tok = blockIdx.x / ncb, o0 = (blockIdx.x - tok * ncb) * 16;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int r16 = lane & 15, nb = D.nb, chunks = (nb + 15) / 16;
    const int pitch = mxf_pitch(width), octets = width / 8;
    uint8_t *sx = lds + sizeof(float) * WV * 64 * 4 + w * P * pitch;
    const int row = min(o0 + r16, D.rows - 1);
    const uint8_t *xv = sx + (P == 3 ? min(r16 / 5, 2) : 0) * pitch;

    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int j = w; j < f.k; j += WV) {
        const int pair = tok * f.k + j, e = f.ids[pair];
        if (e < 0 || e >= f.experts) continue;
        const float wj = topk_w[pair];
        const uint8_t *q[1] = {D.q + (int64_t)e * D.q_stride + (int64_t)row * nb * 16};
        const uint8_t *s[1] = {D.s + (int64_t)e * D.s_stride + (int64_t)row * nb};
        MxfChunk<1> f3[MXF_AHEAD];
#pragma unroll
        for (int a = 0; a < MXF_AHEAD; a++) mxf_load(f3[a], q, s, a, nb);
        // this choice's h parts to the wave's LDS
        for (int i = lane; i < P * octets; i += 64) {
            const int p = i / octets, c = i - p * octets;
            const u32x4 v = *reinterpret_cast<const u32x4 *>(h + pair * h_ld + ((int64_t)p * width + c * 8) * 2);
            *reinterpret_cast<u32x4 *>(sx + p * pitch + c * 16) = v;
        }
        __builtin_amdgcn_wave_barrier();
        f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
        for (int c = 0; c < chunks; c += MXF_AHEAD) {
            if (c > 0) {
#pragma unroll
                for (int a = 0; a < MXF_AHEAD; a++) mxf_load(f3[a], q, s, c + a, nb);
            }
#pragma unroll
            for (int a = 0; a < MXF_AHEAD; a++) mxf_mul(acc, f3[a], xv, c + a, nb);
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int v = 0; v < 4; v++) sum[v] += wj * acc[0][v];
    }
    *reinterpret_cast<f32x4 *>(red[w][lane]) = sum;
    __syncthreads();
    if (threadIdx.x < 16) {
        const int r = threadIdx.x, n = o0 + r;
        float a = 0.f;
        for (int k = 0; k < WV; k++)
#pragma unroll
            for (int p = 0; p < P; p++) a += red[k][(r >> 2) * 16 + 5 * p][r & 3];
        if (n < D.rows) {
            const int64_t at = (int64_t)tok * D.rows + n;
            if (P == 3) static_cast<float *>(out)[at] = a;
            else static_cast<uint16_t *>(out)[at] = mx_bf16(a);
        }
    }
}

static int few_lds(int parts, int rows, int width) {
    return (int)sizeof(float) * MXF_WV * 2 * 64 * 4 + rows * parts * mxf_pitch(width);
}
static int few_down_lds(int parts, int width) {
    return (int)sizeof(float) * MXF_WV * 64 * 4 + MXF_WV * parts * mxf_pitch(width);
}

bool mx_few_matmul_fits(int parts, int rows, int width) {
    return rows <= (parts == 3 ? 5 : 16) && few_lds(parts, rows, width) <= MXF_LDS;
}
bool mx_few_layer_fits(int parts, int width, int h_width) {
    return few_lds(parts, 1, width) <= MXF_LDS && few_down_lds(parts, h_width) <= MXF_DOWN_LDS;
}

// A block may have up to 160 KB of LDS; above 64 KB the launch needs the
// kernel's dynamic limit raised, once per device.
constexpr int MXF_MAX_DEVICES = 64;
template <typename K>
static hipError_t allow_lds(K kernel, int lds, int most, std::atomic<bool> (&raised)[MXF_MAX_DEVICES]) {
    if (lds <= 65536) return hipSuccess;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const bool known = dev >= 0 && dev < MXF_MAX_DEVICES;
    if (known && raised[dev].load()) return hipSuccess;
    e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                            hipFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == hipSuccess && known) raised[dev].store(true);
    return e;
}

template <int P, bool PAIR>
static hipError_t go(const MxMat &w, const MxMat &up, const MxFew &f, const MxOut &out,
                     hipStream_t st) {
    static std::atomic<bool> raised[MXF_MAX_DEVICES];
    const int lds = few_lds(P, PAIR ? 1 : f.rows, f.width);
    const hipError_t e = allow_lds(mx_few_kernel<P, PAIR>, lds, MXF_LDS, raised);
    if (e != hipSuccess) return e;
    const int64_t ncb = ((PAIR ? out.width : w.rows) + 15) / 16;
    hipLaunchKernelGGL((mx_few_kernel<P, PAIR>), dim3((unsigned)(ncb * (PAIR ? f.rows : 1))),
                       dim3(MXF_WV * 64), lds, st, w, up, f, out);
    return hipGetLastError();
}

hipError_t launch_mx_few(const MxMat &w, const MxMat &up, int parts, const MxFew &f,
                         const MxOut &out, hipStream_t st) {
    if (up.q) return parts == 3 ? go<3, true>(w, up, f, out, st) : go<1, true>(w, up, f, out, st);
    return parts == 3 ? go<3, false>(w, up, f, out, st) : go<1, false>(w, up, f, out, st);
}

template <int P>
static hipError_t go_down(const MxMat &d, const MxFew &f, const uint8_t *h, int64_t h_ld, int width,
                          const float *topk_w, int tokens, void *out, hipStream_t st) {
    static std::atomic<bool> raised[MXF_MAX_DEVICES];
    const int lds = few_down_lds(P, width);
    const hipError_t e = allow_lds(mx_few_down_kernel<P>, lds, MXF_DOWN_LDS, raised);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((d.rows + 15) / 16 * (int64_t)tokens));
    hipLaunchKernelGGL((mx_few_down_kernel<P>), grid, dim3(MXF_WV * 64), lds, st, d, f, h, h_ld, width,
                       topk_w, out);
    return hipGetLastError();
}

hipError_t launch_mx_few_down(const MxMat &d, int parts, const MxFew &f, const uint8_t *h,
                              int64_t h_ld, int width, const float *topk_w, int tokens, void *out,
                              hipStream_t st) {
    return parts == 3 ? go_down<3>(d, f, h, h_ld, width, topk_w, tokens, out, st)
                      : go_down<1>(d, f, h, h_ld, width, topk_w, tokens, out, st);
}

}  // namespace qmoe
