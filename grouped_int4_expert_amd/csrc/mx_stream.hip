// MXFP4 products for few rows per matrix: the weights are streamed once per
// pass of at most 16 rows.
//
// A block takes RT row tiles of 16 weight rows and one pass; its waves split
// the inputs (wave w takes the 128-input steps w, w + WV, ...) and meet in
// LDS at the end.  In a step a lane holds one whole block of a weight row
// (row lane % 16, block lane / 16: 16 bytes of codes and the scale byte), so
// the codes go from memory to the matrix cores through registers only:
//  * bf16 parts: dword j of the block is decoded to 8 exact bf16 values and
//    multiplied with inputs 32 b + 8 j .. + 7 of the same block b of x
//    (16x16x32 MFMA; the order of the products inside a sum is free, so both
//    operands may take their inputs in this order).  Products are exact, sums
//    f32; the three parts of an f32 row go into one accumulator.
//  * MXFP4 x: the scaled 16x16x128 MFMA takes both blocks and their scale
//    bytes as they are.
// The x operand is read straight from global memory (a pass's rows stay in
// L2).  Columns past the pass read its first row and are not stored.
#include "mx.h"

namespace qmoe {

constexpr int MXS_ROWS = 16;   // rows per pass

// parts: 0, 1, 3; PAIR: tiles RT/2.. are of the second matrix (up) and the
// block writes h = silu(g) * u.
template <int PARTS, int RT, int WV, bool PAIR>
__global__ void __launch_bounds__(WV * 64) mx_stream_kernel(MxMat W, MxMat U, MxX x, MxGroups g,
                                                            MxOut o) {
    constexpr int RTM = PAIR ? RT / 2 : RT;      // tiles of one matrix
    constexpr int P = PARTS == 0 ? 1 : PARTS;
    __shared__ __attribute__((aligned(16))) float red[WV][RT][64][4];
    const int ncb = ((PAIR ? o.width : W.rows) + 16 * RTM - 1) / (16 * RTM);
    MxTile t;
    if (!mx_find(g, MXS_ROWS, ncb, t)) return;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int r16 = lane & 15, quarter = lane >> 4;
    const int o0 = t.cb * 16 * RTM;

    // this lane's x row
    const int col = min(r16, t.rows - 1);
    int64_t src = mx_source(g, x, t.pos0 + col);
    const uint8_t *xv = x.v + (src < 0 ? 0 : src) * x.ld;
    const uint8_t *xs = PARTS == 0 ? x.s + (src < 0 ? 0 : src) * W.nb : nullptr;

    const uint8_t *wq[RT], *wsc[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const bool second = PAIR && i >= RTM;
        const MxMat &M = second ? U : W;
        const int row = min(o0 + 16 * (i - (second ? RTM : 0)) + r16, M.rows - 1);
        wq[i] = M.q + (int64_t)t.e * M.q_stride + (int64_t)row * M.nb * 16;
        wsc[i] = M.s + (int64_t)t.e * M.s_stride + (int64_t)row * M.nb;
    }

    f32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int nb = W.nb, steps = (nb + 3) / 4;
    for (int st = w; st < steps; st += WV) {
        const int b = 4 * st + quarter;
        const bool in = b < nb;            // blocks past the row: code 0
        const int bc = in ? b : nb - 1;
        u32x4 cq[RT];
        uint32_t cs[RT];
#pragma unroll
        for (int i = 0; i < RT; i++) {
            cq[i] = *reinterpret_cast<const u32x4 *>(wq[i] + (int64_t)bc * 16);
            cs[i] = wsc[i][bc];
        }
        if constexpr (PARTS == 0) {
            u32x4 xq = *reinterpret_cast<const u32x4 *>(xv + (int64_t)bc * 16);
            const uint32_t xc = xs[bc];
            if (!in) xq = u32x4{0, 0, 0, 0};
            const i32x8 xb = {(int)xq[0], (int)xq[1], (int)xq[2], (int)xq[3], 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < RT; i++) {
                if (!in) cq[i] = u32x4{0, 0, 0, 0};
                const i32x8 wb = {(int)cq[i][0], (int)cq[i][1], (int)cq[i][2], (int)cq[i][3], 0, 0, 0, 0};
                acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    wb, xb, acc[i], 4, 4, 0, in ? (int)cs[i] : 127, 0, in ? (int)xc : 127);
            }
        } else {
            // x rows are padded to whole steps (zeros), so b needs no bound there
            bf16x8 xf[P][4];
#pragma unroll
            for (int p = 0; p < P; p++)
#pragma unroll
                for (int j = 0; j < 4; j++)
                    xf[p][j] = *reinterpret_cast<const bf16x8 *>(xv + (int64_t)p * x.width * 2 +
                                                                 (int64_t)b * 64 + j * 16);
#pragma unroll
            for (int i = 0; i < RT; i++) {
                // a block past the row: finite codes times the zeros of x
                const float sc = in ? mx_scale(cs[i]) : 1.0f;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const bf16x8 wf = __builtin_bit_cast(bf16x8, mx_decode8(cq[i][j], sc));
#pragma unroll
                    for (int p = 0; p < P; p++)
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[p][j], acc[i], 0, 0, 0);
                }
            }
        }
    }

#pragma unroll
    for (int i = 0; i < RT; i++) *reinterpret_cast<f32x4 *>(red[w][i][lane]) = acc[i];
    __syncthreads();
    // output (row c of the pass, weight row o0 + r): accumulator r % 4 of lane
    // (r % 16 / 4) * 16 + c of tile r / 16
    for (int idx = threadIdx.x; idx < 16 * RTM * 16; idx += WV * 64) {
        const int r = idx % (16 * RTM), c = idx / (16 * RTM);
        if (c >= t.rows) break;
        const int ln = ((r & 15) >> 2) * 16 + c, v = r & 3, n = o0 + r;
        float a = 0.f, u = 0.f;
#pragma unroll
        for (int k = 0; k < WV; k++) {
            a += red[k][r >> 4][ln][v];
            if (PAIR) u += red[k][RTM + (r >> 4)][ln][v];
        }
        const int pos = t.pos0 + c;
        if constexpr (PAIR) {
            if (n >= o.width) continue;
            uint8_t *dst = static_cast<uint8_t *>(o.y) + (int64_t)pos * o.ld;
            const float h = n < W.rows ? silu(a) * u : 0.0f;
            if constexpr (P == 3) {
                uint16_t p[3];
                mx_split3(h, p);
#pragma unroll
                for (int k = 0; k < 3; k++) reinterpret_cast<uint16_t *>(dst)[k * o.width + n] = p[k];
            } else {
                reinterpret_cast<uint16_t *>(dst)[n] = mx_bf16(h);
            }
        } else {
            if (n >= W.rows) continue;
            if (o.w) a *= o.w[o.wpairs[pos]];
            else if (mx_source(g, x, pos) < 0) a = 0.0f;
            if (o.type == MX_OUT_F32) static_cast<float *>(o.y)[(int64_t)pos * o.ld + n] = a;
            else static_cast<uint16_t *>(o.y)[(int64_t)pos * o.ld + n] = mx_bf16(a);
        }
    }
}

template <int PARTS, int RT, int WV, bool PAIR>
static hipError_t go(const MxMat &w, const MxMat &up, const MxX &x, const MxGroups &g,
                     const MxOut &out, hipStream_t st) {
    constexpr int RTM = PAIR ? RT / 2 : RT;
    const int64_t ncb = ((PAIR ? out.width : w.rows) + 16 * RTM - 1) / (16 * RTM);
    const dim3 grid(mx_grid(mx_max_tiles(g, MXS_ROWS) * ncb));
    hipLaunchKernelGGL((mx_stream_kernel<PARTS, RT, WV, PAIR>), grid, dim3(WV * 64), 0, st, w, up, x,
                       g, out);
    return hipGetLastError();
}

hipError_t launch_mx_stream(const MxMat &w, const MxMat &up, const MxX &x, int parts,
                            const MxGroups &g, const MxOut &out, hipStream_t st) {
    if (up.q) return parts == 3 ? go<3, 2, 8, true>(w, up, x, g, out, st)
                                : go<1, 2, 8, true>(w, up, x, g, out, st);
    if (parts == 0) return go<0, 2, 4, false>(w, up, x, g, out, st);
    if (parts == 1) return go<1, 2, 4, false>(w, up, x, g, out, st);
    return go<3, 2, 4, false>(w, up, x, g, out, st);
}

}  // namespace qmoe
