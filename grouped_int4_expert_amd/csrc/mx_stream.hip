// MXFP4 products for few rows per matrix: the weights are streamed once per
// pass of at most 16 rows (5 f32 rows), or twice as many (two column tiles,
// mx_stream_wide).
//
// A block takes RT row tiles of 16 weight rows and one pass; its waves split
// the inputs into chunks of 512 (wave w takes chunks w, w + WV, ...) and meet
// in LDS at the end.  A chunk is four steps of 128 inputs; in a step a lane
// holds one whole block of a weight row (row lane % 16, block lane / 16: 16
// bytes of codes), and the 16 scale bytes of the row's chunk come in one load
// of which each lane picks its four.  The codes go from memory to the matrix
// cores through registers only:
//  * bf16 parts: dword j of the block is decoded to 8 exact bf16 values and
//    multiplied with inputs 32 b + 8 j .. + 7 of the same block b of x
//    (16x16x32 MFMA; the order of the products inside a sum is free, so both
//    operands may take their inputs in this order).  Products are exact, sums
//    f32.  The three parts of up to five f32 rows lie side by side in the 16
//    columns of one MFMA; of more rows they go into one accumulator in turn.
//  * MXFP4 x: the scaled 16x16x128 MFMA takes both blocks and their scale
//    bytes as they are.
// The x operand is read straight from global memory (a pass's rows stay in
// L2); RT sets how often: what bounds this kernel, beside memory, is the
// number of load instructions.  Columns past the pass read its last row and
// are not stored.
//
// 64 tokens, 128 experts, top-8, 1536 x 4096, bf16: 93 us, 4.6 TB/s of weights;
// a 64-token f32 layer (hidden 4096, inter 1536): gate and up 250-264 us, down
// 128-131 us (3.3 TB/s).  There gate and up take 197 us with every x load at one
// address, 167 us with every weight load at one, and as long with the decoding
// left out: what the f32 passes pay beside the weights is x from L2, three parts
// of each row.  Tried and not faster: eight tiles a wave, waves of a block on
// other rows at the same inputs, x stored in the order of its loads.
#include "mx.h"

namespace qmoe {

constexpr int MXS_WIDE_ROWS = 32;   // up to here blocks take two tiles, above four

// The weights of a block: bases of the matrix (or the pair) and the lane's row
// offsets (one matrix stays below 2 GB).
template <int RT>
struct MxsWeights {
    const uint8_t *q[2], *s[2];
    uint32_t qo[RT], so[RT];
};

// acc[k][i] += tile i of the weights times column tile k < USED of x over the
// wave's chunks (MX: x is MXFP4).
template <bool MX, int RT, int RTM, int WV, int USED, int CT>
__device__ __forceinline__ void mxs_body(f32x4 (&acc)[CT][RT], const MxsWeights<RT> &W,
                                         const uint8_t *const (&xv)[CT],
                                         const uint8_t *const (&xs)[CT], int nb, int w) {
    const int quarter = lane_id() >> 4;
    const int chunks = (nb + 15) / 16;
    for (int c = w; c < chunks; c += WV) {
        u32x4 cq[4][RT];
        uint32_t cs[RT], xc[USED] = {};
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const u32x4 v = mx_scales16(W.s[i / RTM] + W.so[i], 16 * c, nb);
#pragma unroll
            for (int s = 0; s < 4; s++) {
                // blocks past the row re-read its last: finite codes times zeros of x
                const int b = min(16 * c + 4 * s + quarter, nb - 1);
                cq[s][i] = *reinterpret_cast<const u32x4 *>(W.q[i / RTM] + (W.qo[i] + (uint32_t)b * 16));
            }
            cs[i] = mx_pick(v, quarter);
        }
        if constexpr (MX)
#pragma unroll
            for (int k = 0; k < USED; k++) xc[k] = mx_pick(mx_scales16(xs[k], 16 * c, nb), quarter);
#pragma unroll
        for (int s = 0; s < 4; s++) {
            const int b = 16 * c + 4 * s + quarter;
            if constexpr (MX) {
#pragma unroll
                for (int k = 0; k < USED; k++) {
                    u32x4 xq = *reinterpret_cast<const u32x4 *>(xv[k] + (int64_t)min(b, nb - 1) * 16);
                    if (b >= nb) xq = u32x4{0, 0, 0, 0};
                    const i32x8 xb = {(int)xq[0], (int)xq[1], (int)xq[2], (int)xq[3], 0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < RT; i++) {
                        const u32x4 e = cq[s][i];
                        const i32x8 wb = {(int)e[0], (int)e[1], (int)e[2], (int)e[3], 0, 0, 0, 0};
#define MXS_STEP(n)                                                                               \
    if (s == n)                                                                                   \
        acc[k][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wb, xb, acc[k][i], 4, 4, n,  \
                                                                     (int)cs[i], n, (int)xc[k]);
                        MXS_STEP(0) MXS_STEP(1) MXS_STEP(2) MXS_STEP(3)
#undef MXS_STEP
                    }
                }
            } else {
                // x rows hold zeros up to a whole step past their end; the steps
                // after that are not computed
                if (16 * c + 4 * s >= nb) break;
                bf16x8 xf[USED][4];
#pragma unroll
                for (int k = 0; k < USED; k++)
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        xf[k][j] =
                            *reinterpret_cast<const bf16x8 *>(xv[k] + (int64_t)b * 64 + j * 16);
#pragma unroll
                for (int i = 0; i < RT; i++) {
                    const float sc = mx_scale((cs[i] >> (8 * s)) & 255u);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const bf16x8 wf = __builtin_bit_cast(bf16x8, mx_decode8(cq[s][i][j], sc));
#pragma unroll
                        for (int k = 0; k < USED; k++)
                            acc[k][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[k][j],
                                                                                acc[k][i], 0, 0, 0);
                    }
                }
            }
        }
    }
}

// parts: 0, 1, 3; PAIR: tiles RT/2.. are of the second matrix (up) and the
// block writes h = silu(g) * u.
template <int PARTS, int RT, int CT, int WV, bool PAIR>
__global__ void __launch_bounds__(WV * 64) mx_stream_kernel(MxMat W, MxMat U, MxX x, MxGroups g,
                                                            MxOut o) {
    constexpr int RTM = PAIR ? RT / 2 : RT;      // tiles of one matrix
    constexpr int ROWS = mxs_rows(PARTS);        // of a column tile
    __shared__ __attribute__((aligned(16))) float red[WV][CT][RT][64][4];
    const int ncb = ((PAIR ? o.width : W.rows) + 16 * RTM - 1) / (16 * RTM);
    MxTile t;
    if (!mx_find(g, CT * ROWS, ncb, t)) return;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int r16 = lane & 15;
    const int o0 = t.cb * 16 * RTM;

    // this lane's x row of each column tile, and of f32 rows its part
    const int part = PARTS == 3 ? min(r16 / MXS_PACK, 2) : 0;
    const uint8_t *xv[CT], *xs[CT];
#pragma unroll
    for (int k = 0; k < CT; k++) {
        const int col = min(k * ROWS + (PARTS == 3 ? r16 % MXS_PACK : r16), t.rows - 1);
        const int64_t src = max(mx_source(g, x, t.pos0 + col), (int64_t)0);
        xv[k] = x.v + src * x.ld + (int64_t)part * x.width * 2;
        xs[k] = PARTS == 0 ? x.s + src * W.nb : nullptr;
    }

    MxsWeights<RT> wt;
    wt.q[0] = W.q + (int64_t)t.e * W.q_stride;
    wt.s[0] = W.s + (int64_t)t.e * W.s_stride;
    wt.q[1] = PAIR ? U.q + (int64_t)t.e * U.q_stride : nullptr;
    wt.s[1] = PAIR ? U.s + (int64_t)t.e * U.s_stride : nullptr;
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const uint32_t row = (uint32_t)min(o0 + 16 * (i % RTM) + r16, W.rows - 1);
        wt.qo[i] = row * (uint32_t)W.nb * 16;
        wt.so[i] = row * (uint32_t)W.nb;
    }

    f32x4 acc[CT][RT];
#pragma unroll
    for (int k = 0; k < CT; k++)
#pragma unroll
        for (int i = 0; i < RT; i++) acc[k][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (CT == 1 || t.rows > ROWS)
        mxs_body<PARTS == 0, RT, RTM, WV, CT>(acc, wt, xv, xs, W.nb, w);
    else
        mxs_body<PARTS == 0, RT, RTM, WV, 1>(acc, wt, xv, xs, W.nb, w);

#pragma unroll
    for (int k = 0; k < CT; k++)
#pragma unroll
        for (int i = 0; i < RT; i++) *reinterpret_cast<f32x4 *>(red[w][k][i][lane]) = acc[k][i];
    __syncthreads();
    // output (row c of the pass, weight row o0 + r): accumulator r % 4 of lane
    // (r % 16 / 4) * 16 + c of tile r / 16
    for (int idx = threadIdx.x; idx < 16 * RTM * CT * ROWS; idx += WV * 64) {
        const int r = idx % (16 * RTM), c = idx / (16 * RTM);
        if (c >= t.rows) break;
        const int ct = CT == 1 ? 0 : c / ROWS;
        const int ln = ((r & 15) >> 2) * 16 + (c - ct * ROWS), v = r & 3, n = o0 + r;
        float a = 0.f, u = 0.f;
#pragma unroll
        for (int p = 0; p < (PARTS == 3 ? 3 : 1); p++)
#pragma unroll
            for (int k = 0; k < WV; k++) {
                a += red[k][ct][r >> 4][ln + p * MXS_PACK][v];
                if (PAIR) u += red[k][ct][RTM + (r >> 4)][ln + p * MXS_PACK][v];
            }
        const int pos = t.pos0 + c;
        if constexpr (PAIR) {
            if (n >= o.width) continue;
            uint8_t *dst = static_cast<uint8_t *>(o.y) + (int64_t)pos * o.ld;
            const float h = n < W.rows ? silu(a) * u : 0.0f;
            if constexpr (PARTS == 3) {
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

template <int PARTS, int RT, int CT, int WV, bool PAIR>
static hipError_t go(const MxMat &w, const MxMat &up, const MxX &x, const MxGroups &g,
                     const MxOut &out, hipStream_t st) {
    constexpr int RTM = PAIR ? RT / 2 : RT;
    const int64_t ncb = ((PAIR ? out.width : w.rows) + 16 * RTM - 1) / (16 * RTM);
    const dim3 grid(mx_grid(mx_max_tiles(g, CT * mxs_rows(PARTS)) * ncb));
    hipLaunchKernelGGL((mx_stream_kernel<PARTS, RT, CT, WV, PAIR>), grid, dim3(WV * 64), 0, st, w, up, x,
                       g, out);
    return hipGetLastError();
}

// Waves per block.  Calls of few rows (two tiles) split the inputs as far as
// they go, for latency.  Larger ones want several blocks per CU, so that one's
// loads run under another's start and end: four waves (bf16, 64 tokens of a
// 128-expert projection: 8 waves 107 us, 4 waves 89, 2 waves 93, 1 wave 93), two
// for f32 rows, whose passes hold fewer rows (64-token layer: gate+up 4 waves
// 243 us, 2 waves 241; down 3 waves 134, 1 wave 118).
template <int PARTS, int RT, int CT, bool PAIR>
static hipError_t by_width(const MxMat &w, const MxMat &up, const MxX &x, const MxGroups &g,
                           const MxOut &out, hipStream_t st) {
    const int chunks = (w.nb + 15) / 16;
    if constexpr (RT == 4 && PARTS == 3) {
        if (chunks <= 3) return go<PARTS, RT, CT, 1, PAIR>(w, up, x, g, out, st);
        return go<PARTS, RT, CT, 2, PAIR>(w, up, x, g, out, st);
    } else {
        if (chunks == 1) return go<PARTS, RT, CT, 1, PAIR>(w, up, x, g, out, st);
        if (chunks == 2) return go<PARTS, RT, CT, 2, PAIR>(w, up, x, g, out, st);
        if (chunks == 3) return go<PARTS, RT, CT, 3, PAIR>(w, up, x, g, out, st);
        if constexpr (RT == 2)
            if (chunks > 4) return go<PARTS, RT, CT, 8, PAIR>(w, up, x, g, out, st);
        return go<PARTS, RT, CT, 4, PAIR>(w, up, x, g, out, st);
    }
}

template <int PARTS, bool PAIR>
static hipError_t by_rows(const MxMat &w, const MxMat &up, const MxX &x, const MxGroups &g,
                          const MxOut &out, hipStream_t st) {
    if (g.n <= MXS_WIDE_ROWS) return by_width<PARTS, 2, 1, PAIR>(w, up, x, g, out, st);
    if constexpr (!PAIR)
        if (mx_stream_wide(g, PARTS, w.rows, w.nb))
            return by_width<PARTS, 4, 2, false>(w, up, x, g, out, st);
    return by_width<PARTS, 4, 1, PAIR>(w, up, x, g, out, st);
}

hipError_t launch_mx_stream(const MxMat &w, const MxMat &up, const MxX &x, int parts,
                            const MxGroups &g, const MxOut &out, hipStream_t st) {
    if (up.q) return parts == 3 ? by_rows<3, true>(w, up, x, g, out, st)
                                : by_rows<1, true>(w, up, x, g, out, st);
    if (parts == 0) return by_rows<0, false>(w, up, x, g, out, st);
    if (parts == 1) return by_rows<1, false>(w, up, x, g, out, st);
    return by_rows<3, false>(w, up, x, g, out, st);
}

}  // namespace qmoe
