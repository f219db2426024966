// MXFP4 weights times MXFP4 rows, many rows per matrix (see mx_tile.h).
//
// A stage is 256 inputs: four k-steps of 64, each one scaled 32x32x64 MFMA per
// operand pair, which takes a block of each operand per lane (block 8 G + 2 s
// + lane / 32 in step s) and their scale bytes as they are stored; nothing is
// decoded.  The scale bytes of a lane's four blocks of a stage are gathered
// into one register (byte s for step s, picked by the instruction).
#include "mx_tile.h"

namespace qmoe {

// WHOLE: rows are a multiple of 8 blocks, so a stage never passes a row's end
// and a row's 8 scale bytes of a stage are one aligned load; otherwise every
// lane checks its block against the row and fetches its scales by bytes.
template <int TF, bool WHOLE>
__global__ void __launch_bounds__(MXT_THREADS, 2) mx_tile_fp4_kernel(MxMat W, MxX x, MxGroups g,
                                                                    MxOut o) {
    constexpr int WF = MXT_WF, WROWS = 256;
    __shared__ __attribute__((aligned(1024))) uint8_t s0[TF * 4096], s1[TF * 4096];
    const int nb = W.nb;
    const int ncb = (W.rows + WROWS - 1) / WROWS;
    MxTile t;
    if (!mx_find(g, 32 * TF, ncb, t)) return;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int hh = lane >> 5, l32 = lane & 31;
    const int n0 = t.cb * WROWS + 64 * w;

    const int64_t first = g.pairs ? 0 : t.pos0;
    const int64_t nrows = g.pairs ? x.rows : t.rows;
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(x.v + first * x.ld, nrows * x.ld);
    const __amdgpu_buffer_rsrc_t xsr = make_rsrc(x.s + first * nb, nrows * nb);
    uint32_t xoff[TF], xsoff[TF];
    int piece[TF];
#pragma unroll
    for (int i = 0; i < TF; i++) {
        const int m = 32 * i + 8 * w + (lane >> 3);
        piece[i] = mxt_slot(m, lane & 7);
        const int64_t src = mx_source(g, x, t.pos0 + (m < t.rows ? m : 0)) - first;
        xoff[i] = (uint32_t)((src < 0 ? 0 : src) * x.ld + piece[i] * 16);
        const int ms = 32 * i + l32;
        const int64_t ss = mx_source(g, x, t.pos0 + (ms < t.rows ? ms : 0)) - first;
        xsoff[i] = (uint32_t)((ss < 0 ? 0 : ss) * nb);
    }
    __amdgpu_buffer_rsrc_t wr, sr;
    uint32_t woff[WF], soff[WF];
    wr = make_rsrc(W.q + (int64_t)t.e * W.q_stride, (int64_t)W.rows * nb * 16);
    sr = make_rsrc(W.s + (int64_t)t.e * W.s_stride, (int64_t)W.rows * nb);
#pragma unroll
    for (int j = 0; j < WF; j++) {
        const int row = min(n0 + 32 * j + l32, W.rows - 1);
        woff[j] = (uint32_t)(row * nb * 16 + 16 * hh);
        soff[j] = (uint32_t)(row * nb);
    }

    f32x16 acc[TF][WF];
#pragma unroll
    for (int i = 0; i < TF; i++)
#pragma unroll
        for (int j = 0; j < WF; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.f;

    const int iters = (nb + 7) / 8;
    u32x4 rq[2][WF][4];
    u32x2 rw[2][WF], rx[2][TF];      // scale bytes as loaded (WHOLE), or gathered
    // The scale bytes of blocks 8 gi + 2 s + hh, s = 0..3, of the row at `row`.
    auto scales = [&](__amdgpu_buffer_rsrc_t r, uint32_t row, int gi) {
        u32x2 v;
        if constexpr (WHOLE) {
            v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, row, gi * 8, 0));
        } else {
            uint32_t d[4];
#pragma unroll
            for (int s = 0; s < 4; s++) {
                const int b = 8 * gi + 2 * s + hh;
                d[s] = __builtin_amdgcn_raw_buffer_load_b8(r, b < nb ? row + b : OOB_OFFSET, 0, 0);
            }
            v = u32x2{(d[0] & 255) | (d[1] & 255) << 16, (d[2] & 255) | (d[3] & 255) << 16};
            if (hh) v = v << 8;      // where the gather of hh = 1 finds them
        }
        return v;
    };
    auto issue = [&](int it, int slot, uint8_t *buf) {
        const int gi = min(it, iters - 1);
#pragma unroll
        for (int i = 0; i < TF; i++) {
            uint32_t off = xoff[i] + gi * 128;
            if (!WHOLE && 8 * gi + piece[i] >= nb) off = OOB_OFFSET;
            mxt_load_lds(xr, buf + (i * 4 + w) * 1024, off, 0);
        }
#pragma unroll
        for (int j = 0; j < WF; j++) {
#pragma unroll
            for (int s = 0; s < 4; s++) {
                uint32_t off = woff[j] + gi * 128 + 32 * s;
                if (!WHOLE && 8 * gi + 2 * s + hh >= nb) off = OOB_OFFSET;
                rq[slot][j][s] = __builtin_amdgcn_raw_buffer_load_b128(wr, off, 0, 0);
            }
            rw[slot][j] = scales(sr, soff[j], gi);
        }
#pragma unroll
        for (int i = 0; i < TF; i++) rx[slot][i] = scales(xsr, xsoff[i], gi);
    };
    // bytes hh, hh + 2, hh + 4, hh + 6 of the pair
    const uint32_t pick = hh ? 0x07050301u : 0x06040200u;
    auto compute = [&](int slot, const uint8_t *buf) {
        uint32_t sw[WF], sx[TF];
#pragma unroll
        for (int j = 0; j < WF; j++) sw[j] = perm_b32(rw[slot][j][1], rw[slot][j][0], pick);
#pragma unroll
        for (int i = 0; i < TF; i++) sx[i] = perm_b32(rx[slot][i][1], rx[slot][i][0], pick);
#define MXT_STEP(s)                                                                               \
    {                                                                                             \
        i32x8 wb[WF];                                                                             \
        _Pragma("unroll") for (int j = 0; j < WF; j++) {                                          \
            const u32x4 c = rq[slot][j][s];                                                       \
            wb[j] = i32x8{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};                \
        }                                                                                         \
        _Pragma("unroll") for (int i = 0; i < TF; i++) {                                          \
            const u32x4 c =                                                                       \
                *reinterpret_cast<const u32x4 *>(&buf[mxt_off(32 * i + l32, 2 * (s) + hh)]);      \
            const i32x8 xb = {(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};            \
            _Pragma("unroll") for (int j = 0; j < WF; j++) acc[i][j] =                            \
                __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wb[j], xb, acc[i][j], 4, 4, s,    \
                                                                (int)sw[j], s, (int)sx[i]);       \
        }                                                                                         \
    }
        MXT_STEP(0)
        MXT_STEP(1)
        MXT_STEP(2)
        MXT_STEP(3)
#undef MXT_STEP
    };
    // Stage `it` is read while `it + 1` is in flight.
    issue(0, 0, s0);
    __syncthreads();
    for (int it = 0; it < iters; it += 2) {
        issue(it + 1, 1, s1);
        compute(0, s0);
        __syncthreads();
        if (it + 1 >= iters) break;
        issue(it + 2, 0, s0);
        compute(1, s1);
        __syncthreads();
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_s_barrier();
    mxt_store<TF, 1, false>(acc, t, n0, W.rows, g, x, o);
}

template <int TF>
static hipError_t go(const MxMat &w, const MxX &x, const MxGroups &g, const MxOut &out,
                     hipStream_t st) {
    const int64_t ncb = (w.rows + 255) / 256;
    const dim3 grid(mx_grid(mx_max_tiles(g, 32 * TF) * ncb));
    if (w.nb % 8 == 0)
        hipLaunchKernelGGL((mx_tile_fp4_kernel<TF, true>), grid, dim3(MXT_THREADS), 0, st, w, x, g, out);
    else
        hipLaunchKernelGGL((mx_tile_fp4_kernel<TF, false>), grid, dim3(MXT_THREADS), 0, st, w, x, g, out);
    return hipGetLastError();
}

hipError_t launch_mx_tile_fp4(const MxMat &w, const MxX &x, const MxGroups &g, const MxOut &out,
                              hipStream_t st) {
    const int64_t per = (g.n + g.experts - 1) / g.experts;    // rows per group on average
    if (per <= 32) return go<1>(w, x, g, out, st);
    if (per <= 64) return go<2>(w, x, g, out, st);
    return go<4>(w, x, g, out, st);
}

}  // namespace qmoe
