// MXFP4 weights times bf16 parts, many rows per matrix (see mx_tile.h).
//
// A stage is 64 inputs of one part; with three parts (f32 rows) the loop runs
// over the parts of a stage's inputs in turn, so the weights of a stage are
// read from memory once and twice more from the caches.  A lane holds block
// 2 g + lane / 32 of its weight rows; MFMA k-step s multiplies inputs 8 s ..
// 8 s + 7 of both blocks of the stage, decoded to exact bf16 values.
#include "mx_tile.h"

namespace qmoe {

// Descriptors of a wave's weight operands.
struct MxtWeights {
    __amdgpu_buffer_rsrc_t q[MXT_WF], s[MXT_WF];
};

template <int TF, int PARTS, bool PAIR>
__global__ void __launch_bounds__(MXT_THREADS, 2) mx_tile_kernel(MxMat W, MxMat U, MxX x,
                                                                MxGroups g, MxOut o) {
    constexpr int WF = MXT_WF;
    constexpr int WROWS = PAIR ? 128 : 256;      // weight rows of one matrix per block
    constexpr int LOADS = TF + 2 * WF;           // loads of a wave per stage
    constexpr int VALU = (16 + TF * WF - 1) / (TF * WF);   // vector instructions after each MFMA
    __shared__ __attribute__((aligned(1024))) uint8_t s0[TF * 4096], s1[TF * 4096], s2[TF * 4096],
        s3[TF * 4096];
    const int ncb = ((PAIR ? o.width : W.rows) + WROWS - 1) / WROWS;
    MxTile t;
    if (!mx_find(g, 32 * TF, ncb, t)) return;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int hh = lane >> 5, l32 = lane & 31;
    const int n0 = t.cb * WROWS + (PAIR ? 32 : 64) * w;

    // x: without a gather the tile's rows are consecutive and the descriptor
    // starts at the first of them
    const int64_t first = g.pairs ? 0 : t.pos0;
    const int64_t nrows = g.pairs ? x.rows : t.rows;
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(x.v + first * x.ld, nrows * x.ld);
    uint32_t xoff[TF];
#pragma unroll
    for (int i = 0; i < TF; i++) {
        // load i of wave w fills rows 32 i + 8 w + lane / 8; lane l fetches the
        // piece that slot l % 8 of its row holds (the swizzle is an involution)
        const int m = 32 * i + 8 * w + (lane >> 3);
        const int piece = mxt_slot(m, lane & 7);
        const int64_t src = mx_source(g, x, t.pos0 + (m < t.rows ? m : 0)) - first;
        xoff[i] = (uint32_t)((src < 0 ? 0 : src) * x.ld + piece * 16);
    }
    MxtWeights wt;
    uint32_t woff[WF], soff[WF];
#pragma unroll
    for (int j = 0; j < WF; j++) {
        const MxMat &M = PAIR && j == 1 ? U : W;
        const int row = min(n0 + (PAIR ? 0 : 32 * j) + l32, M.rows - 1);
        wt.q[j] = make_rsrc(M.q + (int64_t)t.e * M.q_stride, (int64_t)M.rows * M.nb * 16);
        wt.s[j] = make_rsrc(M.s + (int64_t)t.e * M.s_stride, (int64_t)M.rows * M.nb);
        woff[j] = (uint32_t)(row * M.nb * 16 + 16 * hh);
        soff[j] = (uint32_t)(row * M.nb + hh);
    }

    f32x16 acc[TF][WF];
#pragma unroll
    for (int i = 0; i < TF; i++)
#pragma unroll
        for (int j = 0; j < WF; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.f;

    const int groups = (W.nb + 1) / 2, iters = groups * PARTS;
    // a lane whose block lies past the row multiplies finite codes with x's zeros
    const bool odd_tail = (W.nb & 1) && hh;
    u32x4 rq[4][WF];
    uint32_t rs[4][WF];
    u32x4 xf[2][TF], wf[2][WF];
    float sc[WF];
    // Loads of iteration `it` (clamped to the last) into ring slot `slot`.
    auto issue = [&](int it, int slot, uint8_t *buf) {
        const int ic = min(it, iters - 1);
        const int gi = ic / PARTS, p = ic - gi * PARTS;
        const int xs = gi * 128 + p * x.width * 2;
#pragma unroll
        for (int i = 0; i < TF; i++)
            mxt_load_lds(xr, buf + (i * 4 + w) * 1024, xoff[i], xs);
#pragma unroll
        for (int j = 0; j < WF; j++) {
            rq[slot][j] = __builtin_amdgcn_raw_buffer_load_b128(wt.q[j], woff[j], gi * 32, 0);
            rs[slot][j] = __builtin_amdgcn_raw_buffer_load_b8(wt.s[j], soff[j], gi * 2, 0);
        }
    };
    auto operands = [&](int b, int it, int slot, const uint8_t *buf, int ks) {
        if (ks == 0) {
            const bool pad = it >= iters || (odd_tail && it >= iters - PARTS);
#pragma unroll
            for (int j = 0; j < WF; j++) sc[j] = pad ? 1.0f : mx_scale(rs[slot][j] & 255u);
        }
        const uint32_t keep = it < iters ? ~0u : 0u;   // iterations past the last add zeros
#pragma unroll
        for (int i = 0; i < TF; i++)
            xf[b][i] = *reinterpret_cast<const u32x4 *>(&buf[mxt_off(32 * i + l32, 4 * hh + ks)]);
#pragma unroll
        for (int j = 0; j < WF; j++) wf[b][j] = mx_decode8(rq[slot][j][ks] & keep, sc[j]);
    };
    auto mfmas = [&](int b) {
#pragma unroll
        for (int i = 0; i < TF; i++)
#pragma unroll
            for (int j = 0; j < WF; j++)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, wf[b][j]),
                                                                   __builtin_bit_cast(bf16x8, xf[b][i]),
                                                                   acc[i][j], 0, 0, 0);
    };
    // Iteration `it`: k-steps 0..2 read the next step's operands while their
    // MFMAs run; before step 3, iteration it + 1 is synchronised (this wave's
    // LDS reads are done, its own loads of it + 1 have landed: two newer
    // iterations stay in flight; barrier), the loads of it + 4 go into the
    // stage just read, and step 3 reads the first operands of it + 1.
    auto step = [&](int it, int slot, uint8_t *cur, uint8_t *next) {
#pragma unroll
        for (int ks = 0; ks < 3; ks++) {
            operands((ks + 1) & 1, it, slot, cur, ks + 1);
            mfmas(ks & 1);
            mxt_interleave<TF * WF, TF, VALU>();
        }
        MXT_WAIT_LDS();
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(2 * LOADS));
        __builtin_amdgcn_s_barrier();
        issue(it + 4, slot, cur);
        operands(0, it + 1, (slot + 1) & 3, next, 0);
        mfmas(1);
        mxt_interleave<TF * WF, TF, VALU>();
    };
    issue(0, 0, s0);
    issue(1, 1, s1);
    issue(2, 2, s2);
    // all three: the compiler may order a stage's loads among those of the others here
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_s_barrier();
    issue(3, 3, s3);
    operands(0, 0, 0, s0, 0);
    for (int it = 0; it < iters; it += 4) {
        step(it, 0, s0, s1);
        step(it + 1, 1, s1, s2);
        step(it + 2, 2, s2, s3);
        step(it + 3, 3, s3, s0);
    }
    // no load may still be writing LDS when the block ends
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_s_barrier();
    mxt_store<TF, PARTS, PAIR>(acc, t, n0, W.rows, g, x, o);
}

template <int TF, int PARTS, bool PAIR>
static hipError_t go(const MxMat &w, const MxMat &up, const MxX &x, const MxGroups &g,
                     const MxOut &out, hipStream_t st) {
    constexpr int WROWS = PAIR ? 128 : 256;
    const int64_t ncb = ((PAIR ? out.width : w.rows) + WROWS - 1) / WROWS;
    const dim3 grid(mx_grid(mx_max_tiles(g, 32 * TF) * ncb));
    hipLaunchKernelGGL((mx_tile_kernel<TF, PARTS, PAIR>), grid, dim3(MXT_THREADS), 0, st, w, up, x, g,
                       out);
    return hipGetLastError();
}

template <int PARTS, bool PAIR>
static hipError_t by_rows(const MxMat &w, const MxMat &up, const MxX &x, const MxGroups &g,
                          const MxOut &out, hipStream_t st) {
    const int64_t per = (g.n + g.experts - 1) / g.experts;    // rows per group on average
    if (per <= 32) return go<1, PARTS, PAIR>(w, up, x, g, out, st);
    if (per <= 64) return go<2, PARTS, PAIR>(w, up, x, g, out, st);
    return go<4, PARTS, PAIR>(w, up, x, g, out, st);
}

hipError_t launch_mx_tile(const MxMat &w, const MxMat &up, const MxX &x, int parts,
                          const MxGroups &g, const MxOut &out, hipStream_t st) {
    if (parts == 3)
        return up.q ? by_rows<3, true>(w, up, x, g, out, st) : by_rows<3, false>(w, up, x, g, out, st);
    return up.q ? by_rows<1, true>(w, up, x, g, out, st) : by_rows<1, false>(w, up, x, g, out, st);
}

}  // namespace qmoe
