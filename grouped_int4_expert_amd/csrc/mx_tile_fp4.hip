// MXFP4 weights times MXFP4 rows, many rows per matrix, on the scaled 4-bit
// matrix instructions: nothing is decoded.
//
// A block of 4 waves owns 32 XF rows of x and 256 weight rows (64 per wave).
// A stage is 128 inputs, two 32x32x64 MFMA steps per operand pair; a lane holds
// one whole block of each operand (row lane % 32) and its scale byte: step s
// takes block s in lanes 0..31 and block s + 2 in lanes 32..63.  (16x16x128
// MFMAs reach 5.1-6.8 PFLOP/s in a loop of nothing else, these 8.5-9.3.)
//  * x codes: loads write LDS directly, 64 bytes of each row per stage, into a
//    ring of four stages; every wave reads all of them.
//  * Weight codes: straight to registers (only one wave needs them), 16 rows x
//    64 consecutive bytes per load instruction; two such loads hold 32 rows,
//    and exchanging 16-lane groups between them gives the operands of the two
//    steps.
//  * Scale bytes: 16 of a row at a time (four stages, a quad), the weights'
//    to registers, x's through LDS.
// The pipeline: while the MFMAs of a stage run, its successor's x operands are
// read from LDS and three later stages are in flight (two, with x operands
// read half a stage ahead, where more than 128 rows fill the registers); the
// scale bytes of the next quad are fetched during this one.
//
// 2048 rows times 4096 x 4096: 31 us, 2.2 PFLOP/s; 16384 rows in 128 ragged groups
// times 1536 x 4096: 158 us, 1.3 PFLOP/s, 3.0 TB/s.  Bound by the address path: a
// load instruction takes about 28 cycles of a compute unit for 16 lines and 100
// for the 64 lines of scale bytes, whose rows lie nb bytes apart.
#include "mx_tile.h"

namespace qmoe {

constexpr int FP_WROWS = 256;

// Slot of 16-byte piece `o` (0..3) of row m in a stage (64-byte rows): the 16
// rows of a 128-bit read at one piece fall on 16 different bank quads.
__device__ __forceinline__ int fp_slot(int m, int o) { return o ^ ((m >> 2) & 3); }

// x row (relative to `first`) of tile row m; rows past the tile and rows
// without a row of x read one that exists.
__device__ __forceinline__ int64_t fp_source(const MxGroups &g, const MxX &x, const MxTile &t, int m,
                                             int64_t first) {
    const int64_t s = mx_source(g, x, t.pos0 + (m < t.rows ? m : 0)) - first;
    return s < 0 ? 0 : s;
}

// Scheduling hint for a stage: its loads and LDS reads spread among its MFMAs
// (a wave that issues them together stalls at the full address queue with its
// matrix core idle).
template <int N_MFMA, int N_DS, int N_VM>
__device__ __forceinline__ void fp_interleave() {
#pragma unroll
    for (int t = 0; t < N_MFMA; t++) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (t * N_DS / N_MFMA != (t + 1) * N_DS / N_MFMA) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        if (t * N_VM / N_MFMA != (t + 1) * N_VM / N_MFMA) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
    }
}

// Operands and addresses of a wave.
template <int XF>
struct FpSrc {
    static constexpr int WL = 4;                    // weight loads of a wave per stage (16 rows each)
    static constexpr int XL = XF / 2;               // x loads of a wave per stage (16 rows each)
    __amdgpu_buffer_rsrc_t x, w;
    uint32_t xoff[XL], woff[WL];
    int piece;
    const uint8_t *xs, *ws[MXT_WF];                 // scale rows: thread t's x row, lane's weight rows
    int nb, turn;
};

// The products of the first XC operands of x (32 XC >= the tile's rows).
template <int XF, int XC>
__device__ __forceinline__ void fp_mainloop(f32x16 (&acc)[XF][MXT_WF], const FpSrc<XF> &src,
                                            uint8_t *__restrict__ sx0, uint8_t *__restrict__ sx1,
                                            uint8_t *__restrict__ sx2, uint8_t *__restrict__ sx3,
                                            u32x4 *__restrict__ ss) {
    constexpr int WF = MXT_WF, WL = 4, XL = XC / 2, LOADS = XL + WL;
    const int nb = src.nb;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int l32 = lane & 31, hh = lane >> 5;
#pragma unroll
    for (int i = 0; i < XC; i++)
#pragma unroll
        for (int j = 0; j < WF; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.f;

    const int iters = (nb + 3) / 4, quads = (iters + 3) / 4;
    constexpr bool HALF = XC > 4;           // x operands half a stage ahead
    u32x4 rq[4][WL], xc[HALF ? 1 : 2][2][XC], wc[2][WF];
    u32x4 rws[WF], rxs;
    uint32_t sw[2][WF], sc[2][XC];
    // Loads of stage `it`: blocks past the row read as code 0 in x; the weights
    // re-read the last stage there.
    auto issue = [&](int it, int slot, uint8_t *sx) {
        const int wi = min(it, iters - 1);
        const bool out = 4 * it + src.piece >= nb;
#pragma unroll
        for (int i = 0; i < XL; i++)
            mxt_load_lds(src.x, sx + (4 * i + w) * 1024, out ? OOB_OFFSET : src.xoff[i] + it * 64, 0);
#pragma unroll
        for (int j = 0; j < WL; j++)
            rq[slot][j] = __builtin_amdgcn_raw_buffer_load_b128(src.w, src.woff[j], wi * 64, 0);
    };
    auto load_scales = [&](int it) {
#pragma unroll
        for (int j = 0; j < WF; j++) rws[j] = mx_scales16(src.ws[j], 4 * it, nb);
        rxs = mx_scales16(src.xs, 4 * it, nb);
    };
    auto put_scales = [&](int half) {
        // every thread, rows again where there are fewer than threads: a branch
        // here would let the compiler move MFMAs past it, away from their stage
        ss[half * MXT_THREADS + threadIdx.x] = rxs;
    };
    auto take_scales = [&](int half) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
#pragma unroll
            for (int j = 0; j < WF; j++) sw[h][j] = mx_pick(rws[j], 2 * hh + h);
        }
#pragma unroll
        for (int i = 0; i < XC; i++) {
            const u32x4 v = ss[half * MXT_THREADS + 32 * i + l32];
            sc[0][i] = mx_pick(v, 2 * hh);
            sc[1][i] = mx_pick(v, 2 * hh + 1);
        }
    };
    const int xp[2] = {fp_slot(l32, 2 * hh) * 16, fp_slot(l32, 2 * hh + 1) * 16};
    auto read_x = [&](int b, int h, const uint8_t *sx) {
#pragma unroll
        for (int i = 0; i < XC; i++)
            xc[b][h][i] = *reinterpret_cast<const u32x4 *>(&sx[(32 * i + l32) * 64 + xp[h]]);
    };
    auto swap_w = [&](int s) {
#pragma unroll
        for (int j = 0; j < WF; j++)
#pragma unroll
            for (int v = 0; v < 4; v++) {
                const auto e = __builtin_amdgcn_permlane16_swap(rq[s][2 * j][v], rq[s][2 * j + 1][v],
                                                                false, false);
                wc[0][j][v] = e[0];
                wc[1][j][v] = e[1];
            }
    };
#define FP_MFMAS(s, b, h)                                                                         \
    _Pragma("unroll") for (int i = 0; i < XC; i++) {                                              \
        const u32x4 e = xc[b][h][i];                                                              \
        const i32x8 xb = {(int)e[0], (int)e[1], (int)e[2], (int)e[3], 0, 0, 0, 0};                \
        _Pragma("unroll") for (int j = 0; j < WF; j++) {                                          \
            const u32x4 c = wc[h][j];                                                             \
            const i32x8 wb = {(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};            \
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(                          \
                wb, xb, acc[i][j], 4, 4, s, (int)sw[h][j], s, (int)sc[h][i]);                     \
        }                                                                                         \
    }
    // Stage s of a quad.
    //  * Its x operands are in registers.  Its successor has landed when at most
    //    the loads of + 2 and + 3 are outstanding; after the barrier every wave
    //    holds this stage's operands, so the loads of + 4 may overwrite it.
    //  * HALF: the first half of its operands is in registers.  The successor
    //    has landed when at most the loads of + 2 are outstanding; after the
    //    barrier every wave is through with the stage before, so the loads of
    //    + 3 may overwrite that.
#define FP_STAGE(s, prv, cur, nxt)                                                                \
    {                                                                                             \
        __builtin_amdgcn_sched_barrier(0);       /* a stage's MFMAs stay in it */                 \
        MXT_WAIT_LDS();                                                                           \
        __builtin_amdgcn_s_waitcnt(waitcnt_vm((HALF ? 1 : 2) * LOADS));                           \
        __builtin_amdgcn_s_barrier();                                                             \
        swap_w(s);                                                                                \
        if constexpr (HALF) {                                                                     \
            issue((s) == 0 ? it + 3 : next + (s) - 1, ((s) + 3) & 3, prv);                        \
            read_x(0, 1, cur);                                                                    \
            FP_MFMAS(s, 0, 0)                                                                     \
            __builtin_amdgcn_sched_barrier(0);                                                    \
            read_x(0, 0, nxt);                                                                    \
            FP_MFMAS(s, 0, 1)                                                                     \
        } else {                                                                                  \
            issue(next + (s), s, cur);                                                            \
            read_x(((s) + 1) & 1, 0, nxt);                                                        \
            read_x(((s) + 1) & 1, 1, nxt);                                                        \
            FP_MFMAS(s, (s) & 1, 0)                                                               \
            FP_MFMAS(s, (s) & 1, 1)                                                               \
            fp_interleave<2 * XC * WF, 2 * XC, LOADS>();                                          \
        }                                                                                         \
    }
    // Rows lie a power of two apart at the usual widths, so the same inputs of
    // all rows come from few of the L2's channels: blocks that walked the inputs
    // in the same order would queue there.  Each column block and matrix starts
    // at another quad (the tiles of one matrix in step: they share its weights).
    int at = src.turn % quads;
    auto following = [&]() {
        at = at + 1 == quads ? 0 : at + 1;
        return 4 * at;
    };
    issue(4 * at, 0, sx0);
    issue(4 * at + 1, 1, sx1);
    issue(4 * at + 2, 2, sx2);
    if constexpr (!HALF) issue(4 * at + 3, 3, sx3);
    load_scales(4 * at);
    put_scales(0);
    // all stages in flight: the compiler may order their loads among each other here
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __syncthreads();
    read_x(0, 0, sx0);
    if constexpr (!HALF) read_x(0, 1, sx0);
    for (int k = 0; k < quads; k++) {
        const int it = 4 * at, next = following();
        (void)it;
        take_scales(k & 1);
        load_scales(next);
        FP_STAGE(0, sx3, sx0, sx1)
        FP_STAGE(1, sx0, sx1, sx2)
        FP_STAGE(2, sx1, sx2, sx3)
        put_scales(~k & 1);
        FP_STAGE(3, sx2, sx3, sx0)
    }
#undef FP_STAGE
#undef FP_MFMAS
    // no load may still write LDS when the block ends
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_s_barrier();
}

// Tiles of 32 XF rows.  A tile of XF = 8 computes the operands its rows need,
// in steps of two.
template <int XF>
__global__ void __launch_bounds__(MXT_THREADS, 1) mx_tile_fp4_kernel(MxMat W, MxX x, MxGroups g,
                                                                    MxOut o) {
    constexpr int XROWS = 32 * XF;
    // one array per stage: reads of a stage then do not wait for loads into another
    __shared__ __attribute__((aligned(1024))) uint8_t sx0[XROWS * 64], sx1[XROWS * 64],
        sx2[XROWS * 64], sx3[XROWS * 64];
    __shared__ u32x4 ss[2 * MXT_THREADS];
    const int nb = W.nb;
    const int ncb = (W.rows + FP_WROWS - 1) / FP_WROWS;
    MxTile t;
    if (!mx_find(g, XROWS, ncb, t)) return;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int n0 = t.cb * FP_WROWS + 64 * w;

    FpSrc<XF> src;
    src.nb = nb;
    src.turn = t.cb + t.e;
    const int64_t first = g.pairs ? 0 : t.pos0;
    src.x = make_rsrc(x.v + first * x.ld, (g.pairs ? x.rows : t.rows) * x.ld);
    src.w = make_rsrc(W.q + (int64_t)t.e * W.q_stride, (int64_t)W.rows * nb * 16);
    src.xs = x.s + (first + fp_source(g, x, t, threadIdx.x % XROWS, first)) * nb;
    const uint8_t *ws = W.s + (int64_t)t.e * W.s_stride;
#pragma unroll
    for (int j = 0; j < MXT_WF; j++)
        src.ws[j] = ws + (int64_t)min(n0 + 32 * j + (lane & 31), W.rows - 1) * nb;
    // x load i of wave w fills rows 64 i + 16 w + lane / 4; lane l fetches the
    // piece that slot l % 4 of its row holds (the swizzle is an involution)
    src.piece = fp_slot(lane >> 2, lane & 3);
#pragma unroll
    for (int i = 0; i < FpSrc<XF>::XL; i++)
        src.xoff[i] = (uint32_t)(fp_source(g, x, t, 64 * i + 16 * w + (lane >> 2), first) * x.ld +
                                 src.piece * 16);
#pragma unroll
    for (int j = 0; j < FpSrc<XF>::WL; j++)
        src.woff[j] = (uint32_t)(min(n0 + 16 * j + (lane & 15), W.rows - 1) * nb * 16 + 16 * (lane >> 4));

    f32x16 acc[XF][MXT_WF];
    if constexpr (XF == 8) {
        if (t.rows <= 64) fp_mainloop<XF, 2>(acc, src, sx0, sx1, sx2, sx3, ss);
        else if (t.rows <= 128) fp_mainloop<XF, 4>(acc, src, sx0, sx1, sx2, sx3, ss);
        else if (t.rows <= 192) fp_mainloop<XF, 6>(acc, src, sx0, sx1, sx2, sx3, ss);
        else fp_mainloop<XF, 8>(acc, src, sx0, sx1, sx2, sx3, ss);
    } else {
        fp_mainloop<XF, XF>(acc, src, sx0, sx1, sx2, sx3, ss);
    }
    mxt_store<XF, 1, false>(acc, t, n0, W.rows, g, x, o);
}

template <int XF>
static hipError_t go(const MxMat &w, const MxX &x, const MxGroups &g, const MxOut &out,
                     hipStream_t st) {
    const int64_t ncb = (w.rows + FP_WROWS - 1) / FP_WROWS;
    const dim3 grid(mx_grid(mx_max_tiles(g, 32 * XF) * ncb));
    hipLaunchKernelGGL((mx_tile_fp4_kernel<XF>), grid, dim3(MXT_THREADS), 0, st, w, x, g,
                       out);
    return hipGetLastError();
}

hipError_t launch_mx_tile_fp4(const MxMat &w, const MxX &x, int size, const MxGroups &g,
                              const MxOut &out, hipStream_t st) {
    if (size == 0) return go<2>(w, x, g, out, st);
    if (size == 1) return go<4>(w, x, g, out, st);
    return go<8>(w, x, g, out, st);
}

}  // namespace qmoe
