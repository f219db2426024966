// MXFP4 weights times MXFP4 rows, many rows per matrix, on the scaled 4-bit
// matrix instructions: nothing is decoded.
//
// A block of 4 waves owns 16 XF rows of x and 256 weight rows (64 per wave).
// A stage is 128 inputs: in the 16x16x128 MFMA a lane holds one whole block of
// each operand (row lane % 16, block lane / 16) and its scale byte.
//  * x codes: loads write LDS directly, 64 bytes of each row per stage, into a
//    ring of four stages; every wave reads all of them.
//  * Weight codes: straight to registers (only one wave needs them), 64
//    consecutive bytes of a row per load instruction.
//  * Scale bytes of up to 64 blocks (2048 inputs, a panel) of all the tile's
//    rows and weight rows are brought to LDS before the panel's stages.  They
//    are 1/17 of the bytes but, fetched row by row in the loop, they would
//    need more load instructions than the codes.  They lie so that one 32-bit
//    read holds a lane's scale of four consecutive stages (the instruction
//    picks the byte).
#include "mx_tile.h"

namespace qmoe {

constexpr int FP_PANEL = 64;               // blocks per scale panel
constexpr int FP_PITCH = FP_PANEL + 4;     // bytes per row of a panel in LDS
constexpr int FP_WROWS = 256;

// Slot of 16-byte piece `o` (0..3) of row m in a stage (64-byte rows): the 16
// rows of a 128-bit read at one piece fall on 16 different bank quads.
__device__ __forceinline__ int fp_slot(int m, int o) { return o ^ ((m >> 2) & 3); }

// One row's scale bytes b0 .. b0 + 15 (zero past nb) to its panel row: byte
// (block) 4 g + q goes to q * FP_PANEL / 4 + g.
__device__ __forceinline__ void fp_panel16(uint8_t *dst, const uint8_t *src, int b0, int local,
                                           int nb) {
    u32x4 v = {0, 0, 0, 0};
    if (nb % 16 == 0) {
        if (b0 < nb) v = *reinterpret_cast<const u32x4 *>(src + b0);
    } else {
#pragma unroll
        for (int j = 0; j < 16; j++)
            if (b0 + j < nb) v[j / 4] |= (uint32_t)src[b0 + j] << (8 * (j & 3));
    }
#pragma unroll
    for (int q = 0; q < 4; q++) {
        const uint32_t lo = perm_b32(v[1], v[0], 0x0c0c0400u + 0x0101u * q);
        const uint32_t hi = perm_b32(v[3], v[2], 0x0c0c0400u + 0x0101u * q);
        *reinterpret_cast<uint32_t *>(dst + q * (FP_PANEL / 4) + local / 4) = lo | hi << 16;
    }
}

template <int XF>
__global__ void __launch_bounds__(MXT_THREADS, 2) mx_tile_fp4_kernel(MxMat W, MxX x, MxGroups g,
                                                                    MxOut o) {
    constexpr int WF = 4;                    // weight operands (16 rows) per wave
    constexpr int XROWS = 16 * XF;
    constexpr int XL = XF >= 4 ? XF / 4 : 1; // x loads of a wave per stage (16 rows each)
    constexpr int LOADS = XL + WF;
    constexpr int AHEAD = 2;                 // stages in flight beyond the one computed
    static_assert(AHEAD == 2, "the stages' arrays below");
    // one array per stage: reads of a stage then do not wait for loads into another
    __shared__ __attribute__((aligned(1024))) uint8_t sx0[XROWS * 64], sx1[XROWS * 64],
        sx2[XROWS * 64], sx3[XROWS * 64];
    __shared__ __attribute__((aligned(16))) uint8_t panel[(XROWS + FP_WROWS) * FP_PITCH];
    const int nb = W.nb;
    const int ncb = (W.rows + FP_WROWS - 1) / FP_WROWS;
    MxTile t;
    if (!mx_find(g, XROWS, ncb, t)) return;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int r16 = lane & 15, quarter = lane >> 4;
    const int n0 = t.cb * FP_WROWS + 64 * w;

    const int64_t first = g.pairs ? 0 : t.pos0;
    const int64_t nrows = g.pairs ? x.rows : t.rows;
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(x.v + first * x.ld, nrows * x.ld);
    auto source = [&](int m) {
        const int64_t s = mx_source(g, x, t.pos0 + (m < t.rows ? m : 0)) - first;
        return s < 0 ? 0 : s;
    };
    // x load i of wave w fills rows 16 (i + XL w) + lane / 4; lane l fetches the
    // piece that slot l % 4 of its row holds (the swizzle is an involution).
    // With XF = 2 two waves fill a stage and the others repeat their rows.
    uint32_t xoff[XL];
    int piece = 0;
#pragma unroll
    for (int i = 0; i < XL; i++) {
        const int m = (16 * (i + XL * w) + (lane >> 2)) % XROWS;
        piece = fp_slot(m, lane & 3);        // the same for every i (16 rows apart)
        xoff[i] = (uint32_t)(source(m) * x.ld + piece * 16);
    }
    const __amdgpu_buffer_rsrc_t wr =
        make_rsrc(W.q + (int64_t)t.e * W.q_stride, (int64_t)W.rows * nb * 16);
    uint32_t woff[WF];
#pragma unroll
    for (int j = 0; j < WF; j++)
        woff[j] = (uint32_t)(min(n0 + 16 * j + r16, W.rows - 1) * nb * 16 + 16 * quarter);

    f32x4 acc[XF][WF];
#pragma unroll
    for (int i = 0; i < XF; i++)
#pragma unroll
        for (int j = 0; j < WF; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int iters = (nb + 3) / 4;
    u32x4 rq[4][WF];
    uint32_t sw[WF], sc[XF];
    auto issue = [&](int it, int slot, uint8_t *sx) {
        const int gi = min(it, iters - 1);
        // blocks past a row read as code 0 in x; what the weights hold there is
        // finite (their panel scales are 0, which stands for 2^-127)
        const bool out = 4 * gi + piece >= nb;
#pragma unroll
        for (int i = 0; i < XL; i++)
            mxt_load_lds(xr, sx + (i + XL * w) * 1024 % (XROWS * 64),
                         out ? OOB_OFFSET : xoff[i] + gi * 64, 0);
#pragma unroll
        for (int j = 0; j < WF; j++)
            rq[slot][j] = __builtin_amdgcn_raw_buffer_load_b128(wr, woff[j], gi * 64, 0);
    };
    const int xpiece = fp_slot(r16, quarter) * 16;
#define FP_STAGE(s, cur, ahead)                                                                          \
    {                                                                                             \
        __builtin_amdgcn_s_waitcnt(waitcnt_vm((AHEAD - 1) * LOADS));                              \
        __builtin_amdgcn_s_barrier();                                                             \
        issue((s) + AHEAD < 4 ? it + (s) + AHEAD : next + (s) + AHEAD - 4, ((s) + AHEAD) & 3,     \
              ahead);                                                                             \
        if (it + (s) < last) {                                                                    \
            u32x4 xc[XF];                                                                         \
            _Pragma("unroll") for (int i = 0; i < XF; i++) xc[i] =                                \
                *reinterpret_cast<const u32x4 *>(&cur[(16 * i + r16) * 64 + xpiece]);           \
            _Pragma("unroll") for (int i = 0; i < XF; i++) {                                      \
                const i32x8 xb = {(int)xc[i][0], (int)xc[i][1], (int)xc[i][2], (int)xc[i][3],     \
                                  0, 0, 0, 0};                                                    \
                _Pragma("unroll") for (int j = 0; j < WF; j++) {                                  \
                    const u32x4 c = rq[s][j];                                                     \
                    const i32x8 wb = {(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};    \
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(                 \
                        wb, xb, acc[i][j], 4, 4, s, (int)sw[j], s, (int)sc[i]);                   \
                }                                                                                 \
            }                                                                                     \
            __builtin_amdgcn_sched_group_barrier(0x100, XF, 0);                                   \
            __builtin_amdgcn_sched_group_barrier(0x008, XF * WF, 0);                              \
        }                                                                                         \
    }
    // Rows lie a power of two apart at the usual widths, so the same inputs of
    // all rows come from one or two of the L2's 16 channels: blocks that walked
    // the inputs in the same order would all queue there.  Each column block
    // and matrix starts at another quadruple of stages of another panel (the
    // tiles of one matrix in step: they share its weights).
    const int panels = (nb + FP_PANEL - 1) / FP_PANEL, turn = t.cb + t.e;
    for (int p = 0; p < panels; p++) {
        const int p0 = (p + turn) % panels * FP_PANEL;
        const int it0 = p0 / 4, last = min(iters, it0 + FP_PANEL / 4);
        const int quads = (last - it0 + 3) / 4;
        int quad = turn / panels % quads;
        int it = it0 + 4 * quad;
        issue(it, 0, sx0);
        issue(it + 1, 1, sx1);
        const int chunks = (min(nb - p0, FP_PANEL) + 15) / 16;      // of 16 blocks per row
        for (int c = threadIdx.x; c < (XROWS + FP_WROWS) * chunks; c += MXT_THREADS) {
            const int row = c / chunks, b = (c - row * chunks) * 16;
            const uint8_t *src = row < XROWS
                ? x.s + (first + source(row)) * nb
                : W.s + (int64_t)t.e * W.s_stride +
                      (int64_t)min(t.cb * FP_WROWS + row - XROWS, W.rows - 1) * nb;
            fp_panel16(panel + row * FP_PITCH, src, p0 + b, b, nb);
        }
        // the stages in flight: all of them, the compiler may order their loads
        // among each other here
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        __syncthreads();
        for (int k = 0; k < quads; k++) {
            quad = quad + 1 == quads ? 0 : quad + 1;
            const int next = it0 + 4 * quad;
            const int at = quarter * (FP_PANEL / 4) + (it - it0);
#pragma unroll
            for (int j = 0; j < WF; j++)
                sw[j] = *reinterpret_cast<const uint32_t *>(
                    panel + (XROWS + 64 * w + 16 * j + r16) * FP_PITCH + at);
#pragma unroll
            for (int i = 0; i < XF; i++)
                sc[i] = *reinterpret_cast<const uint32_t *>(panel + (16 * i + r16) * FP_PITCH + at);
            FP_STAGE(0, sx0, sx2)
            FP_STAGE(1, sx1, sx3)
            FP_STAGE(2, sx2, sx0)
            FP_STAGE(3, sx3, sx1)
            it = next;
        }
        // no load may still write LDS and no wave read the panel when the next
        // panel (or the end) comes
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        __syncthreads();
    }
#undef FP_STAGE

#pragma unroll
    for (int i = 0; i < XF; i++) {
        const int m = 16 * i + r16;
        if (m >= t.rows) continue;
        const int64_t pos = t.pos0 + m;
        const bool none = mx_source(g, x, (int)pos) < 0;
#pragma unroll
        for (int j = 0; j < WF; j++) {
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; r++) v[r] = none ? 0.0f : acc[i][j][r];
            mxt_put4(o, pos, n0 + 16 * j + 4 * quarter, W.rows, v);
        }
    }
}

template <int XF>
static hipError_t go(const MxMat &w, const MxX &x, const MxGroups &g, const MxOut &out,
                     hipStream_t st) {
    const int64_t ncb = (w.rows + FP_WROWS - 1) / FP_WROWS;
    const dim3 grid(mx_grid(mx_max_tiles(g, 16 * XF) * ncb));
    hipLaunchKernelGGL((mx_tile_fp4_kernel<XF>), grid, dim3(MXT_THREADS), 0, st, w, x, g, out);
    return hipGetLastError();
}

hipError_t launch_mx_tile_fp4(const MxMat &w, const MxX &x, const MxGroups &g, const MxOut &out,
                              hipStream_t st) {
    const int64_t per = (g.n + g.experts - 1) / g.experts;    // rows per group on average
    if (per <= 32) return go<2>(w, x, g, out, st);
    if (per <= 64) return go<4>(w, x, g, out, st);
    return go<8>(w, x, g, out, st);
}

}  // namespace qmoe
