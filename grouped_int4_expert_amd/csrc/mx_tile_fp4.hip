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
    __shared__ __attribute__((aligned(1024))) uint8_t sx[4][XROWS * 64];
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
    auto issue = [&](int it, int slot) {
        const int gi = min(it, iters - 1);
        // blocks past a row read as code 0 in x; what the weights hold there is
        // finite (their panel scales are 0, which stands for 2^-127)
        const bool out = 4 * gi + piece >= nb;
#pragma unroll
        for (int i = 0; i < XL; i++)
            mxt_load_lds(xr, sx[slot] + (i + XL * w) * 1024 % (XROWS * 64), out ? OOB_OFFSET : xoff[i] + gi * 64, 0);
#pragma unroll
        for (int j = 0; j < WF; j++)
            rq[slot][j] = __builtin_amdgcn_raw_buffer_load_b128(wr, woff[j], gi * 64, 0);
    };
    const int xpiece = fp_slot(r16, quarter) * 16;
#define FP_STAGE(it, s)                                                                           \
    {                                                                                             \
        __builtin_amdgcn_s_waitcnt(waitcnt_vm((AHEAD - 1) * LOADS));                              \
        __builtin_amdgcn_s_barrier();                                                             \
        issue((it) + AHEAD, ((s) + AHEAD) & 3);                                                   \
        if ((it) < last) {                                                                        \
            i32x8 wb[WF];                                                                         \
            _Pragma("unroll") for (int j = 0; j < WF; j++) {                                      \
                const u32x4 c = rq[s][j];                                                         \
                wb[j] = i32x8{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};            \
            }                                                                                     \
            _Pragma("unroll") for (int i = 0; i < XF; i++) {                                      \
                const u32x4 c =                                                                   \
                    *reinterpret_cast<const u32x4 *>(&sx[s][(16 * i + r16) * 64 + xpiece]);       \
                const i32x8 xb = {(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};        \
                _Pragma("unroll") for (int j = 0; j < WF; j++) acc[i][j] =                        \
                    __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(                             \
                        wb[j], xb, acc[i][j], 4, 4, s, (int)sw[j], s, (int)sc[i]);                \
            }                                                                                     \
        }                                                                                         \
    }
    for (int p0 = 0; p0 < nb; p0 += FP_PANEL) {
        const int chunks = (min(nb - p0, FP_PANEL) + 15) / 16;      // of 16 blocks per row
        for (int c = threadIdx.x; c < (XROWS + FP_WROWS) * chunks; c += MXT_THREADS) {
            const int row = c / chunks, b = (c - row * chunks) * 16;
            const uint8_t *src = row < XROWS
                ? x.s + (first + source(row)) * nb
                : W.s + (int64_t)t.e * W.s_stride +
                      (int64_t)min(t.cb * FP_WROWS + row - XROWS, W.rows - 1) * nb;
            fp_panel16(panel + row * FP_PITCH, src, p0 + b, b, nb);
        }
        const int it0 = p0 / 4, last = min(iters, it0 + FP_PANEL / 4);
#pragma unroll
        for (int a = 0; a < AHEAD; a++) issue(it0 + a, a);
        // the stages in flight: all of them, the compiler may order their loads
        // among each other here
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        __syncthreads();
        for (int it = it0; it < last; it += 4) {
            const int at = quarter * (FP_PANEL / 4) + (it - it0);
#pragma unroll
            for (int j = 0; j < WF; j++)
                sw[j] = *reinterpret_cast<const uint32_t *>(
                    panel + (XROWS + 64 * w + 16 * j + r16) * FP_PITCH + at);
#pragma unroll
            for (int i = 0; i < XF; i++)
                sc[i] = *reinterpret_cast<const uint32_t *>(panel + (16 * i + r16) * FP_PITCH + at);
            FP_STAGE(it, 0)
            FP_STAGE(it + 1, 1)
            FP_STAGE(it + 2, 2)
            FP_STAGE(it + 3, 3)
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
