// MXFP4 weights times bf16 parts, many rows per matrix (see mx_tile.h).
//
// A stage is 64 inputs of one part, a unit 128 inputs: two stages, of each part
// in turn.  A lane holds block 2 g + lane / 32 of its weight rows in stage g;
// MFMA k-step s multiplies inputs 8 s .. 8 s + 7 of both blocks, decoded to
// exact bf16 values.  Codes are loaded a unit at a time, 16 rows x 64
// consecutive bytes per instruction (half as many cache lines as 32 rows x 32
// bytes), and exchanging 16-lane groups between two such loads gives the
// operands of the unit's two stages; with three parts the codes stay in
// registers for all of them.  Scale bytes come eight of a row at a time, two
// units ahead.
//
// 8192 tokens, 128 experts 4096 / 1536, top-8, bf16 (128-row tiles): gate and up
// 1.41 ms (1.17 PFLOP/s), down 0.89 ms (0.92 PFLOP/s, 0.3 ms of it the f32 rows for
// the sum).  Gate and up without any load take 1.15 ms, their MFMAs alone would
// take 0.69: the decoding and the LDS reads issued beside the MFMAs bound this
// kernel, more so with smaller tiles, which decode the same codes more often.
#include "mx_tile.h"

namespace qmoe {

// Descriptors of a wave's weight operands.
struct MxtWeights {
    __amdgpu_buffer_rsrc_t q[MXT_WF];
};

// Scale bytes b0 .. b0 + 7 of a row of nb, 0 past its end, moved down by `hh`
// bytes: block 2 g + hh of each pair at byte 2 g.
__device__ __forceinline__ u32x2 mxt_scales8(const uint8_t *row, int b0, int nb, int hh) {
    uint64_t v = 0;
    if (b0 + 8 <= nb) {
        __builtin_memcpy(&v, row + b0, 8);
    } else {
#pragma unroll 1
        for (int j = 0; b0 + j < nb; j++) v |= (uint64_t)row[b0 + j] << (8 * j);
    }
    v >>= 8 * hh;
    return u32x2{(uint32_t)v, (uint32_t)(v >> 32)};
}

template <int TF, int PARTS, bool PAIR>
__global__ void __launch_bounds__(MXT_THREADS, TF == 1 ? 3 : 2) mx_tile_kernel(MxMat W, MxMat U, MxX x,
                                                                MxGroups g, MxOut o) {
    constexpr int WF = MXT_WF;
    constexpr int WROWS = PAIR ? 128 : 256;      // weight rows of one matrix per block
    constexpr int SPU = 2 * PARTS;               // stages per unit
    // Stages in the ring: four; a 32-row tile of three parts, whose stages are the
    // shortest, needs eight to cover the way to memory (512 rows, 4096 x 4096, 69 ->
    // 61 us; with registers for three blocks of a unit a 1024-token layer 1065 -> 1029).
    constexpr int DEPTH = TF == 1 && PARTS == 3 ? 8 : 4;
    // loads a wave surely issued after those of a stage and before it waits for it
    constexpr int NEWER = (DEPTH - 2) * TF + (PARTS == 1 ? 2 * WF : 0);
    constexpr int VALU = (16 + TF * WF - 1) / (TF * WF);   // vector instructions after each MFMA
    // one array per stage: reads of a stage then do not wait for loads into another
    __shared__ __attribute__((aligned(1024))) uint8_t s0[TF * 4096], s1[TF * 4096], s2[TF * 4096],
        s3[TF * 4096];
    constexpr int MORE = DEPTH == 8 ? TF * 4096 : 16;
    __shared__ __attribute__((aligned(1024))) uint8_t s4[MORE], s5[MORE], s6[MORE], s7[MORE];
    const int ncb = ((PAIR ? o.width : W.rows) + WROWS - 1) / WROWS;
    MxTile t;
    if (!mx_find(g, 32 * TF, ncb, t)) return;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int hh = lane >> 5, l32 = lane & 31, nb = W.nb;
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
    uint32_t woff[WF][2];
    const uint8_t *srow[WF];
    // 16-lane group c of a code load holds block {0, 2, 1, 3}[c] of its rows: the
    // exchange then leaves blocks 0 and 1 in one register, 2 and 3 in the other
    const int wblock = (lane >> 5) | ((lane >> 4) & 1) << 1;
#pragma unroll
    for (int j = 0; j < WF; j++) {
        const MxMat &M = PAIR && j == 1 ? U : W;
        const int row = n0 + (PAIR ? 0 : 32 * j);
        wt.q[j] = make_rsrc(M.q + (int64_t)t.e * M.q_stride, (int64_t)M.rows * nb * 16);
#pragma unroll
        for (int a = 0; a < 2; a++)
            woff[j][a] = (uint32_t)(min(row + 16 * a + (lane & 15), M.rows - 1) * nb * 16 + 16 * wblock);
        srow[j] = M.s + (int64_t)t.e * M.s_stride + (int64_t)min(row + l32, M.rows - 1) * nb;
    }

    f32x16 acc[TF][WF];
#pragma unroll
    for (int i = 0; i < TF; i++)
#pragma unroll
        for (int j = 0; j < WF; j++)
#pragma unroll
            for (int v = 0; v < 16; v++) acc[i][j][v] = 0.f;

    const int groups = (nb + 1) / 2, units = (nb + 3) / 4;
    u32x4 rq[2][WF][2], xf[2][TF], wf[2][WF];     // rq: by unit, weight operand, then stage of the unit
    u32x2 raw[WF], sv[WF];
    float sc[WF];
    // Stage s (0 .. 2 SPU - 1) of the two units from u0 on: its inputs of x.
    // Stages past the last read as zeros (their weights are finite: any codes,
    // and scale bytes of 0, which stand for 2^-127).
    auto issue_x = [&](int u0, int s, uint8_t *buf) {
        const int u = u0 + s / SPU, p = s % SPU / 2, half = s & 1;
        const bool in = 2 * u + half < groups;
        // row offsets are below 2^31: with the top bit set they are past the end
        // whatever else the range check counts in
        const uint32_t off = in ? 0 : OOB_OFFSET;
        const int so = in ? u * 256 + half * 128 + p * x.width * 2 : 0;
#pragma unroll
        for (int i = 0; i < TF; i++) mxt_load_lds(xr, buf + (i * 4 + w) * 1024, xoff[i] | off, so);
    };
    auto issue_w = [&](int u, int slot) {
#pragma unroll
        for (int j = 0; j < WF; j++)
#pragma unroll
            for (int a = 0; a < 2; a++)
                rq[slot][j][a] = __builtin_amdgcn_raw_buffer_load_b128(wt.q[j], woff[j][a], min(u, units - 1) * 64, 0);
    };
    auto load_scales = [&](int u) {
#pragma unroll
        for (int j = 0; j < WF; j++) raw[j] = mxt_scales8(srow[j], 4 * u, nb, hh);
    };
    // Operands of k-step ks of stage s into buffer b.
    auto operands = [&](int b, int s, const uint8_t *buf, int ks) {
        const int slot = s / SPU, half = s & 1;
        if (ks == 0) {
            if (s % SPU == 0) {
#pragma unroll
                for (int j = 0; j < WF; j++)
#pragma unroll
                    for (int v = 0; v < 4; v++) {
                        const auto e = __builtin_amdgcn_permlane16_swap(rq[slot][j][0][v],
                                                                        rq[slot][j][1][v], false, false);
                        rq[slot][j][0][v] = e[0];
                        rq[slot][j][1][v] = e[1];
                    }
            }
#pragma unroll
            for (int j = 0; j < WF; j++) sc[j] = mx_scale((sv[j][slot] >> (16 * half)) & 255u);
        }
#pragma unroll
        for (int i = 0; i < TF; i++)
            xf[b][i] = *reinterpret_cast<const u32x4 *>(&buf[mxt_off(32 * i + l32, 4 * hh + ks)]);
#pragma unroll
        for (int j = 0; j < WF; j++) wf[b][j] = mx_decode8(rq[slot][j][half][ks], sc[j]);
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
    // Stage s of the loop body: k-steps 0..2 read the next step's operands while
    // their MFMAs run; before step 3 the next stage is synchronised (this wave's
    // LDS reads are done; its own loads of the next stage have landed when only
    // those issued after them are outstanding; barrier), the loads of stage
    // s + DEPTH go into the stage just read, and step 3 reads the next stage's
    // first operands.  A unit's last stage frees its codes' registers for the
    // unit after the next.
    auto stage = [&](int u0, int s, uint8_t *cur, uint8_t *next) {
#pragma unroll
        for (int ks = 0; ks < 3; ks++) {
            operands((ks + 1) & 1, s, cur, ks + 1);
            mfmas(ks & 1);
            mxt_interleave<TF * WF, TF, VALU>();
        }
        MXT_WAIT_LDS();
        __builtin_amdgcn_s_waitcnt(waitcnt_vm(NEWER));
        __builtin_amdgcn_s_barrier();
        issue_x(u0, s + DEPTH, cur);
        if (s % SPU == SPU - 1) issue_w(u0 + s / SPU + 2, s / SPU);
        if (s == 2 * SPU - 1) {
#pragma unroll
            for (int j = 0; j < WF; j++) sv[j] = raw[j];
        }
        operands(0, (s + 1) % (2 * SPU), next, 0);
        mfmas(1);
        mxt_interleave<TF * WF, TF, VALU>();
    };
    uint8_t *const ring[8] = {s0, s1, s2, s3, s4, s5, s6, s7};
#pragma unroll
    for (int s = 0; s < DEPTH; s++) issue_x(0, s, ring[s]);
    issue_w(0, 0);
    issue_w(1, 1);
    load_scales(0);
#pragma unroll
    for (int j = 0; j < WF; j++) sv[j] = raw[j];
    // all four: the compiler may order a stage's loads among those of the others here
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_s_barrier();
    operands(0, 0, s0, 0);
    for (int u0 = 0; u0 < units; u0 += DEPTH / 2) {
        load_scales(u0 + 2);
#pragma unroll
        for (int s = 0; s < 2 * SPU; s++) stage(u0, s, ring[s % DEPTH], ring[(s + 1) % DEPTH]);
        if constexpr (DEPTH == 8) {
            // two more units: 2 SPU is 4 modulo 8
            load_scales(u0 + 4);
#pragma unroll
            for (int s = 0; s < 2 * SPU; s++) stage(u0 + 2, s, ring[(s + 4) % 8], ring[(s + 5) % 8]);
        }
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
static hipError_t by_size(const MxMat &w, const MxMat &up, const MxX &x, int size,
                          const MxGroups &g, const MxOut &out, hipStream_t st) {
    if (size == 0) return go<1, PARTS, PAIR>(w, up, x, g, out, st);
    // 128 rows of three parts do not fit the registers: 16384 rows in 128 groups,
    // 1024 inputs, 194 us against 162 with 64-row tiles
    if constexpr (PARTS == 1)
        if (size == 2) return go<4, PARTS, PAIR>(w, up, x, g, out, st);
    return go<2, PARTS, PAIR>(w, up, x, g, out, st);
}

hipError_t launch_mx_tile(const MxMat &w, const MxMat &up, const MxX &x, int parts,
                          int size, const MxGroups &g, const MxOut &out, hipStream_t st) {
    if (parts == 3)
        return up.q ? by_size<3, true>(w, up, x, size, g, out, st)
                    : by_size<3, false>(w, up, x, size, g, out, st);
    return up.q ? by_size<1, true>(w, up, x, size, g, out, st)
                : by_size<1, false>(w, up, x, size, g, out, st);
}

}  // namespace qmoe
