// MXFP4 products for many rows per matrix on the matrix cores: the pieces
// that the bf16 kernel (mx_tile.hip) and the MXFP4 x MXFP4 kernel
// (mx_tile_fp4.hip) share.
//
// A block of 4 waves owns a tile of 32 TF rows of x and 256 weight rows (64
// per wave: two MFMA operands of 32 rows; with a gate / up pair 32 of each).
// The weights are the first MFMA operand, so a lane ends with four
// consecutive outputs of one row of y and stores them at once.
//
// One stage holds 128 bytes of each x row of the tile (64 bf16 inputs, or 256
// MXFP4 inputs): loads write LDS directly, 16 bytes a lane, into a ring of four
// or eight stages.  Weights go to registers: a lane holds whole blocks of its
// weight row, so one 16-byte load feeds 32 inputs and LDS carries x only.
#pragma once

#include "mx.h"

namespace qmoe {

constexpr int MXT_THREADS = 256;
constexpr int MXT_WF = 2;        // weight operands (32 rows) per wave

// Slot of 16-byte piece `o` (0..7) of row m in a stage (128-byte rows): 128-bit
// LDS reads are served 16 lanes at a time over 64 banks; lanes on 16
// consecutive rows at one piece then hit 16 different bank quads.
__device__ __forceinline__ int mxt_slot(int m, int o) { return o ^ (m & 7) ^ ((m >> 3) & 1); }
__device__ __forceinline__ int mxt_off(int m, int o) { return m * 128 + mxt_slot(m, o) * 16; }

// s_waitcnt for LDS (lgkmcnt 0) with the other counters left alone.
#define MXT_WAIT_LDS() __builtin_amdgcn_s_waitcnt(0xc07f)

// 16 bytes a lane from global memory straight into LDS: lane l's go to
// lds + 16 l.
__device__ __forceinline__ void mxt_load_lds(__amdgpu_buffer_rsrc_t r, uint8_t *lds, uint32_t off,
                                             int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, QMOE_LDS(lds), 16, off, soff, 0, 0);
}

// Scheduling hint for a k-step: n_mfma MFMAs, each followed by one LDS read
// (while any remain) and up to `valu` vector instructions.
template <int N_MFMA, int N_DS, int VALU>
__device__ __forceinline__ void mxt_interleave() {
#pragma unroll
    for (int t = 0; t < N_MFMA; t++) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (t < N_DS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    }
}

// Four consecutive outputs n .. n + 3 (below `rows`) of row `pos` of y.
__device__ __forceinline__ void mxt_put4(const MxOut &o, int64_t pos, int n, int rows,
                                         const float v[4]) {
    const int64_t at = pos * o.ld + n;
    if (o.type == MX_OUT_F32 && o.vec) {
        if (n < rows) __builtin_memcpy(__builtin_assume_aligned(static_cast<float *>(o.y) + at, 16), v, 16);
        return;
    }
#pragma unroll
    for (int r = 0; r < 4; r++) {
        if (n + r >= rows) continue;
        if (o.type == MX_OUT_F32) static_cast<float *>(o.y)[at + r] = v[r];
        else static_cast<uint16_t *>(o.y)[at + r] = mx_bf16(v[r]);
    }
}

// 16-bit results: the two lanes that share a row of y exchange, so that each
// holds eight consecutive outputs of it and stores 16 bytes: of outputs 16 p ..
// 16 p + 15 lane / 32 = 0 the lower eight, 1 the upper.  `a` and `b` are a lane's
// four at 16 p + 4 (lane / 32) and at 16 p + 8 + 4 (lane / 32).
__device__ __forceinline__ u32x4 mxt_eight(const uint16_t a[4], const uint16_t b[4]) {
    u32x2 u, v;
    __builtin_memcpy(&u, a, 8);
    __builtin_memcpy(&v, b, 8);
    const auto lo = __builtin_amdgcn_permlane32_swap(u[0], v[0], false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(u[1], v[1], false, false);
    return u32x4{lo[0], hi[0], lo[1], hi[1]};
}

// Writes the accumulators of a wave.  acc[i][j][4 q + r]: x row 32 i +
// lane % 32 of the tile, weight row 8 q + 4 (lane / 32) + r of operand j.
template <int TF, int PARTS, bool PAIR>
__device__ __forceinline__ void mxt_store(const f32x16 (&acc)[TF][MXT_WF], const MxTile &t, int n0,
                                          int rows_w, const MxGroups &g, const MxX &x,
                                          const MxOut &o) {
    const int lane = lane_id(), hh = lane >> 5;
#pragma unroll
    for (int i = 0; i < TF; i++) {
        const int m = 32 * i + (lane & 31);
        if (m >= t.rows) continue;
        const int64_t pos = t.pos0 + m;
        if constexpr (PAIR) {
            // operand 0: gate rows n0 .., operand 1: the same rows of up
            uint16_t *dst = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(o.y) + pos * o.ld);
#pragma unroll
            for (int p2 = 0; p2 < 2; p2++) {
                uint16_t p[PARTS][2][4];
#pragma unroll
                for (int d = 0; d < 2; d++)
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        const int v = 8 * p2 + 4 * d + r;
                        const float a = acc[i][0][v], u = acc[i][1][v];
                        // the padding of a part is zero
                        const bool in = n0 + 16 * p2 + 8 * d + 4 * hh + r < rows_w;
                        if constexpr (PARTS == 3) {
                            uint16_t s[3];
                            mx_split3(in ? silu(a) * u : 0.0f, s);
#pragma unroll
                            for (int k = 0; k < 3; k++) p[k][d][r] = s[k];
                        } else {
                            // h is rounded to bf16, x's own type
                            p[0][d][r] = mx_bf16(in ? silu_fast(a) * u : 0.0f);
                        }
                    }
                const int n = n0 + 16 * p2 + 8 * hh;      // o.width is a multiple of 8
#pragma unroll
                for (int k = 0; k < PARTS; k++) {
                    const u32x4 e = mxt_eight(p[k][0], p[k][1]);
                    if (n < o.width) *reinterpret_cast<u32x4 *>(dst + k * o.width + n) = e;
                }
            }
        } else {
            float f = 1.0f;
            bool none = false;
            if (o.w) f = o.w[o.wpairs[pos]];
            else none = mx_source(g, x, (int)pos) < 0;
#pragma unroll
            for (int j = 0; j < MXT_WF; j++) {
                if (o.type == MX_OUT_BF16 && o.vec) {
#pragma unroll
                    for (int p2 = 0; p2 < 2; p2++) {
                        uint16_t p[2][4];
#pragma unroll
                        for (int d = 0; d < 2; d++)
#pragma unroll
                            for (int r = 0; r < 4; r++)
                                p[d][r] = mx_bf16(none ? 0.0f : acc[i][j][8 * p2 + 4 * d + r] * f);
                        const u32x4 e = mxt_eight(p[0], p[1]);
                        const int n = n0 + 32 * j + 16 * p2 + 8 * hh;
                        if (n < rows_w) *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(o.y) + pos * o.ld + n) = e;
                    }
                    continue;
                }
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; r++) v[r] = none ? 0.0f : acc[i][j][4 * q + r] * f;
                    mxt_put4(o, pos, n0 + 32 * j + 8 * q + 4 * hh, rows_w, v);
                }
            }
        }
    }
}

}  // namespace qmoe
