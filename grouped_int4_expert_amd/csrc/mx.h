// MXFP4 (microscaled 4-bit floats): operand descriptions and device helpers
// shared by the mx_*.hip kernels.
//
// Format.  A row of K values is ceil(K / 32) blocks; a block is 16 bytes of
// codes (element 2j in the low nibble of byte j) and one scale byte c that
// stands for 2^(c - 127), c = 255 for NaN.  A code is sign, 2 exponent bits
// and 1 mantissa bit: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6.
#pragma once

#include "common.h"

namespace qmoe {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int MX_BLOCK = 32;

__host__ __device__ inline int mx_blocks(int64_t cols) { return (int)((cols + MX_BLOCK - 1) / MX_BLOCK); }

// A stack of MXFP4 matrices: codes [rows][nb][16], scales [rows][nb].
struct MxMat {
    const uint8_t *q, *s;
    int64_t q_stride, s_stride;   // bytes between experts
    int rows, nb;
};

// Rows of the other operand.  bf16 parts: `parts` (1, or 3 that sum to an f32
// value exactly) rows of `width` bf16 behind each other, width a multiple of
// 128, zero past the row's own columns; ld = bytes per row of all parts.
// MXFP4: ld = nb * 16 bytes of codes, scales in s with nb bytes per row.
struct MxX {
    const uint8_t *v;
    const uint8_t *s;
    int64_t ld;
    int64_t rows;
    int width;
};

// Row groups.  offsets == nullptr: one group of n rows (matrix 0).  Else rows
// offsets[e] .. offsets[e + 1] of the output belong to matrix e; row r reads
// x row pairs[r] / k, or r itself without pairs.
struct MxGroups {
    const int32_t *offsets;
    const int32_t *pairs;
    int k, experts, n;
};

// Rows of f32 or bf16 as a caller holds them (any stride, any alignment of the
// element), with the routing of a layer call (ids [tokens][k]; nullptr: one
// matrix).  rows: rows of x, or pairs with ids.
struct MxFew {
    const void *x;
    int64_t ld;         // elements
    int cols, width;    // width: cols padded to 128
    const int32_t *ids;
    int k, experts, rows;
};

// What a product writes.
enum { MX_OUT_F32 = 0, MX_OUT_BF16 = 1 };
struct MxOut {
    void *y;            // rows of y (f32 or bf16), or the parts of h
    int64_t ld;         // elements between rows of y; bytes between rows of h
    int type;           // MX_OUT_*
    const float *w;     // row r is multiplied by w[wpairs[r]] (nullptr: no weights)
    const int32_t *wpairs;
    int width;          // h: padded width of a part
    int vec;            // rows of y consist of whole, aligned 16-byte pieces
};

__device__ __forceinline__ float mx_scale(uint32_t c) {
    uint32_t b = c << 23;
    b = c == 0 ? 0x00400000u : b;      // 2^-127 is subnormal
    b = c == 255 ? 0x7fc00000u : b;
    return __uint_as_float(b);
}

// Eight codes (a dword) times a power of two as bf16, exact: a code has two
// significant bits and bf16 the exponent range of the scales (results below
// 2^-126 are subnormal and kept).
__device__ __forceinline__ u32x4 mx_decode8(uint32_t d, float scale) {
    union { bf16x2 p[4]; u32x4 v; } r;
    r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0);
    r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1);
    r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2);
    r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3);
    return r.v;
}

// Scale bytes b0 .. b0 + 15 of a row of nb, 0 past its end (which stands for
// 2^-127; what it multiplies there is 0 in x).
__device__ __forceinline__ u32x4 mx_scales16(const uint8_t *row, int b0, int nb) {
    u32x4 v;
    if (b0 + 16 <= nb) {
        __builtin_memcpy(&v, row + b0, 16);
    } else {
        uint64_t part[2] = {0, 0};
#pragma unroll 1
        for (int j = 0; b0 + j < nb; j++) {
            const uint64_t c = (uint64_t)row[b0 + j] << (8 * (j & 7));
            if (j < 8) part[0] |= c;
            else part[1] |= c;
        }
        __builtin_memcpy(&v, part, 16);
    }
    return v;
}

// Byte q of each dword: the scales of block q of four consecutive stages, the
// byte of stage s at place s.
__device__ __forceinline__ uint32_t mx_pick(u32x4 v, int q) {
    const uint32_t sel = 0x0c0c0400u + 0x0101u * q;
    return perm_b32(v[1], v[0], sel) | perm_b32(v[3], v[2], sel) << 16;
}

// f32 as three bf16 parts, exact: each part takes the top 8 significant bits
// that are left (truncation), 3 x 8 = 24.  A NaN or infinity goes into the
// first part alone (inf - inf would make a NaN of it).  Bits below 2^-133
// (bf16's smallest subnormal) are lost.
__device__ __forceinline__ void mx_split3(float x, uint16_t p[3]) {
    const uint32_t b = __float_as_uint(x);
    const bool fin = (b & 0x7f800000u) != 0x7f800000u;
    // a NaN whose bits all lie in the lower half stays a NaN
    const uint32_t top = (b & 0xffff0000u) | (!fin && (b & 0x007fffffu) ? 0x00400000u : 0u);
    const float r1 = fin ? x - __uint_as_float(top) : 0.0f;
    const uint32_t m = __float_as_uint(r1) & 0xffff0000u;
    const float r2 = r1 - __uint_as_float(m);
    p[0] = (uint16_t)(top >> 16);
    p[1] = (uint16_t)(m >> 16);
    p[2] = (uint16_t)(__float_as_uint(r2) >> 16);
}

// Eight elements of a row from column c on as f32, zero past `cols`.  Rows
// may start at any element: a load at less than its size's alignment is one
// instruction on this GPU all the same.
template <bool F32>
__device__ __forceinline__ void mx_load8(const void *x, int64_t at, int left, float v[8]) {
    if (left >= 8) {
        if (F32) {
            f32x4 a, b;
            const float *p = static_cast<const float *>(x) + at;
            __builtin_memcpy(&a, p, 16);
            __builtin_memcpy(&b, p + 4, 16);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[i] = a[i];
                v[4 + i] = b[i];
            }
        } else {
            u32x4 a;
            __builtin_memcpy(&a, static_cast<const uint16_t *>(x) + at, 16);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[2 * i] = __uint_as_float(a[i] << 16);
                v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        v[i] = 0.0f;
        if (i < left)
            v[i] = F32 ? static_cast<const float *>(x)[at + i]
                       : __uint_as_float((uint32_t) static_cast<const uint16_t *>(x)[at + i] << 16);
    }
}

__device__ __forceinline__ uint16_t mx_bf16(float x) {
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}

struct MxTile {
    int e, pos0, rows, cb;
};

// Inclusive sum over the lanes of a wave (DPP: within rows of 16 lanes, then
// the row totals passed on).
__device__ __forceinline__ int mx_wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31
    return v;
}

// The work item of this block: a tile of at most bm rows of one group and a
// column block.  Every wave of the block runs it (no LDS): lane l of round r
// holds the offset of expert 64 r + l, all loads in flight at once, and a scan
// over the lanes gives each expert's first tile.  Offsets are clamped to
// [0, n], so no value of theirs leads outside the output.  The GPU hands linear
// block ids to its 8 XCDs round-robin and each XCD has an L2 of its own; each
// is given one contiguous run of the items.
__device__ __forceinline__ bool mx_item(int total, int ncb, int64_t &item, int &tile) {
    const int64_t items = (int64_t)total * ncb;
    const int64_t per_xcd = (items + 7) / 8;
    item = (int64_t)(blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per_xcd || item >= items) return false;
    tile = (int)((uint64_t)item >> 32 ? item / ncb : (uint32_t)item / (uint32_t)ncb);
    return true;
}

// Item `local` of a group of `rows` rows: the tiles of one column block side by
// side, so that what they share of the weights is read from memory once.
__device__ __forceinline__ void mx_place(MxTile &t, int first, int rows, int bm, int64_t local) {
    const int tiles = (rows + bm - 1) / bm;
    t.cb = (int)((uint64_t)local >> 32 ? local / tiles : (uint32_t)local / (uint32_t)tiles);
    const int at = (int)(local - (int64_t)t.cb * tiles) * bm;
    t.pos0 = first + at;
    t.rows = min(bm, rows - at);
}

template <int ROUNDS>
__device__ __forceinline__ bool mx_find_in(const MxGroups &g, int bm, int ncb, MxTile &t) {
    const int lane = lane_id();
    int o[ROUNDS + 1], last[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; r++)
        o[r] = g.offsets[min(QMOE_WAVE * r + lane, g.experts)];
    o[ROUNDS] = g.offsets[min(QMOE_WAVE * ROUNDS, g.experts)];
    int total = 0;
#pragma unroll
    for (int r = 0; r < ROUNDS; r++) {
        o[r] = min(max(o[r], 0), g.n);
        int next = __shfl_down(o[r], 1, QMOE_WAVE);
        const int after = min(max(__builtin_amdgcn_readfirstlane(o[r + 1]), 0), g.n);
        if (lane == QMOE_WAVE - 1) next = after;
        // inclusive number of tiles up to this expert
        last[r] = total + mx_wave_scan((max(next - o[r], 0) + bm - 1) / bm);
        total = __builtin_amdgcn_readlane(last[r], QMOE_WAVE - 1);
    }
    int64_t item;
    int tile;
    if (!mx_item(total, ncb, item, tile)) return false;
    // the first expert whose tiles end behind `tile`
#pragma unroll
    for (int r = 0; r < ROUNDS; r++) {
        const uint64_t behind = __ballot(last[r] > tile);
        if (behind == 0) continue;
        const int l = __ffsll((unsigned long long)behind) - 1;
        const int first = __builtin_amdgcn_readlane(o[r], l);
        const int end = l == QMOE_WAVE - 1 ? min(max(__builtin_amdgcn_readfirstlane(o[r + 1]), 0), g.n)
                                           : __builtin_amdgcn_readlane(o[r], l + 1 & 63);
        const int before = __builtin_amdgcn_readlane(last[r], l) - (max(end - first, 0) + bm - 1) / bm;
        t.e = QMOE_WAVE * r + l;
        mx_place(t, first, end - first, bm, item - (int64_t)before * ncb);
        return true;
    }
    return false;
}

__device__ __forceinline__ bool mx_find(const MxGroups &g, int bm, int ncb, MxTile &t) {
    if (!g.offsets) {
        int64_t item;
        int tile;
        if (!mx_item((g.n + bm - 1) / bm, ncb, item, tile)) return false;
        t.e = 0;
        mx_place(t, 0, g.n, bm, item);
        return true;
    }
    if (g.experts <= QMOE_WAVE) return mx_find_in<1>(g, bm, ncb, t);
    if (g.experts <= 2 * QMOE_WAVE) return mx_find_in<2>(g, bm, ncb, t);
    if (g.experts <= 4 * QMOE_WAVE) return mx_find_in<4>(g, bm, ncb, t);
    return mx_find_in<16>(g, bm, ncb, t);
}

// x row of output row `pos`; -1 where its pair names no row of x.
__device__ __forceinline__ int64_t mx_source(const MxGroups &g, const MxX &x, int pos) {
    if (!g.pairs) return pos;
    const int p = g.pairs[pos];
    const int r = p / g.k;
    return p < 0 || r >= x.rows ? -1 : r;
}

inline unsigned mx_grid(int64_t items) { return (unsigned)(((items + 7) / 8) * 8); }
// Upper bound of the tiles of bm rows that n rows in `experts` groups make.
inline int64_t mx_max_tiles(const MxGroups &g, int bm) {
    const int64_t t = (g.n + (int64_t)bm - 1) / bm;
    return g.offsets ? t + (g.n < g.experts ? g.n : g.experts) : t;
}

// Rows whose parts share the 16 columns of an MFMA in mx_stream.hip.
constexpr int MXS_PACK = 5;
constexpr int mxs_rows(int parts) { return parts == 3 ? MXS_PACK : 16; }

// Passes of two column tiles read and decode the weights half as often, but
// make half as many blocks, of fewer waves.  They pay from 2048 inputs on, if
// their blocks still are one per compute unit: 4096 x 4096, one and two tiles
// (us), f32 64 rows 38 and 32, 256 rows 114 and 103; bf16 64 rows 12 and 17, 128
// rows 20 and 17, 256 rows 35 and 28; MXFP4 256 rows 26 and 18; of 1024 inputs
// bf16 256 rows 12 and 12.5.  Layers, whose groups often hold fewer rows than one
// tile, lose (64 f32 tokens 374 and 391).
inline bool mx_stream_wide(const MxGroups &g, int parts, int rows, int nb) {
    const int64_t groups = g.offsets ? (g.n < g.experts ? g.n : g.experts) : 1;
    const int64_t passes = groups * (g.n / groups / (2 * mxs_rows(parts)));
    return nb >= 64 && passes * (rows / 64) >= 256;
}

// ---- launchers (host side; shapes are validated by the C ABI layer) -------

hipError_t launch_mx_quantize(const void *x, bool f32, int64_t rows, int cols, int64_t ld,
                              uint8_t *q, uint8_t *s, hipStream_t st);
hipError_t launch_mx_dequantize(const uint8_t *q, const uint8_t *s, int64_t rows, int cols, void *y,
                                bool f32, int64_t ld, hipStream_t st);
// x [rows][cols] -> bf16 parts (3 for f32, 1 for bf16) of `width` columns.
hipError_t launch_mx_parts(const void *x, bool f32, int64_t rows, int cols, int64_t ld,
                           uint16_t *parts, int width, hipStream_t st);
// Products.  parts: 0 (x is MXFP4), 1 or 3.  up.q != nullptr: h parts of
// silu(W x) * (up x) instead of y (out.y, out.ld, out.width).
hipError_t launch_mx_stream(const MxMat &w, const MxMat &up, const MxX &x, int parts,
                            const MxGroups &g, const MxOut &out, hipStream_t st);
// A decode step (mx_decode.hip): a matrix times rows that fit one block's LDS
// (up.q == nullptr), h parts of every pair, and the weighted sum of a token's
// down projections.
constexpr int MXF_LDS = 80 * 1024;          // two blocks per CU
constexpr int MXF_DOWN_LDS = 152 * 1024;
bool mx_few_matmul_fits(int parts, int rows, int width);
bool mx_few_layer_fits(int parts, int width, int h_width);
hipError_t launch_mx_few(const MxMat &w, const MxMat &up, int parts, const MxFew &f,
                         const MxOut &out, hipStream_t st);
hipError_t launch_mx_few_down(const MxMat &d, int parts, const MxFew &f, const uint8_t *h,
                              int64_t h_ld, int width, const float *topk_w, int tokens, void *out,
                              hipStream_t st);
// size: 0 .. 2, tiles of 32, 64, 128 rows (128 not of three parts).
hipError_t launch_mx_tile(const MxMat &w, const MxMat &up, const MxX &x, int parts, int size,
                          const MxGroups &g, const MxOut &out, hipStream_t st);
// size: 0 .. 2, tiles of 64, 128, 256 rows.
hipError_t launch_mx_tile_fp4(const MxMat &w, const MxX &x, int size, const MxGroups &g,
                              const MxOut &out, hipStream_t st);
// out[t] = sum_j y[inv[t * k + j]] in pick order (f32 sums), as f32 or bf16.
hipError_t launch_mx_combine(const float *y, const int32_t *inv, int tokens, int k, int cols,
                             void *out, bool f32, hipStream_t st);

}  // namespace qmoe
