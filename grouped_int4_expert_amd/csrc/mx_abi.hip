// C ABI of the MXFP4 entry points: checks, workspace layout and launch
// sequencing.  As in abi.hip every check runs before the first HIP call.
#include <algorithm>

#include "abi_util.h"
#include "launch.h"
#include "mx.h"

using namespace qmoe;

namespace {

constexpr int64_t LIM31 = (int64_t)1 << 31;

// The kernels address one matrix through buffer descriptors whose lanes past
// a row's end use an offset of 2^31.
int check_mxmat(const qmoe_mxmat *m, int experts) {
    if (!m) return QMOE_ERR_NULL;
    if (m->struct_size != sizeof(qmoe_mxmat)) return QMOE_ERR_ABI;
    if (m->rows <= 0 || m->cols <= 0 || experts < 1 || experts > MAX_EXPERTS) return QMOE_ERR_SHAPE;
    const int64_t nb = mx_blocks(m->cols), qb = m->rows * nb * 16, sb = m->rows * nb;
    if (qb >= LIM31) return QMOE_ERR_UNSUPPORTED;
    if (!m->q || !m->s) return QMOE_ERR_NULL;
    if (!aligned16(m->q) || !aligned16(m->s)) return QMOE_ERR_ALIGN;
    if (experts > 1) {
        if (m->q_expert_stride < qb || m->s_expert_stride < sb) return QMOE_ERR_SHAPE;
        if (m->q_expert_stride % 16 != 0) return QMOE_ERR_ALIGN;
        // 2^50: no stack is larger, and the sizes below stay within 64 bits
        if (m->q_expert_stride >> 40 || m->s_expert_stride >> 40) return QMOE_ERR_SHAPE;
    }
    return QMOE_OK;
}

// Bytes from the first to the last one a stack of `experts` matrices uses.
int64_t span_q(const qmoe_mxmat *m, int experts) {
    return (experts - 1) * m->q_expert_stride + (int64_t)m->rows * mx_blocks(m->cols) * 16;
}
int64_t span_s(const qmoe_mxmat *m, int experts) {
    return (experts - 1) * m->s_expert_stride + (int64_t)m->rows * mx_blocks(m->cols);
}
bool overlaps_mat(const void *p, int64_t n, const qmoe_mxmat *m, int experts) {
    return overlap(p, n, m->q, span_q(m, experts)) || overlap(p, n, m->s, span_s(m, experts));
}

MxMat to_mx(const qmoe_mxmat *m) {
    return MxMat{m->q, m->s, m->q_expert_stride, m->s_expert_stride, m->rows, mx_blocks(m->cols)};
}

int pad128(int64_t cols) { return (int)((cols + 127) / 128 * 128); }
int parts_of(int dtype) { return dtype == QMOE_F32 ? 3 : 1; }
int elem_bytes(int dtype) { return dtype == QMOE_F32 ? 4 : 2; }
bool float_type(int dtype) { return dtype == QMOE_F32 || dtype == QMOE_BF16; }

// bf16 rows of whole 128-input steps that start at 16-byte boundaries are the
// products' operand as they are; any other f32 or bf16 rows are first turned
// into parts in the workspace.
bool direct_rows(int dtype, int64_t cols, int64_t ld) {
    return dtype == QMOE_BF16 && cols % 128 == 0 && ld % 8 == 0;
}
int64_t parts_bytes(int dtype, int64_t rows, int64_t cols, int64_t ld) {
    if (dtype == QMOE_MXFP4 || direct_rows(dtype, cols, ld)) return 0;
    return align256(rows * parts_of(dtype) * pad128(cols) * 2);
}

// Bytes a strided [rows][cols] array spans.
int64_t span(int64_t rows, int64_t cols, int64_t ld, int bytes) {
    return rows > 0 ? ((rows - 1) * ld + cols) * bytes : 0;
}

// The operand x of a product, with its parts written first where it needs
// them.
hipError_t operand(int dtype, const void *x, const uint8_t *x_s, int64_t rows, int cols, int64_t ld,
                   void *ws, MxX &o, hipStream_t st) {
    o = MxX{};
    o.rows = rows;
    if (dtype == QMOE_MXFP4) {
        o.v = static_cast<const uint8_t *>(x);
        o.s = x_s;
        o.ld = (int64_t)mx_blocks(cols) * 16;
        return hipSuccess;
    }
    o.width = pad128(cols);
    if (direct_rows(dtype, cols, ld)) {
        o.v = static_cast<const uint8_t *>(x);
        o.ld = ld * 2;
        return hipSuccess;
    }
    o.v = static_cast<const uint8_t *>(ws);
    o.ld = (int64_t)parts_of(dtype) * o.width * 2;
    return launch_mx_parts(x, dtype == QMOE_F32, rows, cols, ld, static_cast<uint16_t *>(ws), o.width,
                           st);
}

// Which kernel a product takes: passes that stream the weights (mx_stream.hip;
// -1), or tiles (mx_tile.hip, mx_tile_fp4.hip) of size 0, 1 or 2.  The stream's
// time grows with rows x weights (every group's last pass half empty).  A tile's
// grows with the inputs alone while every compute unit has one; each further
// tile of a unit adds about as much again, less for small tiles, which hide one
// another's waits.  Both have to read the weights, which the stream does faster.
// Measured: one matrix of 4096 x 4096 (us; tiles by the rows of one):
//   rows            64   128   256   512  1024  2048  4096
//   f32  stream     32    55   102   188   419
//        tiles 32   54    56    58    61   100   191   371
//              64   84    87    90    91   100   184   354
//             128        181   182   184   188   228   401      (spills; not built)
//   bf16 stream     12    17    28    53   130
//        tiles 32   31    31    32    36    51    97   189
//              64   36    36    36    40    43    72   143
//             128         50    51    54    56    63   125
//   MXFP4 stream   9.1    12    18    34    91
//        tiles 64   25    24    25    26    27    49    93
//             128         27    28    29    31    35    65
//             256               36    37    40    43    57
// the same at 1024 inputs: f32 512 rows 24, 31, 55, bf16 12, 14, 20.  Groups,
// bf16: 8 of 128 rows, 2048 x 4096, tiles 37, 41, 55; 128 of 64, 1536 x 4096, 184,
// 145, 181; 128 of 128, 1536 x 1024, 83, 67, 59.  Ragged MXFP4 groups of more than
// 64 rows take 256-row tiles, which compute 64, 128 or 192 rows where no more are
// left.  A layer of 128 experts 4096 / 1536, top-8: f32 stream 374 us, tiles 409 at
// 64 tokens, 480 and 430 at 96; bf16 310 and 338 at 96, 412 and 380 at 200; tiles of
// 32, 64, 128 rows: 1024 tokens f32 1045, 1105, 1752, bf16 647, 561, 614; 2048
// tokens f32 1852, 1837, 2437, bf16 1098, 901, 848.
struct TileCost {
    int rows;
    double start, first, more;   // ns; per input of a unit's first tile, of a further one
};
int tile_size(const MxGroups &g, int parts, bool pair, int64_t rows, int64_t cols) {
    static const TileCost cost[3][3] = {
        {{64, 6300, 4.8, 5.4}, {128, 9400, 5.8, 7.3}, {256, 11600, 7.9, 7.9}},
        {{32, 4200, 7.5, 5.4}, {64, 5400, 8.8, 8.3}, {128, 7700, 12.3, 13.3}},
        {{32, 4800, 12.5, 10.0}, {64, 5500, 20.6, 18.0}, {}}};
    // ns per row, weight row and input: passes of one column tile, of two
    static const double stream[2][3] = {{5.3e-6, 7.5e-6, 24.4e-6}, {3.4e-6, 5.5e-6, 21.5e-6}};
    static const double bytes_per_ns[3] = {4100, 3600, 3100};    // weights through the tiles; streamed:
    const double streamed_per_ns = 4600, stream_start = 4000;
    const int type = parts == 3 ? 2 : parts;
    const int64_t groups = g.offsets ? (g.n < g.experts ? g.n : g.experts) : 1;
    int best = 0;
    double tiles_ns = 0;
    for (int i = 0; i < 3; i++) {
        const TileCost &c = cost[type][i];
        if (c.rows == 0) continue;
        // ragged groups: half a tile of each is empty
        const int64_t tiles = g.offsets ? std::max(groups, g.n / c.rows + groups / 2)
                                        : (g.n + c.rows - 1) / c.rows;
        const int64_t blocks = tiles * ((rows + 255) / 256);
        const double turns = std::max((double)blocks / 256, 1.0);     // tiles of a unit
        const double ns = c.start + (c.first + (turns - 1) * c.more) * cols;
        if (type == 0 && g.offsets && (i == 1 || (i == 2 && g.n <= 64 * groups))) continue;
        if (i == 0 || ns < tiles_ns) {
            best = i;
            tiles_ns = ns;
        }
    }
    const double bytes = (double)groups * rows * cols * 17 / 32;
    tiles_ns = std::max(tiles_ns, bytes / bytes_per_ns[type]);
    const bool wide = !pair && mx_stream_wide(g, parts, (int)rows, (int)(cols / MX_BLOCK));
    const int64_t half_pass = mxs_rows(parts) * (wide ? 2 : 1) / 2;
    const double stream_ns =
        stream_start + std::max(stream[wide][type] * (double)(g.n + groups * half_pass) * rows * cols,
                                bytes / streamed_per_ns);
    return stream_ns > tiles_ns ? best : -1;
}

hipError_t product(const MxMat &w, const MxMat &up, const MxX &x, int dtype, const MxGroups &g,
                   const MxOut &o, hipStream_t st) {
    const int parts = dtype == QMOE_MXFP4 ? 0 : parts_of(dtype);
    const int64_t rows = up.q ? 2 * (int64_t)w.rows : w.rows;
    const int size = tile_size(g, parts, up.q != nullptr, rows, (int64_t)w.nb * MX_BLOCK);
    if (size < 0) return launch_mx_stream(w, up, x, parts, g, o, st);
    if (parts == 0) return launch_mx_tile_fp4(w, x, size, g, o, st);
    return launch_mx_tile(w, up, x, parts, size, g, o, st);
}

// Grids stay below 2^31 blocks: tiles (16 rows and more) times column blocks
// (32 weight rows and more).
bool grid_fits(int64_t n, int64_t experts, int64_t rows) {
    return (n / 16 + experts + 1) * (rows / 16 + 1) < LIM31 - 8;
}

// Checks shared by qmoe_mx_matmul (experts == 0) and qmoe_mx_grouped.
int product_checks(const qmoe_mxmat *W, int experts, int32_t x_dtype, const void *x,
                   const uint8_t *x_s, int64_t x_rows, int64_t x_ld, const int32_t *offsets,
                   const int32_t *pairs, int64_t n, int32_t y_dtype, void *y, int64_t y_ld, void *ws,
                   size_t ws_bytes) {
    const int E = experts > 0 ? experts : 1;
    const int s = check_mxmat(W, E);
    if (s) return s;
    if (!float_type(x_dtype) && x_dtype != QMOE_MXFP4) return QMOE_ERR_UNSUPPORTED;
    if (!float_type(y_dtype)) return QMOE_ERR_UNSUPPORTED;
    if (x_rows < 0 || n < 0 || x_rows > (1 << 30) || n > (1 << 30)) return QMOE_ERR_SHAPE;
    if (x_dtype != QMOE_MXFP4 && (x_ld < W->cols || x_ld >> 31)) return QMOE_ERR_SHAPE;
    if (y_ld < W->rows || y_ld >> 31) return QMOE_ERR_SHAPE;
    if (!grid_fits(n, E, W->rows)) return QMOE_ERR_SHAPE;
    if (n == 0) return QMOE_OK;
    if (x_rows == 0) return QMOE_ERR_SHAPE;
    if (!x || !y || (x_dtype == QMOE_MXFP4 && !x_s)) return QMOE_ERR_NULL;
    if (experts > 0 && !offsets) return QMOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !aligned4(offsets) || !aligned4(pairs)) return QMOE_ERR_ALIGN;
    if (x_dtype == QMOE_MXFP4 && !aligned16(x_s)) return QMOE_ERR_ALIGN;
    const int64_t nb = mx_blocks(W->cols);
    // 31-bit offsets: a gather spans all rows of x, otherwise a tile's rows do
    const bool dir = direct_rows(x_dtype, W->cols, x_ld);
    const int64_t row = x_dtype == QMOE_MXFP4 ? nb * 16
                        : dir                 ? x_ld * 2
                                              : (int64_t)parts_of(x_dtype) * pad128(W->cols) * 2;
    if ((pairs ? x_rows : 256) * row >= LIM31) return QMOE_ERR_UNSUPPORTED;
    const int64_t xb = x_dtype == QMOE_MXFP4 ? x_rows * nb * 16
                                             : span(x_rows, W->cols, x_ld, elem_bytes(x_dtype));
    const int64_t xsb = x_dtype == QMOE_MXFP4 ? x_rows * nb : 0;
    const int64_t yb = span(n, W->rows, y_ld, elem_bytes(y_dtype));
    const int64_t need = parts_bytes(x_dtype, x_rows, W->cols, x_ld);
    if (need > 0 && (!ws || (int64_t)ws_bytes < need)) return QMOE_ERR_WORKSPACE;
    if (need > 0 && !aligned16(ws)) return QMOE_ERR_ALIGN;
    const int64_t ob = offsets ? 4 * (int64_t)(E + 1) : 0, pb = pairs ? 4 * n : 0;
    if (overlap(y, yb, x, xb) || overlap(y, yb, x_s, xsb) || overlap(y, yb, offsets, ob) ||
        overlap(y, yb, pairs, pb) || overlaps_mat(y, yb, W, E) || overlap(y, yb, ws, need) ||
        overlap(ws, need, x, xb) || overlap(ws, need, offsets, ob) || overlap(ws, need, pairs, pb) ||
        overlaps_mat(ws, need, W, E))
        return QMOE_ERR_ALIAS;
    return QMOE_OK;
}

int run_product(const qmoe_mxmat *W, int32_t x_dtype, const void *x, const uint8_t *x_s,
                int64_t x_rows, int64_t x_ld, const MxGroups &g, int32_t y_dtype, void *y,
                int64_t y_ld, void *ws, hipStream_t st) {
    MxOut out{};
    out.y = y;
    out.ld = y_ld;
    out.type = y_dtype == QMOE_F32 ? MX_OUT_F32 : MX_OUT_BF16;
    const int wide = y_dtype == QMOE_F32 ? 4 : 8;      // outputs of a 16-byte store
    out.vec = W->rows % wide == 0 && y_ld % wide == 0;
    if (!g.offsets && x_dtype != QMOE_MXFP4 &&
        mx_few_matmul_fits(parts_of(x_dtype), g.n, pad128(W->cols)))
        return status_of(launch_mx_few(to_mx(W), MxMat{}, parts_of(x_dtype),
                                       MxFew{x, x_ld, W->cols, pad128(W->cols), nullptr, 1, 1, g.n},
                                       out, st));
    MxX o;
    const hipError_t e = operand(x_dtype, x, x_s, x_rows, W->cols, x_ld, ws, o, st);
    if (e != hipSuccess) return QMOE_ERR_HIP;
    return status_of(product(to_mx(W), MxMat{}, o, x_dtype, g, out, st));
}

// Layer calls of at most this many pairs run as two launches without a worklist
// (mx_decode.hip), which read an expert once per pair.  128 experts 4096 / 1536,
// top-8, replayed graphs: 1 token 31 us against 43 with the worklist, 4 tokens
// 98 against 104, 6 tokens 139 against 118.
constexpr int FEW_PAIRS = 32;

struct MxLayerWs {
    Worklist wl;
    int32_t *hist;
    void *x;             // parts of x (nullptr where x is the operand as it is)
    uint8_t *h;          // parts of h [pairs][parts][pad128(inter)]
    float *y;            // weighted expert rows [pairs][hidden]
    int64_t bytes;
};

MxLayerWs carve(void *ws, int E, int H, int F, int T, int k, int dtype) {
    MxLayerWs L{};
    Carver c(ws);
    const int64_t n = (int64_t)T * k;
    L.wl.counts = c.take<int32_t>(E);
    L.wl.offsets = c.take<int32_t>(E + 1);
    L.wl.pairs = c.take<int32_t>(n);
    L.wl.inv = c.take<int32_t>(n);
    L.wl.n_invalid = c.take<int32_t>(1);
    L.wl.tile_m = MFMA_BM;
    L.hist = c.take<int32_t>(wl_scratch_ints(n, E));
    L.x = c.take<uint8_t>(parts_bytes(dtype, T, H, H));
    L.h = c.take<uint8_t>(n * parts_of(dtype) * pad128(F) * 2);
    L.y = c.take<float>(n * H);
    L.bytes = c.off;
    return L;
}

int check_mx_layer(const qmoe_mx_layer_desc *d) {
    if (!d) return QMOE_ERR_NULL;
    if (d->struct_size != sizeof(qmoe_mx_layer_desc)) return QMOE_ERR_ABI;
    if (d->experts < 1 || d->experts > MAX_EXPERTS || d->hidden <= 0 || d->inter <= 0)
        return QMOE_ERR_SHAPE;
    const qmoe_mxmat *m[3] = {&d->gate, &d->up, &d->down};
    for (int i = 0; i < 3; i++) {
        const int s = check_mxmat(m[i], d->experts);
        if (s) return s;
        if (m[i]->rows != (i < 2 ? d->inter : d->hidden) || m[i]->cols != (i < 2 ? d->hidden : d->inter))
            return QMOE_ERR_SHAPE;
    }
    // the padded rows of h and the part rows of x stay within a tile's 32-bit offsets
    if ((int64_t)256 * 3 * 2 * pad128(d->hidden > d->inter ? d->hidden : d->inter) >= LIM31)
        return QMOE_ERR_UNSUPPORTED;
    return QMOE_OK;
}

}  // namespace

extern "C" {

size_t qmoe_mx_code_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return 0;
    return (size_t)(rows * ((cols + 31) / 32) * 16);
}

size_t qmoe_mx_scale_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return 0;
    return (size_t)(rows * ((cols + 31) / 32));
}

static int convert_checks(const void *v, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                          const uint8_t *q, const uint8_t *s) {
    if (rows < 0 || cols < 0 || cols >> 31 || ld < cols || ld >> 31 || rows >> 40) return QMOE_ERR_SHAPE;
    if (!float_type(dtype)) return QMOE_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return QMOE_OK;
    if (!v || !q || !s) return QMOE_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(v) % elem_bytes(dtype) || !aligned16(q)) return QMOE_ERR_ALIGN;
    const int64_t vb = span(rows, cols, ld, elem_bytes(dtype));
    const int64_t qb = (int64_t)qmoe_mx_code_bytes(rows, cols), sb = qb / 16;
    if (overlap(v, vb, q, qb) || overlap(v, vb, s, sb) || overlap(q, qb, s, sb)) return QMOE_ERR_ALIAS;
    return QMOE_OK;
}

int qmoe_mx_quantize(const void *x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t x_ld,
                     uint8_t *q, uint8_t *s, void *stream) {
    const int c = convert_checks(x, x_dtype, rows, cols, x_ld, q, s);
    if (c || rows == 0 || cols == 0) return c;
    return status_of(launch_mx_quantize(x, x_dtype == QMOE_F32, rows, (int)cols, x_ld, q, s,
                                        as_stream(stream)));
}

int qmoe_mx_dequantize(const uint8_t *q, const uint8_t *s, int64_t rows, int64_t cols, void *y,
                       int32_t y_dtype, int64_t y_ld, void *stream) {
    const int c = convert_checks(y, y_dtype, rows, cols, y_ld, q, s);
    if (c || rows == 0 || cols == 0) return c;
    return status_of(launch_mx_dequantize(q, s, rows, (int)cols, y, y_dtype == QMOE_F32, y_ld,
                                          as_stream(stream)));
}

size_t qmoe_mx_workspace_bytes(const qmoe_mxmat *W, int32_t x_dtype, int32_t x_rows, int64_t x_ld) {
    if (!W || W->cols <= 0 || x_rows < 0 || x_ld < 0) return 0;
    if (!float_type(x_dtype)) return 0;
    return (size_t)parts_bytes(x_dtype, x_rows, W->cols, x_ld);
}

int qmoe_mx_matmul(const qmoe_mxmat *W, int32_t x_dtype, const void *x, const uint8_t *x_s,
                   int32_t batch, int64_t x_ld, int32_t y_dtype, void *y, int64_t y_ld, void *ws,
                   size_t ws_bytes, void *stream) {
    const int s = product_checks(W, 0, x_dtype, x, x_s, batch, x_ld, nullptr, nullptr, batch, y_dtype,
                                 y, y_ld, ws, ws_bytes);
    if (s || batch == 0) return s;
    MxGroups g{};
    g.k = 1;
    g.experts = 1;
    g.n = batch;
    return run_product(W, x_dtype, x, x_s, batch, x_ld, g, y_dtype, y, y_ld, ws, as_stream(stream));
}

int qmoe_mx_grouped(const qmoe_mxmat *W, int32_t experts, int32_t x_dtype, const void *x,
                    const uint8_t *x_s, int32_t x_rows, int64_t x_ld, const int32_t *offsets,
                    const int32_t *pairs, int32_t k, int32_t n, int32_t y_dtype, void *y,
                    int64_t y_ld, void *ws, size_t ws_bytes, void *stream) {
    if (experts < 1 || experts > MAX_EXPERTS || k < 1) return QMOE_ERR_SHAPE;
    if (!pairs && x_rows < n) return QMOE_ERR_SHAPE;
    const int s = product_checks(W, experts, x_dtype, x, x_s, x_rows, x_ld, offsets, pairs, n, y_dtype,
                                 y, y_ld, ws, ws_bytes);
    if (s || n == 0) return s;
    MxGroups g{};
    g.offsets = offsets;
    g.pairs = pairs;
    g.k = k;
    g.experts = experts;
    g.n = n;
    return run_product(W, x_dtype, x, x_s, x_rows, x_ld, g, y_dtype, y, y_ld, ws, as_stream(stream));
}

size_t qmoe_mx_layer_workspace_bytes(const qmoe_mx_layer_desc *desc, int32_t tokens, int32_t k,
                                     int32_t x_dtype) {
    if (!desc || tokens < 0 || k < 1 || k > MAX_TOPK || desc->experts < 1 || desc->hidden < 1 ||
        desc->inter < 1 || !float_type(x_dtype))
        return 0;
    return (size_t)carve(nullptr, desc->experts, desc->hidden, desc->inter, tokens, k, x_dtype).bytes;
}

int qmoe_mx_layer(const qmoe_mx_layer_desc *desc, int32_t x_dtype, const void *x, int32_t tokens,
                  const int32_t *topk_ids, const float *topk_w, int32_t k, void *out, void *ws,
                  size_t ws_bytes, void *stream) {
    const int s = check_mx_layer(desc);
    if (s) return s;
    if (!float_type(x_dtype)) return QMOE_ERR_UNSUPPORTED;
    if (tokens < 0 || k < 1 || k > MAX_TOPK || (int64_t)tokens * k > (1 << 30)) return QMOE_ERR_SHAPE;
    const int E = desc->experts, H = desc->hidden, F = desc->inter;
    const int64_t n = (int64_t)tokens * k;
    if (!grid_fits(n, E, H > F ? H : F)) return QMOE_ERR_SHAPE;
    const int64_t xrow = direct_rows(x_dtype, H, H) ? 2 * (int64_t)H
                                                    : (int64_t)parts_of(x_dtype) * pad128(H) * 2;
    if (tokens * xrow >= LIM31) return QMOE_ERR_UNSUPPORTED;
    if (tokens == 0) return QMOE_OK;
    if (!x || !topk_ids || !topk_w || !out) return QMOE_ERR_NULL;
    if (!aligned16(x) || !aligned16(out) || !aligned4(topk_ids) || !aligned4(topk_w))
        return QMOE_ERR_ALIGN;
    const MxLayerWs L = carve(ws, E, H, F, tokens, k, x_dtype);
    if (!ws || (int64_t)ws_bytes < L.bytes) return QMOE_ERR_WORKSPACE;
    if (!aligned16(ws)) return QMOE_ERR_ALIGN;
    const int64_t xb = (int64_t)tokens * H * elem_bytes(x_dtype);
    if (overlap(out, xb, x, xb) || overlap(out, xb, topk_ids, 4 * n) || overlap(out, xb, topk_w, 4 * n) ||
        overlap(out, xb, ws, L.bytes) || overlap(ws, L.bytes, x, xb) ||
        overlap(ws, L.bytes, topk_ids, 4 * n) || overlap(ws, L.bytes, topk_w, 4 * n))
        return QMOE_ERR_ALIAS;
    const qmoe_mxmat *m[3] = {&desc->gate, &desc->up, &desc->down};
    for (const qmoe_mxmat *a : m)
        if (overlaps_mat(out, xb, a, E) || overlaps_mat(ws, L.bytes, a, E)) return QMOE_ERR_ALIAS;

    const hipStream_t st = as_stream(stream);
    const int P = parts_of(x_dtype);
    if (n <= FEW_PAIRS && mx_few_layer_fits(P, pad128(H), pad128(F))) {
        const MxFew f{x, H, H, pad128(H), topk_ids, k, E, (int)n};
        MxOut h{};
        h.y = L.h;
        h.width = pad128(F);
        h.ld = (int64_t)P * h.width * 2;
        hipError_t e = launch_mx_few(to_mx(&desc->gate), to_mx(&desc->up), P, f, h, st);
        if (e == hipSuccess)
            e = launch_mx_few_down(to_mx(&desc->down), P, f, L.h, h.ld, h.width, topk_w, tokens, out, st);
        return status_of(e);
    }
    hipError_t e = launch_worklist(topk_ids, (int)n, k, E, L.wl, L.hist, st);
    MxX xo;
    if (e == hipSuccess) e = operand(x_dtype, x, nullptr, tokens, H, H, L.x, xo, st);
    MxGroups g{};
    g.offsets = L.wl.offsets;
    g.pairs = L.wl.pairs;
    g.k = k;
    g.experts = E;
    g.n = (int)n;
    MxOut h{};
    h.y = L.h;
    h.width = pad128(F);
    h.ld = (int64_t)parts_of(x_dtype) * h.width * 2;
    if (e == hipSuccess) e = product(to_mx(&desc->gate), to_mx(&desc->up), xo, x_dtype, g, h, st);
    MxX ho{};
    ho.v = L.h;
    ho.ld = h.ld;
    ho.rows = n;
    ho.width = h.width;
    g.pairs = nullptr;
    MxOut y{};
    y.y = L.y;
    y.ld = H;
    y.type = MX_OUT_F32;
    y.w = topk_w;
    y.wpairs = L.wl.pairs;
    y.vec = H % 4 == 0;
    if (e == hipSuccess) e = product(to_mx(&desc->down), MxMat{}, ho, x_dtype, g, y, st);
    if (e == hipSuccess)
        e = launch_mx_combine(L.y, L.wl.inv, tokens, k, H, out, x_dtype == QMOE_F32, st);
    return status_of(e);
}

}  // extern "C"
