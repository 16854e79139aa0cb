// C entry points of the 8-bit dense layer and gated up-projection (declared in
// include/gemm.h): argument checks, choice of kernel, workspace layout.  Host code
// only; the kernels live in i8_kernels.hip.
#include <stdint.h>

#include "i8.h"
#include "ring_plan.h"

namespace {

using dgor::I8Epilogue;
using dgor::I8Pack;
using dgor::Product;
using dgor::ceil_div;

constexpr size_t kWsAlign = 256;
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// As for the 16-bit layers: every launch then holds fewer than 2^32 threads.
bool too_large(long long rows, long long cols) { return (rows + 127) / 128 * ((cols + 63) / 64) >= (1LL << 22); }
bool ld_ok(int ld, int row) { return ld >= (row > 1 ? row : 1); }
bool missing(const void *p, long long rows, long long cols) { return rows > 0 && cols > 0 && !p; }

// The operands that are copied to the front of the workspace: rows that are not
// whole 16-byte units at strides on them, K x N matrices, and all where the caller
// says that they may start anywhere.
struct Copies {
    I8Pack r{};
    size_t at[3] = {}, bytes = 0;
    // Returns the copy's index, -1 where the operand is used as it is; ld becomes
    // the stride that the product reads.
    int add(int rows, int K, bool transpose, bool anywhere, int &ld)
    {
        // (rows of 2^23 bytes apart are past the rings' strides)
        if (rows == 0 || K == 0 || (!transpose && !anywhere && K % 16 == 0 && ld % 16 == 0 && ld < (1 << 23))) {
            ld = K == 0 ? 16 : ld;
            return -1;
        }
        const int i = r.jobs++;
        r.job[i] = {nullptr, nullptr, rows, K, ld, (int)round_up((size_t)K, 16), transpose, 0};
        at[i] = bytes;
        bytes += round_up((size_t)rows * r.job[i].ld_to, kWsAlign);
        ld = r.job[i].ld_to;
        return i;
    }
    const uint16_t *use(int i, const int8_t *from, uint8_t *ws)
    {
        if (i >= 0) {
            r.job[i].from = from;
            r.job[i].to = (int8_t *)(ws + at[i]);
        }
        return (const uint16_t *)(i >= 0 ? r.job[i].to : from);
    }
};

struct Layer {
    int M, N, K, op_w, ldx, ldw, ldy, activation, unaligned;
    bool gated;
};

struct Plan {
    Product p;
    Copies c;
    int copy[3];
    bool rows;             // the few-row kernel, else the rings:
    dgor::RingTile tile;
    size_t part, bytes;    // of the partial sums; of the whole workspace
};

// The ring's tile and split by the 16-bit rings' times: a stage moves the same
// bytes and takes as many cycles of the matrix cores.  Over 60 products (65 to 4096
// rows, sums of 64 to 8192) the chosen tile is at most 1.05 times the shortest for 53
// and 1.10 for 59; 1.31 (23.0 and 17.5 us) for 3776 x 2752 of a sum of 91, shorter than
// those that the times are fitted to.
void choose_ring(Plan &l)
{
    Product &p = l.p;
    const int stages = dgor::product_stages(p);
    double best = 0;
    bool any = false;
    for (const dgor::RingCost &c : dgor::kRings) {
        if (c.tile == dgor::kRing256x128)   // of 60 never the shortest, with its half lines: 152, 127 on 256 x 256
            continue;
        const long long n = dgor::tiles(p, ring_tile_m(c.tile), ring_tile_n(c.tile));
        for (int parts : {1, 2, 3, 4, 6, 8, 12, 16}) {
            if (parts > 1 && (2 * parts > stages || n * parts > 512 * c.share))
                break;
            const double us = dgor::microseconds(p, c, n, parts);
            if (!any || us < best) {
                any = true, best = us, l.tile = c.tile;
                p.chunk = parts > 1 ? ceil_div(stages, parts) : 0;
                p.splits = parts > 1 ? ceil_div(stages, p.chunk) : 1;
            }
        }
    }
    l.part = p.splits > 1 ? round_up((p.gated ? 2 : 1) * p.splits * dgor::part_size(p) * sizeof(int), kWsAlign) : 0;
}

int make_plan(const Layer &q, Plan &l)
{
    if (q.M < 0 || q.N < 0 || q.K < 0 || q.K > dgor::kI8LongestK || too_large(q.M, q.N) || too_large(q.M, q.K) ||
        too_large(q.K, q.N))
        return GEMM_ERR_INVALID_DIM;
    if ((q.op_w != GEMM_OP_N && q.op_w != GEMM_OP_T) || !ld_ok(q.ldx, q.K) || !ld_ok(q.ldw, q.op_w ? q.K : q.N) ||
        !ld_ok(q.ldy, q.N))
        return GEMM_ERR_INVALID_LAYOUT;
    if (q.activation < GEMM_ACT_NONE || q.activation > GEMM_ACT_SILU)
        return GEMM_ERR_INVALID_ACTIVATION;
    l = Plan{};
    l.copy[0] = l.copy[1] = l.copy[2] = -1;
    if (q.M == 0 || q.N == 0)
        return GEMM_OK;
    int ldx = q.ldx, ldw = q.ldw, ldu = q.ldw;
    l.copy[0] = l.c.add(q.M, q.K, false, q.unaligned != 0, ldx);
    l.copy[1] = l.c.add(q.N, q.K, q.op_w == GEMM_OP_N, q.unaligned != 0, ldw);
    if (q.gated)
        l.copy[2] = l.c.add(q.N, q.K, q.op_w == GEMM_OP_N, q.unaligned != 0, ldu);
    Product &p = l.p;
    p.M = q.M, p.N = q.N, p.K = (int)round_up((size_t)q.K, 16) / 2;
    p.lda = ldx / 2, p.ldb = ldw / 2;
    p.trans_b = p.units = true;
    p.gated = q.gated;
    p.nseg = p.nbatch = p.terms = p.splits = 1;
    p.e.act = q.activation;
    l.rows = q.M <= dgor::kSkinnyRows && 512LL * ceil_div(q.N, dgor::kI8Strip) < (1LL << 32);
    if (!l.rows)
        choose_ring(l);
    l.bytes = l.c.bytes + l.part;
    return GEMM_OK;
}

int run(const Layer &q, Plan &l, I8Epilogue e, const int8_t *X, const int8_t *W, const int8_t *U, void *ws,
        size_t ws_bytes, void *stream)
{
    if (missing(X, q.M, q.K) || missing(W, q.K, q.N) || (q.gated && missing(U, q.K, q.N)) || missing(e.Y, q.M, q.N) ||
        missing(e.row, q.M, 1) || missing(e.col, q.N, 1) || (q.gated && missing(e.up, q.N, 1)))
        return GEMM_ERR_NULL_PTR;
    if (q.M == 0 || q.N == 0)
        return GEMM_OK;
    const auto off = [](const void *p, int copy) { return copy < 0 && ((uintptr_t)p & 15) != 0; };
    if (q.K > 0 && (off(X, l.copy[0]) || off(W, l.copy[1]) || (q.gated && off(U, l.copy[2]))))
        return GEMM_ERR_INVALID_LAYOUT;
    if (l.bytes && (!ws || ws_bytes < l.bytes || ((uintptr_t)ws & (kWsAlign - 1)) != 0))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    hipStream_t s = (hipStream_t)stream;
    uint8_t *base = (uint8_t *)ws;
    Product &p = l.p;
    const uint16_t *a = l.c.use(l.copy[0], X, base), *b = l.c.use(l.copy[1], W, base),
                   *u = q.gated ? l.c.use(l.copy[2], U, base) : b;
    p.A = {a, 0, 0, 0};
    p.B = {b, (long long)((uintptr_t)u - (uintptr_t)b), 0, 0};
    p.part = (float *)(base + l.c.bytes);
    e.act = q.activation, e.ldy = q.ldy;
    hipError_t err = dgor::launch_i8_pack(l.c.r, s);
    if (err == hipSuccess)
        err = l.rows ? dgor::launch_i8_rows(p, e, s) : dgor::launch_i8_ring(p, e, l.tile, s);
    if (err == hipSuccess && p.splits > 1)
        err = dgor::launch_i8_join(p, e, s);
    return err == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

Layer layer_of(const gemm_linear_i8_params &q)
{
    return {q.M, q.N, q.K, q.op_w, q.ldx, q.ldw, q.ldy, q.activation, q.unaligned, false};
}
Layer layer_of(const gemm_gated_i8_params &q)
{
    return {q.M, q.F, q.K, q.op_w, q.ldx, q.ldw, q.ldh, q.activation, q.unaligned, true};
}
template <class Params>
int workspace(const Params *q, size_t *bytes)
{
    if (!q || !bytes)
        return GEMM_ERR_NULL_PTR;
    Plan l;
    const int rc = make_plan(layer_of(*q), l);
    if (rc == GEMM_OK)
        *bytes = l.bytes;
    return rc;
}

int run_linear(int fmt, const gemm_linear_i8_params *q, const int8_t *X, const float *xs, const int8_t *W,
               const float *ws, const float *bias, const void *R, void *Y, void *work, size_t work_bytes, void *stream)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    Plan l;
    const Layer d = layer_of(*q);
    const int rc = make_plan(d, l);
    if (rc != GEMM_OK)
        return rc;
    if (R && !ld_ok(q->ldr, q->N))
        return GEMM_ERR_INVALID_LAYOUT;
    I8Epilogue e{};
    e.row = xs, e.col = ws, e.bias = bias;
    e.R = R, e.ldr = q->ldr;
    e.Y = Y, e.fmt = fmt;
    return run(d, l, e, X, W, nullptr, work, work_bytes, stream);
}

int run_gated(int fmt, const gemm_gated_i8_params *q, const int8_t *X, const float *xs, const int8_t *Wg,
              const float *gs, const int8_t *Wu, const float *us, void *H, void *work, size_t work_bytes, void *stream)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    Plan l;
    const Layer d = layer_of(*q);
    const int rc = make_plan(d, l);
    if (rc != GEMM_OK)
        return rc;
    I8Epilogue e{};
    e.row = xs, e.col = gs, e.up = us;
    e.Y = H, e.fmt = fmt;
    return run(d, l, e, X, Wg, Wu, work, work_bytes, stream);
}

}  // namespace

extern "C" {

int gemm_linear_i8_workspace(const gemm_linear_i8_params *params, size_t *bytes) { return workspace(params, bytes); }
int gemm_linear_i8_f32(const gemm_linear_i8_params *params, const int8_t *X, const float *x_scale, const int8_t *W,
                       const float *w_scale, const float *bias, const float *R, float *Y, void *workspace,
                       size_t workspace_bytes, void *stream)
{
    return run_linear(dgor::kF32, params, X, x_scale, W, w_scale, bias, R, Y, workspace, workspace_bytes, stream);
}
int gemm_linear_i8_f16(const gemm_linear_i8_params *params, const int8_t *X, const float *x_scale, const int8_t *W,
                       const float *w_scale, const float *bias, const uint16_t *R, uint16_t *Y, void *workspace,
                       size_t workspace_bytes, void *stream)
{
    return run_linear(dgor::kF16, params, X, x_scale, W, w_scale, bias, R, Y, workspace, workspace_bytes, stream);
}
int gemm_linear_i8_bf16(const gemm_linear_i8_params *params, const int8_t *X, const float *x_scale, const int8_t *W,
                        const float *w_scale, const float *bias, const uint16_t *R, uint16_t *Y, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    return run_linear(dgor::kBF16, params, X, x_scale, W, w_scale, bias, R, Y, workspace, workspace_bytes, stream);
}

int gemm_gated_i8_workspace(const gemm_gated_i8_params *params, size_t *bytes) { return workspace(params, bytes); }
int gemm_gated_i8_f32(const gemm_gated_i8_params *params, const int8_t *X, const float *x_scale, const int8_t *Wg,
                      const float *wg_scale, const int8_t *Wu, const float *wu_scale, float *H, void *workspace,
                      size_t workspace_bytes, void *stream)
{
    return run_gated(dgor::kF32, params, X, x_scale, Wg, wg_scale, Wu, wu_scale, H, workspace, workspace_bytes,
                     stream);
}
int gemm_gated_i8_f16(const gemm_gated_i8_params *params, const int8_t *X, const float *x_scale, const int8_t *Wg,
                      const float *wg_scale, const int8_t *Wu, const float *wu_scale, uint16_t *H, void *workspace,
                      size_t workspace_bytes, void *stream)
{
    return run_gated(dgor::kF16, params, X, x_scale, Wg, wg_scale, Wu, wu_scale, H, workspace, workspace_bytes,
                     stream);
}
int gemm_gated_i8_bf16(const gemm_gated_i8_params *params, const int8_t *X, const float *x_scale, const int8_t *Wg,
                       const float *wg_scale, const int8_t *Wu, const float *wu_scale, uint16_t *H, void *workspace,
                       size_t workspace_bytes, void *stream)
{
    return run_gated(dgor::kBF16, params, X, x_scale, Wg, wg_scale, Wu, wu_scale, H, workspace, workspace_bytes,
                     stream);
}

}  // extern "C"
