// C entry points of the dense layer and the gated up-projection (declared in
// include/gemm.h): argument checks, choice of kernel, workspace layout.
// Host code only; the kernels live in linear_skinny.hip, linear_ring.hip,
// linear_tile.hip and act_grad.hip.
#include <stdint.h>

#include "linear.h"

namespace {

using dgor::Epilogue;
using dgor::Product;

constexpr size_t kWsAlign = 256;
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// A launch holds 2^32 threads: at most 2^22 tiles of 128 x 64, twice.
bool too_large(long long rows, long long cols) { return (rows + 127) / 128 * ((cols + 63) / 64) > (1LL << 22); }
bool ld_ok(int ld, int row) { return ld >= (row > 1 ? row : 1); }
bool op_ok(int op) { return op == GEMM_OP_N || op == GEMM_OP_T; }
bool act_ok(int act) { return act >= GEMM_ACT_NONE && act <= GEMM_ACT_SILU; }
bool missing(const void *p, long long rows, long long cols) { return rows > 0 && cols > 0 && !p; }

// How a product runs: the kernel, the tile and, where its tiles
// leave compute units idle, into how many parts the sum over k is split.
enum Kernel { kSkinny, kRing, kTile };
struct Way {
    Kernel kernel;
    int tile, splits, chunk;
};

long long tiles(const Product &p, int t)
{
    const int ft = p.gated ? t / 2 : t;
    return (long long)ceil_div(p.M, t) * ceil_div(p.N, ft) * p.nbatch;
}

// Whether sizes and strides let the rings run (the addresses apart): rows of
// whole 16-byte units, lane offsets within a tile below 2^31.
bool ring_sizes(const Product &p)
{
    const auto ok = [](int ld) { return ld % 8 == 0 && ld < (1 << 22); };
    const int a_row = p.trans_a ? p.M : p.K, b_row = p.trans_b ? p.K : p.N;
    return ok(p.lda) && ok(p.ldb) && a_row % 8 == 0 && b_row % 8 == 0;
}
bool ring_addresses(const Product &p)
{
    return (((uintptr_t)p.A[0] | (uintptr_t)p.A[1] | (uintptr_t)p.B[0] | (uintptr_t)p.B[1]) & 15) == 0;
}

// Fewer tiles than compute units: split k until two workgroups a unit,
// keeping at least four stages a part.
void split_over_k(const Product &p, Way &w)
{
    const long long n = tiles(p, w.tile);
    const int stages = dgor::product_stages(p);
    if (n <= 0 || n >= 256 || stages < 8)
        return;
    long long want = 512 / n;
    want = want < stages / 4 ? want : stages / 4;
    want = want < 16 ? want : 16;
    if (want > 1) {
        w.chunk = ceil_div(stages, want);
        w.splits = ceil_div(stages, w.chunk);
    }
}

Way choose(const Product &p, bool ring)
{
    Way w{ring ? kRing : kTile, 128, 1, 0};
    if (!p.trans_a && p.nbatch == 1 && p.M <= dgor::kSkinnyRows)
        return Way{kSkinny, 0, 1, 0};
    if (ring) {
        // cycles of a compute unit: a 256 tile's stage of 32 k is 1024 of its
        // matrix cores, four 128 tiles' the same at a lower rate, two at a time
        const long long stages = 2LL * dgor::product_stages(p), n256 = tiles(p, 256), n128 = tiles(p, 128);
        const long long c256 = (n256 + 255) / 256 * (stages * 1024 + 4000);
        const long long c128 = n128 <= 256 ? stages * 420 + 3000 : (n128 + 511) / 512 * (stages * 660 + 3000);
        if (c256 <= c128) {
            w.tile = 256;
            return w;
        }
    } else if (tiles(p, 128) < 512) {
        w.tile = 64;
    }
    split_over_k(p, w);
    return w;
}

// FP32 partial sums of a split product, on whichever kernel the operands'
// addresses will give it.
size_t part_bytes(const Product &p)
{
    size_t most = 0;
    for (int ring = 0; ring < (ring_sizes(p) ? 2 : 1); ++ring) {
        const Way w = choose(p, ring);
        const size_t b = w.splits <= 1 ? 0 : (size_t)(p.gated ? 2 : p.nbatch) * w.splits * p.M * p.N * sizeof(float);
        most = b > most ? b : most;
    }
    return round_up(most, kWsAlign);
}

// Runs a product; ws has part_bytes(p) bytes.
hipError_t run_product(Product p, void *ws, hipStream_t s)
{
    if (p.M == 0 || p.N == 0)
        return hipSuccess;
    const Way w = choose(p, ring_sizes(p) && ring_addresses(p));
    p.splits = w.splits;
    p.chunk = w.chunk;
    p.part = (float *)ws;
    if (w.kernel == kSkinny)
        return dgor::launch_linear_skinny(p, s);
    const hipError_t err =
        w.kernel == kRing ? dgor::launch_linear_ring(p, w.tile, s) : dgor::launch_tile(p, w.tile, s);
    if (err != hipSuccess || p.splits <= 1)
        return err;
    return dgor::launch_join(p, s);
}

Product plain_product(int M, int N, int K)
{
    Product p{};
    p.M = M, p.N = N, p.K = K;
    p.nseg = p.nbatch = 1;
    return p;
}

// The three products of a layer with n weights W (1, or 2 for the gated one)
// of K inputs x N outputs.
Product forward_product(int M, int N, int K, int op_w, int ldx, int ldw, bool gated)
{
    Product p = plain_product(M, N, K);
    p.lda = ldx, p.ldb = ldw;
    p.trans_b = op_w == GEMM_OP_T;
    p.gated = gated;
    return p;
}
Product input_gradient_product(int M, int N, int K, int op_w, int lddz, int ldw, int n)   // dX = sum of dZ W^T
{
    Product p = plain_product(M, K, N);
    p.lda = lddz, p.ldb = ldw;
    p.trans_b = op_w == GEMM_OP_N;
    p.nseg = n;
    return p;
}
Product weight_gradient_product(int M, int N, int K, int op_w, int ldx, int lddz, int n)   // X^T dZ, or dZ^T X
{
    Product p = op_w == GEMM_OP_N ? plain_product(K, N, M) : plain_product(N, K, M);
    p.lda = op_w == GEMM_OP_N ? ldx : lddz, p.ldb = op_w == GEMM_OP_N ? lddz : ldx;
    p.trans_a = true;
    p.nbatch = n;
    return p;
}

bool workspace_ok(const void *ws, size_t have, size_t need)
{
    return need == 0 || (ws && have >= need && ((uintptr_t)ws & (kWsAlign - 1)) == 0);
}

int done(hipError_t e) { return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH; }

// ------------------------------------------------------------ dense layer --

int check_linear(const gemm_linear_params *q, Product &p)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->N < 0 || q->K < 0 || too_large(q->M, q->N) || too_large(q->M, q->K) || too_large(q->K, q->N))
        return GEMM_ERR_INVALID_DIM;
    if (!op_ok(q->op_w) || !ld_ok(q->ldx, q->K) || !ld_ok(q->ldw, q->op_w ? q->K : q->N) || !ld_ok(q->ldy, q->N))
        return GEMM_ERR_INVALID_LAYOUT;
    if (!act_ok(q->activation))
        return GEMM_ERR_INVALID_ACTIVATION;
    p = forward_product(q->M, q->N, q->K, q->op_w, q->ldx, q->ldw, false);
    return GEMM_OK;
}

int run_linear(bool bf16, const gemm_linear_params *q, const uint16_t *X, const uint16_t *W, const uint16_t *bias,
               const void *R, void *Y, uint16_t *pre, void *ws, size_t ws_bytes, void *stream)
{
    Product p;
    const int rc = check_linear(q, p);
    if (rc != GEMM_OK)
        return rc;
    if ((R && !ld_ok(q->ldr, q->N)) || (pre && !ld_ok(q->ldp, q->N)))
        return GEMM_ERR_INVALID_LAYOUT;
    if (missing(X, q->M, q->K) || missing(W, q->K, q->N) || missing(Y, q->M, q->N))
        return GEMM_ERR_NULL_PTR;
    if (q->M == 0 || q->N == 0)
        return GEMM_OK;
    if (!workspace_ok(ws, ws_bytes, part_bytes(p)))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    p.bf16 = bf16;
    p.A[0] = p.A[1] = X;
    p.B[0] = p.B[1] = W;
    p.e.Y = Y, p.e.ldy = q->ldy, p.e.y_f32 = q->y_f32 != 0;
    p.e.bias = bias, p.e.act = q->activation;
    p.e.R = R, p.e.ldr = q->ldr;
    p.e.pre = pre, p.e.ldp = q->ldp;
    return done(run_product(p, ws, (hipStream_t)stream));
}

// Workspace of the dense layer's backward pass: dZ, the column sums of each
// row block, and the partial sums of whichever product is running.
struct BackwardLayout {
    int lddz;
    size_t dz, sums, part, bytes;   // offsets, and the whole size
};

int row_blocks(int M) { return ceil_div(M, dgor::kGradRows); }

int check_linear_backward(const gemm_linear_backward_params *q, Product &px, Product &pw, BackwardLayout &l)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->N < 0 || q->K < 0 || too_large(q->M, q->N) || too_large(q->M, q->K) || too_large(q->K, q->N))
        return GEMM_ERR_INVALID_DIM;
    if (!op_ok(q->op_w) || !ld_ok(q->lddy, q->N))
        return GEMM_ERR_INVALID_LAYOUT;
    if (!act_ok(q->activation))
        return GEMM_ERR_INVALID_ACTIVATION;
    l.lddz = q->activation == GEMM_ACT_NONE ? q->lddy : (int)round_up((size_t)q->N, 8);
    px = input_gradient_product(q->M, q->N, q->K, q->op_w, l.lddz, q->ldw, 1);
    pw = weight_gradient_product(q->M, q->N, q->K, q->op_w, q->ldx, l.lddz, 1);
    l.dz = 0;
    l.sums = q->activation == GEMM_ACT_NONE ? 0 : round_up((size_t)q->M * l.lddz * 2, kWsAlign);
    l.part = l.sums + round_up((size_t)row_blocks(q->M) * q->N * sizeof(float), kWsAlign);
    const size_t a = part_bytes(px), b = part_bytes(pw);
    l.bytes = l.part + (a > b ? a : b);
    return GEMM_OK;
}

int run_linear_backward(bool bf16, const gemm_linear_backward_params *q, const uint16_t *dY, const uint16_t *X,
                        const uint16_t *W, const uint16_t *pre, uint16_t *dX, uint16_t *dW, uint16_t *dbias, void *ws,
                        size_t ws_bytes, void *stream)
{
    Product px, pw;
    BackwardLayout l;
    const int rc = check_linear_backward(q, px, pw, l);
    if (rc != GEMM_OK)
        return rc;
    const bool act = q->activation != GEMM_ACT_NONE;
    const int w_row = q->op_w ? q->K : q->N;
    if ((dX && (!ld_ok(q->ldw, w_row) || !ld_ok(q->lddx, q->K))) ||
        (dW && (!ld_ok(q->ldx, q->K) || !ld_ok(q->lddw, w_row))) || (act && !ld_ok(q->ldp, q->N)))
        return GEMM_ERR_INVALID_LAYOUT;
    if (missing(dY, q->M, q->N) || (act && missing(pre, q->M, q->N)) || (dX && missing(W, q->K, q->N)) ||
        (dW && missing(X, q->M, q->K)))
        return GEMM_ERR_NULL_PTR;
    if (!workspace_ok(ws, ws_bytes, l.bytes))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    hipStream_t s = (hipStream_t)stream;
    uint8_t *base = (uint8_t *)ws;
    const uint16_t *dZ = dY;
    float *sums = dbias ? (float *)(base + l.sums) : nullptr;
    if (q->M > 0 && q->N > 0 && ((act && (dX || dW)) || dbias)) {
        uint16_t *out = act && (dX || dW) ? (uint16_t *)(base + l.dz) : nullptr;
        const hipError_t e = dgor::launch_act_grad(q->M, q->N, dY, q->lddy, act ? pre : nullptr, q->ldp, out, l.lddz,
                                                   q->activation, sums, bf16, s);
        if (e != hipSuccess)
            return GEMM_ERR_LAUNCH;
        if (out)
            dZ = out;
    }
    if (dbias && q->N > 0 &&
        dgor::launch_sum_blocks(row_blocks(q->M), q->N, sums, dbias, bf16, s) != hipSuccess)
        return GEMM_ERR_LAUNCH;
    px.bf16 = pw.bf16 = bf16;
    if (dX) {
        px.A[0] = px.A[1] = dZ;
        px.B[0] = px.B[1] = W;
        px.e.Y = dX, px.e.ldy = q->lddx;
        if (run_product(px, base + l.part, s) != hipSuccess)
            return GEMM_ERR_LAUNCH;
    }
    if (dW) {
        const bool t = q->op_w == GEMM_OP_T;
        pw.A[0] = pw.A[1] = t ? dZ : X;
        pw.B[0] = pw.B[1] = t ? X : dZ;
        pw.e.Y = dW, pw.e.ldy = q->lddw;
        if (run_product(pw, base + l.part, s) != hipSuccess)
            return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

// ---------------------------------------------------- gated up-projection --

int check_gated(const gemm_gated_params *q, Product &p)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->F < 0 || q->K < 0 || too_large(q->M, q->F) || too_large(q->M, q->K) || too_large(q->K, q->F))
        return GEMM_ERR_INVALID_DIM;
    if (!op_ok(q->op_w) || !ld_ok(q->ldx, q->K) || !ld_ok(q->ldw, q->op_w ? q->K : q->F) || !ld_ok(q->ldh, q->F))
        return GEMM_ERR_INVALID_LAYOUT;
    if (!act_ok(q->activation))
        return GEMM_ERR_INVALID_ACTIVATION;
    p = forward_product(q->M, q->F, q->K, q->op_w, q->ldx, q->ldw, true);
    return GEMM_OK;
}

int run_gated(bool bf16, const gemm_gated_params *q, const uint16_t *X, const uint16_t *Wg, const uint16_t *Wu,
              uint16_t *H, uint16_t *G, uint16_t *U, void *ws, size_t ws_bytes, void *stream)
{
    Product p;
    const int rc = check_gated(q, p);
    if (rc != GEMM_OK)
        return rc;
    if (G && !ld_ok(q->ldp, q->F))
        return GEMM_ERR_INVALID_LAYOUT;
    if (missing(X, q->M, q->K) || missing(Wg, q->K, q->F) || missing(Wu, q->K, q->F) || missing(H, q->M, q->F) ||
        (G != nullptr) != (U != nullptr))
        return GEMM_ERR_NULL_PTR;
    if (q->M == 0 || q->F == 0)
        return GEMM_OK;
    if (!workspace_ok(ws, ws_bytes, part_bytes(p)))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    p.bf16 = bf16;
    p.A[0] = p.A[1] = X;
    p.B[0] = Wg, p.B[1] = Wu;
    p.e.Y = H, p.e.ldy = q->ldh, p.e.act = q->activation;
    p.e.pre = G, p.e.pre2 = U, p.e.ldp = q->ldp;
    return done(run_product(p, ws, (hipStream_t)stream));
}

// Workspace of the gated backward pass: dG and dU, then the partial sums of
// whichever product is running.
struct GatedBackwardLayout {
    int ldd;
    size_t du, part, bytes;
};

int check_gated_backward(const gemm_gated_backward_params *q, Product &px, Product &pw, GatedBackwardLayout &l)
{
    if (!q)
        return GEMM_ERR_NULL_PTR;
    if (q->M < 0 || q->F < 0 || q->K < 0 || too_large(q->M, q->F) || too_large(q->M, q->K) || too_large(q->K, q->F))
        return GEMM_ERR_INVALID_DIM;
    if (!op_ok(q->op_w) || !ld_ok(q->lddh, q->F) || !ld_ok(q->ldp, q->F))
        return GEMM_ERR_INVALID_LAYOUT;
    if (!act_ok(q->activation))
        return GEMM_ERR_INVALID_ACTIVATION;
    l.ldd = (int)round_up((size_t)q->F, 8);
    px = input_gradient_product(q->M, q->F, q->K, q->op_w, l.ldd, q->ldw, 2);
    pw = weight_gradient_product(q->M, q->F, q->K, q->op_w, q->ldx, l.ldd, 2);
    l.du = round_up((size_t)q->M * l.ldd * 2, kWsAlign);
    l.part = 2 * l.du;
    const size_t a = part_bytes(px), b = part_bytes(pw);
    l.bytes = l.part + (a > b ? a : b);
    return GEMM_OK;
}

int run_gated_backward(bool bf16, const gemm_gated_backward_params *q, const uint16_t *dH, const uint16_t *X,
                       const uint16_t *Wg, const uint16_t *Wu, const uint16_t *G, const uint16_t *U, uint16_t *dX,
                       uint16_t *dWg, uint16_t *dWu, void *ws, size_t ws_bytes, void *stream)
{
    Product px, pw;
    GatedBackwardLayout l;
    const int rc = check_gated_backward(q, px, pw, l);
    if (rc != GEMM_OK)
        return rc;
    const int w_row = q->op_w ? q->K : q->F;
    if ((dX && (!ld_ok(q->ldw, w_row) || !ld_ok(q->lddx, q->K))) ||
        (dWg && (!ld_ok(q->ldx, q->K) || !ld_ok(q->lddw, w_row))))
        return GEMM_ERR_INVALID_LAYOUT;
    if (missing(dH, q->M, q->F) || missing(G, q->M, q->F) || missing(U, q->M, q->F) ||
        (dX && (missing(Wg, q->K, q->F) || missing(Wu, q->K, q->F))) || (dWg && missing(X, q->M, q->K)) ||
        (dWg != nullptr) != (dWu != nullptr))
        return GEMM_ERR_NULL_PTR;
    if (!dX && !dWg)
        return GEMM_OK;
    if (!workspace_ok(ws, ws_bytes, l.bytes))
        return GEMM_ERR_WORKSPACE;
    const int dev = dgor::device_status();
    if (dev != GEMM_OK)
        return dev;
    hipStream_t s = (hipStream_t)stream;
    uint8_t *base = (uint8_t *)ws;
    uint16_t *dG = (uint16_t *)base, *dU = (uint16_t *)(base + l.du);
    if (q->M > 0 && q->F > 0 &&
        dgor::launch_gate_grad(q->M, q->F, dH, q->lddh, G, U, q->ldp, dG, dU, l.ldd, q->activation, bf16, s) !=
            hipSuccess)
        return GEMM_ERR_LAUNCH;
    px.bf16 = pw.bf16 = bf16;
    if (dX) {
        px.A[0] = dG, px.A[1] = dU;
        px.B[0] = Wg, px.B[1] = Wu;
        px.e.Y = dX, px.e.ldy = q->lddx;
        if (run_product(px, base + l.part, s) != hipSuccess)
            return GEMM_ERR_LAUNCH;
    }
    if (dWg) {
        const bool t = q->op_w == GEMM_OP_T;
        pw.A[0] = t ? dG : X, pw.A[1] = t ? dU : X;
        pw.B[0] = t ? X : dG, pw.B[1] = t ? X : dU;
        pw.e.Y = dWg, pw.Y1 = dWu, pw.e.ldy = q->lddw;
        if (run_product(pw, base + l.part, s) != hipSuccess)
            return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_linear_workspace(const gemm_linear_params *params, size_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_NULL_PTR;
    Product p;
    const int rc = check_linear(params, p);
    if (rc == GEMM_OK)
        *bytes = p.M && p.N ? part_bytes(p) : 0;
    return rc;
}
int gemm_linear_f16(const gemm_linear_params *params, const uint16_t *X, const uint16_t *W, const uint16_t *bias,
                    const void *R, void *Y, uint16_t *pre, void *workspace, size_t workspace_bytes, void *stream)
{
    return run_linear(false, params, X, W, bias, R, Y, pre, workspace, workspace_bytes, stream);
}
int gemm_linear_bf16(const gemm_linear_params *params, const uint16_t *X, const uint16_t *W, const uint16_t *bias,
                     const void *R, void *Y, uint16_t *pre, void *workspace, size_t workspace_bytes, void *stream)
{
    return run_linear(true, params, X, W, bias, R, Y, pre, workspace, workspace_bytes, stream);
}

int gemm_linear_backward_workspace(const gemm_linear_backward_params *params, size_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_NULL_PTR;
    Product px, pw;
    BackwardLayout l;
    const int rc = check_linear_backward(params, px, pw, l);
    if (rc == GEMM_OK)
        *bytes = l.bytes;
    return rc;
}
int gemm_linear_backward_f16(const gemm_linear_backward_params *params, const uint16_t *dY, const uint16_t *X,
                             const uint16_t *W, const uint16_t *pre, uint16_t *dX, uint16_t *dW, uint16_t *dbias,
                             void *workspace, size_t workspace_bytes, void *stream)
{
    return run_linear_backward(false, params, dY, X, W, pre, dX, dW, dbias, workspace, workspace_bytes, stream);
}
int gemm_linear_backward_bf16(const gemm_linear_backward_params *params, const uint16_t *dY, const uint16_t *X,
                              const uint16_t *W, const uint16_t *pre, uint16_t *dX, uint16_t *dW, uint16_t *dbias,
                              void *workspace, size_t workspace_bytes, void *stream)
{
    return run_linear_backward(true, params, dY, X, W, pre, dX, dW, dbias, workspace, workspace_bytes, stream);
}

int gemm_gated_workspace(const gemm_gated_params *params, size_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_NULL_PTR;
    Product p;
    const int rc = check_gated(params, p);
    if (rc == GEMM_OK)
        *bytes = p.M && p.N ? part_bytes(p) : 0;
    return rc;
}
int gemm_gated_f16(const gemm_gated_params *params, const uint16_t *X, const uint16_t *Wg, const uint16_t *Wu,
                   uint16_t *H, uint16_t *G, uint16_t *U, void *workspace, size_t workspace_bytes, void *stream)
{
    return run_gated(false, params, X, Wg, Wu, H, G, U, workspace, workspace_bytes, stream);
}
int gemm_gated_bf16(const gemm_gated_params *params, const uint16_t *X, const uint16_t *Wg, const uint16_t *Wu,
                    uint16_t *H, uint16_t *G, uint16_t *U, void *workspace, size_t workspace_bytes, void *stream)
{
    return run_gated(true, params, X, Wg, Wu, H, G, U, workspace, workspace_bytes, stream);
}

int gemm_gated_backward_workspace(const gemm_gated_backward_params *params, size_t *bytes)
{
    if (!bytes)
        return GEMM_ERR_NULL_PTR;
    Product px, pw;
    GatedBackwardLayout l;
    const int rc = check_gated_backward(params, px, pw, l);
    if (rc == GEMM_OK)
        *bytes = l.bytes;
    return rc;
}
int gemm_gated_backward_f16(const gemm_gated_backward_params *params, const uint16_t *dH, const uint16_t *X,
                            const uint16_t *Wg, const uint16_t *Wu, const uint16_t *G, const uint16_t *U,
                            uint16_t *dX, uint16_t *dWg, uint16_t *dWu, void *workspace, size_t workspace_bytes,
                            void *stream)
{
    return run_gated_backward(false, params, dH, X, Wg, Wu, G, U, dX, dWg, dWu, workspace, workspace_bytes, stream);
}
int gemm_gated_backward_bf16(const gemm_gated_backward_params *params, const uint16_t *dH, const uint16_t *X,
                             const uint16_t *Wg, const uint16_t *Wu, const uint16_t *G, const uint16_t *U,
                             uint16_t *dX, uint16_t *dWg, uint16_t *dWu, void *workspace, size_t workspace_bytes,
                             void *stream)
{
    return run_gated_backward(true, params, dH, X, Wg, Wu, G, U, dX, dWg, dWu, workspace, workspace_bytes, stream);
}

}  // extern "C"
