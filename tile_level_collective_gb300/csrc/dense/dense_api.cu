// C-ABI entry points of the dense block's operators (ptoc_dense.h): argument
// checks on the host before any CUDA call, then the launch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "dense/dense_internal.h"
#include "layers/operands.h"

namespace ptoc {
namespace {

// Zeros in a [rows, cols] matrix of 16-bit elements, padding left alone.
bool clear16(const ptoc_matrix* m, int64_t rows, int64_t cols, cudaStream_t s)
{
    if (!m) return true;
    if (m->ld == cols || rows == 1) return cudaMemsetAsync(m->data, 0, (size_t)(rows * cols) * 2, s) == cudaSuccess;
    return cudaMemset2DAsync(m->data, (size_t)m->ld * 2, 0, (size_t)cols * 2, (size_t)rows, s) == cudaSuccess;
}

ptoc_status check_param(const ptoc_layer_norm_params* q, int64_t cols, int dtype, Operands& o, bool forward)
{
    if (!q) return PTOC_ERR_INVALID_ARG;
    if (q->param_dtype != dtype && q->param_dtype != PTOC_F32) return PTOC_ERR_INVALID_ARG;
    if (forward && (!(q->eps > 0.0f) || !std::isfinite(q->eps))) return PTOC_ERR_INVALID_ARG;
    o.param(q->weight, cols, elem_size(q->param_dtype));
    if (forward) o.param(q->bias, cols, elem_size(q->param_dtype));
    return PTOC_OK;
}

// Sizes and weights that both passes of the gated block check.
ptoc_status check_ffn(const ptoc_gated_ffn_params* q, int64_t tokens, int64_t hidden, int64_t inter, int dtype,
                      Operands& o)
{
    if (!valid_dtype(dtype)) return PTOC_ERR_INVALID_ARG;
    if (dtype != PTOC_F16 && dtype != PTOC_BF16) return PTOC_ERR_UNSUPPORTED;
    if (!q || tokens < 0 || hidden < 1 || inter < 1) return PTOC_ERR_INVALID_ARG;
    if (q->act != PTOC_ACT_SILU && q->act != PTOC_ACT_GELU) return PTOC_ERR_INVALID_ARG;
    if (q->parts < 0 || q->parts > 2) return PTOC_ERR_INVALID_ARG;
    if (tokens > PTOC_FFN_MAX_TOKENS || hidden > PTOC_FFN_MAX_WIDTH || inter > PTOC_FFN_MAX_WIDTH)
        return PTOC_ERR_UNSUPPORTED;
    o.matrix(false, &q->w_in, 2 * inter, hidden, 2);
    o.matrix(false, &q->w_out, hidden, inter, 2);
    // the up rows, and u in a row of pre, begin at 16-byte words too
    if ((hidden | inter) & 7) o.vec = false;
    return PTOC_OK;
}

// Ranges of a call with many operands: [lo, hi) and whether it is written.
struct Mark {
    uintptr_t lo, hi;
    bool write;
};

// No written range may overlap another one.
bool separate(std::vector<Mark>& marks)
{
    std::sort(marks.begin(), marks.end(), [](const Mark& a, const Mark& b) { return a.lo < b.lo; });
    uintptr_t any = 0, written = 0;                          // ends of what began before
    for (const Mark& m : marks) {
        if (m.lo < written || (m.write && m.lo < any)) return false;
        any = std::max(any, m.hi);
        if (m.write) written = std::max(written, m.hi);
    }
    return true;
}

}  // namespace
}  // namespace ptoc

using namespace ptoc;

extern "C" ptoc_status ptoc_layer_norm(const ptoc_group* parts, int64_t ld_parts, const ptoc_matrix* x,
                                       const ptoc_layer_norm_params* params, const ptoc_matrix* out,
                                       const ptoc_matrix* normed, float* stats, int64_t rows, int64_t cols,
                                       ptoc_dtype dtype, cudaStream_t stream)
{
    const TraceRange trace("ptoc_layer_norm");
    ptoc_status st = check_box(rows, cols, dtype);
    if (st != PTOC_OK) return st;
    if (!parts || !parts->tensors || parts->nranks < 1 || parts->nranks > kMaxRanks) return PTOC_ERR_INVALID_ARG;
    if (!normed) return PTOC_ERR_INVALID_ARG;
    const int eb = elem_size(dtype);
    Operands o;
    LayerNormParams p;
    memset(&p, 0, sizeof(p));
    st = check_param(params, cols, dtype, o, true);
    if (st != PTOC_OK) return st;
    o.matrix(true, normed, rows, cols, eb);
    if (out) o.matrix(true, out, rows, cols, eb);
    if (x && !same_matrix(x, out)) o.matrix(false, x, rows, cols, eb);
    o.floats(true, stats, rows > INT64_MAX / 16 ? -1 : 2 * rows);
    if (!o.ok || ld_parts < cols) return PTOC_ERR_INVALID_ARG;
    const int64_t fp = footprint(rows, cols, ld_parts, eb);
    if (fp < 0) return PTOC_ERR_INVALID_ARG;
    Span part_reads[kMaxRanks];
    for (int r = 0; r < parts->nranks; ++r) {
        if ((!parts->tensors[r] && fp > 0) || !aligned(parts->tensors[r], eb)) return PTOC_ERR_INVALID_ARG;
        if (((uintptr_t)parts->tensors[r] | (uintptr_t)(rows > 1 ? ld_parts * eb : 0)) & 15u) o.vec = false;
        if ((uintptr_t)parts->tensors[r] & 15u) o.bases = false;
        part_reads[r] = Span{parts->tensors[r], (uintptr_t)fp};
        p.part[r] = parts->tensors[r];
    }
    st = o.disjoint();
    if (st == PTOC_OK) st = check_disjoint_outputs(o.writes, o.nw, part_reads, parts->nranks);
    if (st != PTOC_OK) return st;
    if (cols > PTOC_NORM_MAX_COLS) return PTOC_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return PTOC_OK;
    p.nparts = parts->nranks;
    p.ld_part = ld_parts;
    if (x) p.x = x->data, p.ld_x = x->ld;
    if (out) p.out = out->data, p.ld_out = out->ld;
    p.normed = normed->data;
    p.ld_normed = normed->ld;
    p.weight = params->weight;
    p.bias = params->bias;
    p.stats = stats;
    p.rows = rows;
    p.cols = cols;
    p.eps = params->eps;
    p.inv_cols = 1.0f / (float)cols;
    p.param_f32 = params->param_dtype == PTOC_F32;
    p.access = o.access(cols, eb);
    return status_of(launch_layer_norm(p, dtype, stream));
}

extern "C" size_t ptoc_layer_norm_backward_workspace(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0 || cols > PTOC_NORM_MAX_COLS) return 0;
    return (size_t)layer_norm_backward_grid(rows, cols) * 2 * (size_t)cols * sizeof(float);
}

extern "C" ptoc_status ptoc_layer_norm_backward(const ptoc_matrix* s, const float* stats,
                                                const ptoc_layer_norm_params* params, const ptoc_matrix* dy,
                                                const ptoc_matrix* du, const ptoc_matrix* dx, float* d_weight,
                                                float* d_bias, void* workspace, size_t workspace_bytes, int64_t rows,
                                                int64_t cols, ptoc_dtype dtype, cudaStream_t stream)
{
    const TraceRange trace("ptoc_layer_norm_backward");
    ptoc_status st = check_box(rows, cols, dtype);
    if (st != PTOC_OK) return st;
    if (!s || !dy || !dx || (!stats && rows > 0)) return PTOC_ERR_INVALID_ARG;
    const int eb = elem_size(dtype);
    Operands o;
    LayerNormBackParams p;
    memset(&p, 0, sizeof(p));
    st = check_param(params, cols, dtype, o, false);
    if (st != PTOC_OK) return st;
    if (rows > INT64_MAX / 16) return PTOC_ERR_INVALID_ARG;
    o.matrix(true, dx, rows, cols, eb);
    o.matrix(false, s, rows, cols, eb);
    if (!same_matrix(dy, dx)) o.matrix(false, dy, rows, cols, eb);
    if (du && !same_matrix(du, dx)) o.matrix(false, du, rows, cols, eb);
    o.floats(false, stats, 2 * rows);
    o.floats(true, d_weight, cols);
    o.floats(true, d_bias, cols);
    if (!o.ok) return PTOC_ERR_INVALID_ARG;
    if (cols > PTOC_NORM_MAX_COLS) return PTOC_ERR_UNSUPPORTED;
    const size_t need = ptoc_layer_norm_backward_workspace(rows, cols);
    if (need > 0) {
        if (!workspace || workspace_bytes < need || !aligned(workspace, kWsAlign)) return PTOC_ERR_INVALID_ARG;
        o.add(true, workspace, (int64_t)need);
    }
    st = o.disjoint();
    if (st != PTOC_OK) return st;
    if (rows == 0 || cols == 0) {
        // no elements: the sums over them are zero
        auto clear = [&](float* sums) {
            return !sums || !cols || cudaMemsetAsync(sums, 0, (size_t)cols * 4, stream) == cudaSuccess;
        };
        return clear(d_weight) && clear(d_bias) ? PTOC_OK : PTOC_ERR_CUDA;
    }
    p.s = s->data;
    p.ld_s = s->ld;
    p.dy = dy->data;
    p.ld_dy = dy->ld;
    if (du) p.du = du->data, p.ld_du = du->ld;
    p.dx = dx->data;
    p.ld_dx = dx->ld;
    p.weight = params->weight;
    p.stats = stats;
    p.d_weight = d_weight;
    p.d_bias = d_bias;
    p.partial = (float*)workspace;
    p.rows = rows;
    p.cols = cols;
    p.inv_cols = 1.0f / (float)cols;
    p.param_f32 = params->param_dtype == PTOC_F32;
    p.access = o.access(cols, eb);
    p.grid = layer_norm_backward_grid(rows, cols);
    return status_of(launch_layer_norm_backward(p, dtype, stream));
}

namespace {
bool ffn_sizes(int64_t tokens, int64_t hidden, int64_t inter)
{
    return tokens > 0 && hidden > 0 && inter > 0 && tokens <= PTOC_FFN_MAX_TOKENS && hidden <= PTOC_FFN_MAX_WIDTH &&
           inter <= PTOC_FFN_MAX_WIDTH;
}
}  // namespace

extern "C" size_t ptoc_gated_ffn_workspace(int64_t tokens, int64_t hidden, int64_t inter)
{
    return ffn_sizes(tokens, hidden, inter) ? ffn_workspace_bytes(tokens, hidden, inter) : 0;
}

extern "C" ptoc_status ptoc_gated_ffn(const ptoc_matrix* x, const ptoc_gated_ffn_params* params, const ptoc_matrix* y,
                                      const ptoc_matrix* pre, void* workspace, size_t workspace_bytes, int64_t tokens,
                                      int64_t hidden, int64_t inter, ptoc_dtype dtype, cudaStream_t stream)
{
    const TraceRange trace("ptoc_gated_ffn");
    Operands o;
    ptoc_status st = check_ffn(params, tokens, hidden, inter, dtype, o);
    if (st != PTOC_OK) return st;
    if (!x || !y) return PTOC_ERR_INVALID_ARG;
    o.matrix(false, x, tokens, hidden, 2);
    o.matrix(true, y, tokens, hidden, 2);
    if (pre) o.matrix(true, pre, tokens, 2 * inter, 2);
    if (!o.ok) return PTOC_ERR_INVALID_ARG;
    const size_t need = ptoc_gated_ffn_workspace(tokens, hidden, inter) * (params->parts == 2 ? 2 : 1);
    if (need > 0) {
        if (!workspace || workspace_bytes < need || !aligned(workspace, kWsAlign)) return PTOC_ERR_INVALID_ARG;
        o.add(true, workspace, (int64_t)need);
    }
    st = o.disjoint();
    if (st != PTOC_OK) return st;
    if (tokens == 0) return PTOC_OK;
    FfnParams p;
    memset(&p, 0, sizeof(p));
    p.x = x->data;
    p.ld_x = x->ld;
    p.w_in = params->w_in.data;
    p.ld_in = params->w_in.ld;
    p.w_out = params->w_out.data;
    p.ld_out = params->w_out.ld;
    p.y = y->data;
    p.ld_y = y->ld;
    if (pre) p.pre = pre->data, p.ld_pre = pre->ld;
    p.ws = (char*)workspace;
    p.tokens = tokens;
    p.hidden = hidden;
    p.inter = inter;
    p.act = params->act;
    p.parts = params->parts;
    p.vec = o.vec;
    return status_of(launch_ffn(p, dtype, stream));
}

extern "C" size_t ptoc_gated_ffn_backward_workspace(int64_t tokens, int64_t hidden, int64_t inter)
{
    return ffn_sizes(tokens, hidden, inter) ? ffn_backward_workspace_bytes(tokens, hidden, inter) : 0;
}

extern "C" ptoc_status ptoc_gated_ffn_backward(const ptoc_matrix* x, const ptoc_matrix* pre,
                                               const ptoc_gated_ffn_params* params, const ptoc_matrix* dy,
                                               const ptoc_matrix* dx, const ptoc_matrix* d_w_in,
                                               const ptoc_matrix* d_w_out, void* workspace, size_t workspace_bytes,
                                               int64_t tokens, int64_t hidden, int64_t inter, ptoc_dtype dtype,
                                               cudaStream_t stream)
{
    const TraceRange trace("ptoc_gated_ffn_backward");
    Operands o;
    ptoc_status st = check_ffn(params, tokens, hidden, inter, dtype, o);
    if (st != PTOC_OK) return st;
    if (!x || !pre || !dy) return PTOC_ERR_INVALID_ARG;
    o.matrix(false, x, tokens, hidden, 2);
    o.matrix(false, pre, tokens, 2 * inter, 2);
    o.matrix(false, dy, tokens, hidden, 2);
    if (dx) o.matrix(true, dx, tokens, hidden, 2);
    if (d_w_in) o.matrix(true, d_w_in, 2 * inter, hidden, 2);
    if (d_w_out) o.matrix(true, d_w_out, hidden, inter, 2);
    if (!o.ok) return PTOC_ERR_INVALID_ARG;
    const size_t need = ptoc_gated_ffn_backward_workspace(tokens, hidden, inter) * (params->parts == 2 ? 2 : 1);
    if (need > 0) {
        if (!workspace || workspace_bytes < need || !aligned(workspace, kWsAlign)) return PTOC_ERR_INVALID_ARG;
        o.add(true, workspace, (int64_t)need);
    }
    st = o.disjoint();
    if (st != PTOC_OK) return st;
    if (tokens == 0)
        return clear16(d_w_in, 2 * inter, hidden, stream) && clear16(d_w_out, hidden, inter, stream) ? PTOC_OK
                                                                                                      : PTOC_ERR_CUDA;
    if (!dx && !d_w_in && !d_w_out) return PTOC_OK;
    FfnBackParams p;
    memset(&p, 0, sizeof(p));
    p.x = x->data;
    p.ld_x = x->ld;
    p.pre = pre->data;
    p.ld_pre = pre->ld;
    p.w_in = params->w_in.data;
    p.ld_in = params->w_in.ld;
    p.w_out = params->w_out.data;
    p.ld_out = params->w_out.ld;
    p.dy = dy->data;
    p.ld_dy = dy->ld;
    if (dx) p.dx = dx->data, p.ld_dx = dx->ld;
    if (d_w_in) p.d_in = d_w_in->data, p.ld_din = d_w_in->ld;
    if (d_w_out) p.d_out = d_w_out->data, p.ld_dout = d_w_out->ld;
    p.ws = (char*)workspace;
    p.tokens = tokens;
    p.hidden = hidden;
    p.inter = inter;
    p.act = params->act;
    p.parts = params->parts;
    p.vec = o.vec;
    return status_of(launch_ffn_backward(p, dtype, stream));
}

extern "C" size_t ptoc_clip_gradients_workspace(int32_t count)
{
    return count < 0 || count > PTOC_CLIP_MAX_GRADIENTS ? 0 : clip_workspace_bytes(count);
}

extern "C" ptoc_status ptoc_clip_gradients(const ptoc_gradient* grads, int32_t count, float max_norm, float* result,
                                           void* workspace, size_t workspace_bytes, cudaStream_t stream)
{
    const TraceRange trace("ptoc_clip_gradients");
    if (count < 0 || (count > 0 && !grads) || !result || !aligned(result, 4) || !(max_norm > 0.0f))
        return PTOC_ERR_INVALID_ARG;
    if (count > PTOC_CLIP_MAX_GRADIENTS) return PTOC_ERR_UNSUPPORTED;
    int64_t elements = 0;
    bool many = false;
    try {
        std::vector<Mark> marks;
        marks.reserve(2 * (size_t)count + 2);
        for (int32_t i = 0; i < count; ++i) {
            const ptoc_gradient& g = grads[i];
            const ptoc_status st = check_box(g.rows, g.cols, g.dtype);
            if (st != PTOC_OK) return st;
            if (g.rows == 0 || g.cols == 0) continue;
            const int eb = elem_size(g.dtype);
            const int64_t bytes = footprint(g.rows, g.cols, g.ld, eb);
            if (!g.data || !aligned(g.data, eb) || g.ld < g.cols || bytes < 0) return PTOC_ERR_INVALID_ARG;
            const bool apart = g.out && (g.out != g.data || g.ld_out != g.ld);
            marks.push_back(Mark{(uintptr_t)g.data, (uintptr_t)g.data + (uintptr_t)bytes, !apart});
            if (g.out) {
                const int64_t out_bytes = footprint(g.rows, g.cols, g.ld_out, eb);
                if (!aligned(g.out, eb) || g.ld_out < g.cols || out_bytes < 0) return PTOC_ERR_INVALID_ARG;
                if (apart) marks.push_back(Mark{(uintptr_t)g.out, (uintptr_t)g.out + (uintptr_t)out_bytes, true});
            }
            many = many || g.rows > ((int64_t)1 << 45) / g.cols;
            elements = many ? 0 : elements + g.rows * g.cols;
            many = many || elements > (int64_t)1 << 45;
        }
        const size_t need = ptoc_clip_gradients_workspace(count);
        if (!workspace || workspace_bytes < need || !aligned(workspace, kWsAlign)) return PTOC_ERR_INVALID_ARG;
        marks.push_back(Mark{(uintptr_t)workspace, (uintptr_t)workspace + need, true});
        marks.push_back(Mark{(uintptr_t)result, (uintptr_t)result + 8, true});
        if (!separate(marks)) return PTOC_ERR_ALIAS;
    } catch (const std::bad_alloc&) {
        return PTOC_ERR_UNSUPPORTED;
    }
    if (many) return PTOC_ERR_UNSUPPORTED;
    return status_of(launch_clip(grads, count, max_norm, result, (double*)workspace, stream));
}
