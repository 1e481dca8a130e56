// C-ABI entry points of the layer operators (ptoc_layers.h): argument checks
// on the host before any CUDA call, then the launch.
#include <cmath>
#include <cstring>

#include "host/host_checks.h"
#include "layers/layers_internal.h"

namespace ptoc {
namespace {

constexpr int kMaxOperands = 16;

// The operands of one call: what it writes, what it reads.
struct Operands {
    Span writes[kMaxOperands] = {}, reads[kMaxOperands] = {};
    int nw = 0, nr = 0;
    bool ok = true;               // sizes, pitches and alignments so far
    bool vec = true;              // every base and pitch allows 16-byte vectors
    bool bases = true;            // everything copied in words of rows at any pitch begins at a multiple of 16 bytes

    void add(bool write, const void* p, int64_t bytes)
    {
        if (bytes < 0) ok = false;
        if (write) writes[nw++] = Span{p, (uintptr_t)(bytes > 0 ? bytes : 0)};
        else reads[nr++] = Span{p, (uintptr_t)(bytes > 0 ? bytes : 0)};
    }
    // A matrix operand. `word`: 8 elements are moved as aligned words of this
    // many bytes (16, or 8 for codes; exponents go byte by byte).
    void rows(bool write, const void* p, int64_t ld, int64_t rows, int64_t cols, int eb, int word)
    {
        if ((!p && rows > 0 && cols > 0) || ld < cols || !aligned(p, eb)) {
            ok = false;
            return;
        }
        if (((uintptr_t)p | (uintptr_t)(rows > 1 ? ld * eb : 0)) & (uintptr_t)(word - 1)) vec = false;
        if (word > 1 && ((uintptr_t)p & 15u)) bases = false;
        add(write, p, footprint(rows, cols, ld, eb));
    }
    void matrix(bool write, const ptoc_matrix* m, int64_t nrows, int64_t cols, int eb)
    {
        rows(write, m->data, m->ld, nrows, cols, eb, 16);
    }
    void ckpt(bool write, const ptoc_ckpt8* k, int64_t nrows, int64_t cols)
    {
        rows(write, k->codes, k->ld_codes, nrows, cols, 1, 8);
        rows(write, k->exps, k->ld_exps, nrows, (cols + PTOC_CKPT_BLOCK - 1) / PTOC_CKPT_BLOCK, 1, 1);
    }
    void floats(bool write, const float* p, int64_t n)
    {
        if (!p) return;
        if (!aligned(p, 4)) ok = false;
        add(write, p, footprint(1, n, n, 4));
    }
    // A parameter read along the columns.
    void param(const void* p, int64_t n, int eb)
    {
        if (!p) return;
        if (!aligned(p, eb)) ok = false;
        if ((uintptr_t)p & 15u) vec = false;
        add(false, p, footprint(1, n, n, eb));
    }
    int access(int64_t cols, int eb) const
    {
        return vec && cols % (16 / eb) == 0 ? kAligned : bases ? kOddPitch : kAnywhere;
    }
    ptoc_status disjoint() const { return check_disjoint_outputs(writes, nw, reads, nr); }
};

bool float_dtype(int dtype) { return dtype == PTOC_F32 || dtype == PTOC_F16 || dtype == PTOC_BF16; }

// dtype, sizes: what every call on [rows, cols] matrices checks first.
ptoc_status check_box(int64_t rows, int64_t cols, int dtype)
{
    if (!valid_dtype(dtype)) return PTOC_ERR_INVALID_ARG;
    if (!float_dtype(dtype)) return PTOC_ERR_UNSUPPORTED;
    if (rows < 0 || cols < 0) return PTOC_ERR_INVALID_ARG;
    return PTOC_OK;
}

ptoc_status status_of(cudaError_t e) { return e == cudaSuccess ? PTOC_OK : PTOC_ERR_CUDA; }

ptoc_status ckpt8_call(const ptoc_matrix* x, const ptoc_ckpt8* k, int64_t rows, int64_t cols, int dtype, bool restore,
                       cudaStream_t stream)
{
    const ptoc_status st = check_box(rows, cols, dtype);
    if (st != PTOC_OK) return st;
    if (!x || !k) return PTOC_ERR_INVALID_ARG;
    Operands o;
    o.matrix(restore, x, rows, cols, elem_size(dtype));
    o.ckpt(!restore, k, rows, cols);
    if (!o.ok) return PTOC_ERR_INVALID_ARG;
    const ptoc_status al = o.disjoint();
    if (al != PTOC_OK) return al;
    if (rows == 0 || cols == 0) return PTOC_OK;
    // columns and work units of 256 columns are counted in 32 bits
    if (cols > INT32_MAX - 255 || rows > INT32_MAX / ((cols + 255) / 256)) return PTOC_ERR_UNSUPPORTED;
    Ckpt8Params p;
    p.x = x->data;
    p.ld = x->ld;
    p.ckpt = *k;
    p.rows = rows;
    p.cols = cols;
    const bool words = ((uintptr_t)k->codes & 7u) == 0 && (rows == 1 || k->ld_codes % 8 == 0);
    p.access = o.vec && cols % (16 / elem_size(dtype)) == 0 ? kAligned : words ? kOddPitch : kAnywhere;
    return status_of(restore ? launch_restore8(p, dtype, stream) : launch_checkpoint8(p, dtype, stream));
}

int gate_kind(const ptoc_block_norm_params* q)
{
    if (!q->gate) return kGateNone;
    if (q->gate_row_stride == 0) return q->gate_col_stride == 0 ? kGateScalar : kGateChannel;
    return q->gate_col_stride == 0 ? kGateToken : kGateElement;
}

// Checks the parameters, adds their operands and fills the kernel's copy.
ptoc_status norm_common(const ptoc_block_norm_params* q, int64_t rows, int64_t cols, int dtype, Operands& o,
                        NormCommon& c)
{
    if (!q) return PTOC_ERR_INVALID_ARG;
    if (q->param_dtype != dtype && q->param_dtype != PTOC_F32) return PTOC_ERR_INVALID_ARG;
    if (q->post_norm != 0 && q->post_norm != 1) return PTOC_ERR_INVALID_ARG;
    if (!(q->eps > 0.0f) || !std::isfinite(q->eps)) return PTOC_ERR_INVALID_ARG;
    if (q->gate && (q->gate_row_stride < 0 || (q->gate_col_stride != 0 && q->gate_col_stride != 1)))
        return PTOC_ERR_INVALID_ARG;
    const int eb = elem_size(q->param_dtype);
    if (q->post_norm) o.param(q->post_weight, cols, eb);
    o.param(q->pre_weight, cols, eb);
    if (q->gate) {
        const int kind = gate_kind(q);
        if (kind == kGateElement) {
            if (q->gate_row_stride < cols) return PTOC_ERR_INVALID_ARG;
            o.rows(false, q->gate, q->gate_row_stride, rows, cols, eb, 16);
        } else if (kind == kGateChannel) {
            o.param(q->gate, cols, eb);
        } else {
            if (!aligned(q->gate, eb)) return PTOC_ERR_INVALID_ARG;
            o.add(false, q->gate, footprint(kind == kGateToken ? rows : 1, 1, q->gate_row_stride, eb));
        }
    }
    c.post_weight = q->post_norm ? q->post_weight : nullptr;
    c.pre_weight = q->pre_weight;
    c.gate = q->gate;
    c.gate_rs = q->gate ? q->gate_row_stride : 0;
    c.gate_cs = q->gate ? q->gate_col_stride : 0;
    c.post_norm = q->post_norm;
    c.param_f32 = q->param_dtype == PTOC_F32;
    c.residual_scale = q->residual_scale;
    c.branch_scale = q->branch_scale;
    c.eps = q->eps;
    c.inv_cols = cols > 0 ? 1.0f / (float)cols : 0.0f;
    c.rows = rows;
    c.cols = cols;
    return PTOC_OK;
}

// An output that may be exactly an input: then the input is no operand of its
// own, as each thread reads its elements before it writes them.
bool same_matrix(const ptoc_matrix* a, const ptoc_matrix* b) { return a && b && a->data == b->data && a->ld == b->ld; }

constexpr size_t kWsAlign = 256;

}  // namespace
}  // namespace ptoc

using namespace ptoc;

extern "C" ptoc_status ptoc_checkpoint8(const ptoc_matrix* x, const ptoc_ckpt8* out, int64_t rows, int64_t cols,
                                        ptoc_dtype dtype, cudaStream_t stream)
{
    const TraceRange trace("ptoc_checkpoint8");
    return ckpt8_call(x, out, rows, cols, dtype, false, stream);
}

extern "C" ptoc_status ptoc_restore8(const ptoc_ckpt8* in, const ptoc_matrix* x, int64_t rows, int64_t cols,
                                     ptoc_dtype dtype, cudaStream_t stream)
{
    const TraceRange trace("ptoc_restore8");
    return ckpt8_call(x, in, rows, cols, dtype, true, stream);
}

extern "C" ptoc_status ptoc_block_norm(const ptoc_group* parts, int64_t ld_parts, const ptoc_matrix* x,
                                       const ptoc_block_norm_params* params, const ptoc_matrix* out,
                                       const ptoc_matrix* normed, const ptoc_matrix* block_out,
                                       const ptoc_ckpt8* block_ckpt, const ptoc_ckpt8* stream_ckpt, float* rstd,
                                       int64_t rows, int64_t cols, ptoc_dtype dtype, cudaStream_t stream)
{
    const TraceRange trace("ptoc_block_norm");
    ptoc_status st = check_box(rows, cols, dtype);
    if (st != PTOC_OK) return st;
    if (!parts || !parts->tensors || parts->nranks < 1 || parts->nranks > kMaxRanks) return PTOC_ERR_INVALID_ARG;
    if (!x || !out) return PTOC_ERR_INVALID_ARG;
    const int eb = elem_size(dtype);
    Operands o;
    NormParams p;
    memset(&p, 0, sizeof(p));
    st = norm_common(params, rows, cols, dtype, o, p.c);
    if (st != PTOC_OK) return st;
    o.matrix(true, out, rows, cols, eb);
    if (!same_matrix(x, out)) o.matrix(false, x, rows, cols, eb);
    if (normed) o.matrix(true, normed, rows, cols, eb);
    if (block_out) o.matrix(true, block_out, rows, cols, eb);
    if (block_ckpt) o.ckpt(true, block_ckpt, rows, cols);
    if (stream_ckpt) o.ckpt(true, stream_ckpt, rows, cols);
    o.floats(true, rstd, rows > INT64_MAX / 16 ? -1 : 2 * rows);
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
    if (st != PTOC_OK) return st;
    st = check_disjoint_outputs(o.writes, o.nw, part_reads, parts->nranks);
    if (st != PTOC_OK) return st;
    if (cols > PTOC_NORM_MAX_COLS) return PTOC_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return PTOC_OK;
    p.c.access = o.access(cols, eb);
    p.nparts = parts->nranks;
    p.ld_part = ld_parts;
    p.x = x->data;
    p.ld_x = x->ld;
    p.out = out->data;
    p.ld_out = out->ld;
    if (normed) p.normed = normed->data, p.ld_normed = normed->ld;
    if (block_out) p.block_out = block_out->data, p.ld_block = block_out->ld;
    if (block_ckpt) p.block_ckpt = *block_ckpt;
    if (stream_ckpt) p.stream_ckpt = *stream_ckpt;
    p.rstd = rstd;
    return status_of(launch_block_norm(p, dtype, stream));
}

extern "C" size_t ptoc_block_norm_backward_workspace(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0 || cols > PTOC_NORM_MAX_COLS) return 0;
    return (size_t)norm_backward_grid(rows, cols) * (2 * (size_t)cols + 1) * sizeof(float);
}

extern "C" ptoc_status ptoc_block_norm_backward(const ptoc_block_norm_saved* saved,
                                                const ptoc_block_norm_params* params, const ptoc_matrix* dy,
                                                const ptoc_matrix* du, const ptoc_matrix* d_residual,
                                                const ptoc_matrix* d_block, float* d_pre_weight, float* d_post_weight,
                                                float* d_gate, void* workspace, size_t workspace_bytes, int64_t rows,
                                                int64_t cols, ptoc_dtype dtype, cudaStream_t stream)
{
    const TraceRange trace("ptoc_block_norm_backward");
    ptoc_status st = check_box(rows, cols, dtype);
    if (st != PTOC_OK) return st;
    if (!saved || !dy || !d_residual || !d_block || (!saved->rstd && rows > 0)) return PTOC_ERR_INVALID_ARG;
    const ptoc_block_norm_saved& sv = *saved;
    // an empty tensor may have no address in either form
    if ((sv.block.data && sv.block_ckpt.codes) || (sv.stream.data && sv.stream_ckpt.codes)) return PTOC_ERR_INVALID_ARG;
    const int eb = elem_size(dtype);
    Operands o;
    NormBackParams p;
    memset(&p, 0, sizeof(p));
    st = norm_common(params, rows, cols, dtype, o, p.c);
    if (st != PTOC_OK) return st;
    if ((d_post_weight && !params->post_norm) || (d_gate && !params->gate)) return PTOC_ERR_INVALID_ARG;
    p.gate_kind = d_gate ? gate_kind(params) : kGateNone;
    if (rows > 0 && cols > 0) {
        if (sv.block_ckpt.codes) o.ckpt(false, &sv.block_ckpt, rows, cols);
        else if (!same_matrix(&sv.block, d_block)) o.matrix(false, &sv.block, rows, cols, eb);
        if (sv.stream_ckpt.codes) o.ckpt(false, &sv.stream_ckpt, rows, cols);
        else o.matrix(false, &sv.stream, rows, cols, eb);
    }
    if (rows > INT64_MAX / 16) return PTOC_ERR_INVALID_ARG;
    o.floats(false, sv.rstd, 2 * rows);
    o.matrix(false, dy, rows, cols, eb);
    if (du && !same_matrix(du, d_residual)) o.matrix(false, du, rows, cols, eb);
    o.matrix(true, d_residual, rows, cols, eb);
    o.matrix(true, d_block, rows, cols, eb);
    o.floats(true, d_pre_weight, cols);
    o.floats(true, d_post_weight, cols);
    const int64_t gate_n = p.gate_kind == kGateScalar ? 1 : p.gate_kind == kGateChannel ? cols : rows;
    if (p.gate_kind == kGateElement) {
        o.rows(true, d_gate, cols, rows, cols, 4, 4);
    } else {
        o.floats(true, d_gate, gate_n);
    }
    if (!o.ok) return PTOC_ERR_INVALID_ARG;
    if (cols > PTOC_NORM_MAX_COLS) return PTOC_ERR_UNSUPPORTED;
    const size_t need = ptoc_block_norm_backward_workspace(rows, cols);
    if (need > 0) {
        if (!workspace || workspace_bytes < need || !aligned(workspace, kWsAlign)) return PTOC_ERR_INVALID_ARG;
        o.add(true, workspace, (int64_t)need);
    }
    st = o.disjoint();
    if (st != PTOC_OK) return st;
    if (rows == 0 || cols == 0) {
        // no elements: the sums over them are zero
        const size_t column_bytes = (size_t)cols * 4, row_bytes = (size_t)rows * 4;
        const size_t gate_bytes = p.gate_kind == kGateScalar ? 4 : p.gate_kind == kGateChannel ? column_bytes
                                                                 : p.gate_kind == kGateToken   ? row_bytes : 0;
        auto clear = [&](float* sums, size_t bytes) {
            return !sums || !bytes || cudaMemsetAsync(sums, 0, bytes, stream) == cudaSuccess;
        };
        return clear(d_pre_weight, column_bytes) && clear(d_post_weight, column_bytes) && clear(d_gate, gate_bytes)
                   ? PTOC_OK : PTOC_ERR_CUDA;
    }
    p.c.access = o.access(cols, eb);
    p.block = sv.block.data;
    p.ld_block = sv.block.ld;
    p.block_ckpt = sv.block_ckpt;
    p.stream = sv.stream.data;
    p.ld_stream = sv.stream.ld;
    p.stream_ckpt = sv.stream_ckpt;
    p.rstd = sv.rstd;
    p.dy = dy->data;
    p.ld_dy = dy->ld;
    if (du) p.du = du->data, p.ld_du = du->ld;
    p.d_residual = d_residual->data;
    p.ld_dres = d_residual->ld;
    p.d_block = d_block->data;
    p.ld_dblk = d_block->ld;
    p.d_pre = d_pre_weight;
    p.d_post = d_post_weight;
    p.d_gate = d_gate;
    p.need_q = d_post_weight || p.gate_kind == kGateChannel;
    p.partial = (float*)workspace;
    p.grid = norm_backward_grid(rows, cols);
    return status_of(launch_block_norm_backward(p, dtype, stream));
}

extern "C" size_t ptoc_moe_few_tokens_workspace(int64_t tokens, int64_t hidden, int64_t inter, int32_t experts,
                                                int32_t top_k)
{
    if (tokens <= 0 || hidden <= 0 || inter <= 0 || experts <= 0 || top_k <= 0) return 0;
    if (tokens > PTOC_MOE_MAX_TOKENS || experts > PTOC_MOE_MAX_EXPERTS || top_k > PTOC_MOE_MAX_TOP_K) return 0;
    if (hidden > INT32_MAX || inter > INT32_MAX) return 0;
    return moe_workspace_bytes(tokens, hidden, inter, experts, top_k);
}

extern "C" ptoc_status ptoc_moe_few_tokens(const ptoc_matrix* x, const ptoc_moe_params* params, const ptoc_matrix* y,
                                           int32_t* ids, float* weights, void* workspace, size_t workspace_bytes,
                                           int64_t tokens, int64_t hidden, int64_t inter, ptoc_dtype dtype,
                                           cudaStream_t stream)
{
    const TraceRange trace("ptoc_moe_few_tokens");
    if (!valid_dtype(dtype)) return PTOC_ERR_INVALID_ARG;
    if (dtype != PTOC_F16 && dtype != PTOC_BF16) return PTOC_ERR_UNSUPPORTED;
    if (!x || !params || !y || tokens < 0 || hidden < 1 || inter < 1) return PTOC_ERR_INVALID_ARG;
    const ptoc_moe_params& q = *params;
    if (!q.router || !q.w_in || !q.w_out) return PTOC_ERR_INVALID_ARG;
    if (q.router_dtype != dtype && q.router_dtype != PTOC_F32) return PTOC_ERR_INVALID_ARG;
    if (q.experts < 1 || q.first_expert < 0 || q.local_experts < 1 || q.local_experts > q.experts - q.first_expert)
        return PTOC_ERR_INVALID_ARG;
    if (q.top_k < 1 || q.top_k > q.experts) return PTOC_ERR_INVALID_ARG;
    if (q.score != PTOC_SCORE_SOFTMAX && q.score != PTOC_SCORE_SIGMOID) return PTOC_ERR_INVALID_ARG;
    if (q.renormalize != 0 && q.renormalize != 1) return PTOC_ERR_INVALID_ARG;
    if (tokens > PTOC_MOE_MAX_TOKENS || q.experts > PTOC_MOE_MAX_EXPERTS || q.top_k > PTOC_MOE_MAX_TOP_K ||
        hidden > INT32_MAX / 2 || inter > INT32_MAX / 4)
        return PTOC_ERR_UNSUPPORTED;
    const int eb = elem_size(dtype);
    Operands o;
    o.rows(true, y->data, y->ld, tokens, hidden, eb, 1);
    o.matrix(false, x, tokens, hidden, eb);
    if ((hidden | inter) & 7) o.vec = false;
    o.rows(false, q.router, hidden, q.experts, hidden, elem_size(q.router_dtype), 16);
    // 2 * inter * local_experts and hidden * local_experts are below 2^41
    o.rows(false, q.w_in, hidden, 2 * inter * q.local_experts, hidden, eb, 16);
    o.rows(false, q.w_out, inter, hidden * q.local_experts, inter, eb, 16);
    o.floats(false, q.bias, q.experts);
    if (ids) {
        if (!aligned(ids, 4)) return PTOC_ERR_INVALID_ARG;
        o.add(true, ids, tokens * q.top_k * 4);
    }
    o.floats(true, weights, tokens * q.top_k);
    if (!o.ok) return PTOC_ERR_INVALID_ARG;
    const size_t need = ptoc_moe_few_tokens_workspace(tokens, hidden, inter, q.experts, q.top_k);
    if (tokens > 0) {
        if (!workspace || workspace_bytes < need || !aligned(workspace, kWsAlign)) return PTOC_ERR_INVALID_ARG;
        o.add(true, workspace, (int64_t)need);
    }
    const ptoc_status st = o.disjoint();
    if (st != PTOC_OK) return st;
    if (tokens == 0) return PTOC_OK;
    MoeParams p;
    memset(&p, 0, sizeof(p));
    p.x = x->data;
    p.ld_x = x->ld;
    p.y = y->data;
    p.ld_y = y->ld;
    p.router = q.router;
    p.w_in = q.w_in;
    p.w_out = q.w_out;
    p.bias = q.bias;
    p.ids = ids;
    p.weights = weights;
    p.ws = (char*)workspace;
    p.hidden = hidden;
    p.inter = inter;
    p.tokens = (int32_t)tokens;
    p.experts = q.experts;
    p.first = q.first_expert;
    p.local = q.local_experts;
    p.top_k = q.top_k;
    p.router_f32 = q.router_dtype == PTOC_F32;
    p.sigmoid = q.score == PTOC_SCORE_SIGMOID;
    p.renormalize = q.renormalize;
    p.scale = q.scale;
    p.vec = o.vec;
    return status_of(launch_moe_few(p, dtype, stream));
}
