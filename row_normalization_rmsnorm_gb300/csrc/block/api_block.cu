// api_block.cu -- C entry points of the block-boundary norm and of the 8-bit
// activation checkpoints: argument checks, then the row kernel and the column
// reductions.
#include "../abi/args.h"
#include "block.h"
#include "ckpt.cuh"

using namespace gb300norm;

namespace {

// The launch-shape caches allocate; nothing may throw through the C ABI.
template <class F>
int guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return cuda_fail(cudaErrorMemoryAllocation);
  }
}

bool fmt_ok(int fmt) { return fmt == NORM_SAVED_E4M3 || fmt == NORM_SAVED_INT8; }

// A checkpoint buffer: M rows of ckpt_row_bytes(N) bytes, `stride` bytes apart.
int check_ckpt(const Mat& m, int64_t M, int64_t N, bool required) {
  if (M == 0) return NORM_OK;
  if (!m.p) return required ? NORM_ERR_NULL : NORM_OK;
  const int64_t rb = ckpt_row_bytes(N);
  if (m.stride < rb) return NORM_ERR_STRIDE;
  if (M - 1 > (INT64_MAX - rb) / m.stride) return NORM_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(m.p) % 16 || m.stride % 16) return NORM_ERR_ALIGN;
  return NORM_OK;
}
Span ckpt_span(const Mat& m, int64_t M, int64_t N, bool out) { return mat_span(m, M, ckpt_row_bytes(N), 1, out, 0); }

int check_shape(int64_t M, int64_t N, int dtype) {
  if (M < 0 || N <= 0 || N > INT32_MAX) return NORM_ERR_SHAPE;
  return elem_size(dtype) ? NORM_OK : NORM_ERR_DTYPE;
}

int check_w(const void* w, int w_dtype) {
  return w && reinterpret_cast<uintptr_t>(w) % (uintptr_t)elem_size(w_dtype) ? NORM_ERR_ALIGN : NORM_OK;
}

// A per-column vector that the aligned-row kernels can take (or none).
bool vec16(const void* v) { return reinterpret_cast<uintptr_t>(v) % 16 == 0; }

// A streamed matrix of elements of es bytes, or (es = 1) of checkpoint rows.
void set_stream(BlockParams& p, int s, const Mat& m, int es) {
  p.in[s] = static_cast<const char*>(m.p);
  p.in_stride[s] = m.stride * es;
  if (m.p && es > 1 && p.in_stride[s] < p.min_stride) p.min_stride = p.in_stride[s];
}

BlockParams base(int64_t M, int64_t N, float offset, float eps, int w_dtype, int fmt, int* status) {
  BlockParams p{};
  p.M = M;
  p.N = (int)N;
  p.R = M;
  p.n_gates = 1;
  p.min_stride = INT64_MAX / (M > 0 ? M : 1);
  p.alpha = p.beta = 1.f;
  p.offset = offset;
  p.eps = eps;
  p.w_code = w_dtype;
  p.fmt = fmt;
  p.status = status;
  p.hold_last = hold_last_hook();
  return p;
}

// ---- the checkpointed forms of the three norms ---------------------------
// kind: 0 RMSNorm, 1 LayerNorm, 2 fused add
int norm_fwd_ckpt(int kind, const Mat& mx, const Mat& mr, const void* w, const void* b, const Mat& my, const Mat& mh,
                  float* mean, float* rstd, const Mat& mq, int fmt, int64_t M, int64_t N, float offset, float eps,
                  int dtype, int w_dtype, cudaStream_t st) {
  RETURN_IF(check_common(M, N, offset, eps, dtype, w_dtype, w));
  if (!fmt_ok(fmt)) return NORM_ERR_DTYPE;
  if (N * elem_size(dtype) > kBlockMaxRowBytes) return NORM_ERR_TOO_LARGE;
  const int es = elem_size(dtype), ews = elem_size(w_dtype);
  RETURN_IF(check_w(b, w_dtype));
  const bool add = kind == 2;
  RETURN_IF(check_mat(mx, M, N, es, true));
  if (add) RETURN_IF(check_mat(mr, M, N, es, true));
  RETURN_IF(check_mat(my, M, N, es, true));
  if (add) RETURN_IF(check_mat(mh, M, N, es, true));
  RETURN_IF(check_ckpt(mq, M, N, true));
  if (M > 0 && !rstd) return NORM_ERR_NULL;
  RETURN_IF(check_vec_f32(rstd));
  RETURN_IF(check_vec_f32(mean));
  const Span sp[] = {mat_span(mx, M, N, es, false, 1), mat_span(mr, M, N, es, false, 1), mat_span(my, M, N, es, true, 1),
                     mat_span(mh, M, N, es, true, 1), vec_span(w, N, ews, false), vec_span(b, N, ews, false),
                     vec_span(mean, M, 4, true), vec_span(rstd, M, 4, true), ckpt_span(mq, M, N, true)};
  RETURN_IF(check_overlaps(sp, 9));
  if (M == 0) return NORM_OK;
  DevInfo di;
  int* status = nullptr;
  RETURN_IF(get_device(&di, &status));
  BlockParams p = base(M, N, offset, eps, w_dtype, fmt, status);
  set_stream(p, SX, mx, es);
  if (add) set_stream(p, SR, mr, es);
  if (add) { p.out_a = static_cast<char*>(const_cast<void*>(mh.p)); p.a_stride = mh.stride * es; }
  p.out_b = static_cast<char*>(const_cast<void*>(my.p));
  p.b_stride = my.stride * es;
  p.hq = static_cast<char*>(const_cast<void*>(mq.p));
  p.q_stride = mq.stride;
  p.w2 = w;
  p.bias = b;
  p.pre = 1;
  p.mean_out = mean;
  p.rs2_out = rstd;
  BlockFlags f;
  f.ln = kind == 1;
  f.norm = kind != 1;
  f.q8 = true;
  f.aligned = row16(mx, M, es) && row16(mr, M, es) && row16(my, M, es) && row16(mh, M, es) && vec16(w) && vec16(b);
  int G = 0;
  return launch_block_fwd(p, dtype, f, di, st, &G);
}

int norm_bwd_ckpt(int kind, const Mat& mdy, const Mat& mdh, const Mat& mq, int fmt, const void* w, const float* rstd,
                  const Mat& mdx, void* dw, void* db, int dw_dtype, void* ws, size_t ws_bytes,
                  int64_t M, int64_t N, float offset, int dtype, int w_dtype, cudaStream_t st) {
  RETURN_IF(check_common(M, N, offset, 0.f, dtype, w_dtype, w));
  if (!fmt_ok(fmt)) return NORM_ERR_DTYPE;
  if (N * elem_size(dtype) > kBlockMaxRowBytes) return NORM_ERR_TOO_LARGE;
  const int es = elem_size(dtype), ews = elem_size(w_dtype);
  const int nbuf = (dw ? 1 : 0) + (db ? 1 : 0);
  if (nbuf && dw_dtype != NORM_F32 && dw_dtype != w_dtype) return NORM_ERR_DTYPE;
  const int dws = nbuf ? elem_size(dw_dtype) : 4;
  for (const void* d : {dw, db})
    if (d && reinterpret_cast<uintptr_t>(d) % (uintptr_t)dws) return NORM_ERR_ALIGN;
  RETURN_IF(check_mat(mdy, M, N, es, true));
  RETURN_IF(check_mat(mdh, M, N, es, false));
  RETURN_IF(check_mat(mdx, M, N, es, true));
  RETURN_IF(check_ckpt(mq, M, N, true));
  if (M > 0 && !rstd) return NORM_ERR_NULL;
  RETURN_IF(check_vec_f32(rstd));
  DevInfo di;
  int* status = nullptr;
  int64_t rows = 0, need = 0;
  if (M == 0) return nbuf ? launch_colreduce(nullptr, dw, nullptr, db, 0, (int)N, dw_dtype, st) : NORM_OK;
  if (nbuf) {
    RETURN_IF(check_workspace_ptr(ws));
    RETURN_IF(get_device(&di, &status));
    rows = partial_rows(M, N, di.sms);
    need = rows * N * 4 * nbuf;
    RETURN_IF(check_workspace(ws, ws_bytes, need));
  }
  const Span sp[] = {mat_span(mdy, M, N, es, false, 1), mat_span(mdh, M, N, es, false, 1), ckpt_span(mq, M, N, false),
                     mat_span(mdx, M, N, es, true, 1), vec_span(w, N, ews, false), vec_span(rstd, M, 4, false),
                     vec_span(dw, N, dws, true), vec_span(db, N, dws, true),
                     vec_span(need ? ws : nullptr, need, 1, true)};
  RETURN_IF(check_overlaps(sp, 9));
  if (!status) RETURN_IF(get_device(&di, &status));
  di.max_partial_rows = rows;
  BlockParams p = base(M, N, offset, 0.f, w_dtype, fmt, status);
  set_stream(p, SDY, mdy, es);
  set_stream(p, SR, mdh, es);
  set_stream(p, SH, mq, 1);
  p.out_a = static_cast<char*>(const_cast<void*>(mdx.p));
  p.a_stride = mdx.stride * es;
  p.w2 = w;
  p.pre = 1;
  p.rs2 = rstd;
  float* wsf = static_cast<float*>(ws);
  p.ws2 = dw ? wsf : nullptr;
  p.ws1 = db ? wsf + (dw ? rows * N : 0) : nullptr;
  BlockFlags f;
  f.ln = kind == 1;
  f.norm = kind != 1;
  f.q8 = true;
  f.acc = nbuf > 0;
  f.aligned = row16(mdy, M, es) && row16(mdh, M, es) && row16(mdx, M, es) && vec16(w);
  int G = 0;
  RETURN_IF(launch_block_bwd(p, dtype, f, di, st, &G));
  if (nbuf) return launch_colreduce(p.ws2, dw, p.ws1, db, G, (int)N, dw_dtype, st);
  return NORM_OK;
}

// ---- the gate's arguments -------------------------------------------------
// used: the gate rows of a call with rows (the gate has exactly those).
int check_gate(const Mat& mg, int64_t gate_rows, int64_t R, int64_t M, int64_t N, int gate_dtype, int dtype,
               int w_dtype, int64_t* used) {
  *used = 0;
  if (!mg.p) return NORM_OK;
  if (gate_rows < 1 || R < 1) return NORM_ERR_SHAPE;
  if (gate_dtype != dtype && !(gate_rows == 1 && gate_dtype == w_dtype)) return NORM_ERR_DTYPE;
  *used = M == 0 ? 0 : (M - 1) / R + 1;
  if (M > 0 && *used != gate_rows) return NORM_ERR_SHAPE;
  return check_mat(mg, gate_rows, N, elem_size(gate_dtype), true);
}

// Partial rows of the block backward's workspace: those of the other norms, but 20
// an SM for rows of a single warp, whose row groups can be that many.
int64_t block_partial_rows(int64_t M, int64_t N, int sms) {
  const int64_t cap = 20 * (int64_t)sms;
  return N > 512 ? partial_rows(M, N, sms) : M < cap ? M : cap;
}

int64_t block_ws_rows(int64_t used, int64_t M, int has_w1, int has_w2, int has_dg) {
  const bool streamed = used > 1 && used == M;
  return (has_w1 ? 1 : 0) + (has_w2 ? 1 : 0) + (has_dg && used && !streamed ? 2 : 0);
}

cudaStream_t cs(gb300norm_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

int norm_ckpt_row_bytes(int64_t N, size_t* bytes) {
  if (!bytes) return NORM_ERR_NULL;
  if (N <= 0 || N > INT32_MAX) return NORM_ERR_SHAPE;
  *bytes = (size_t)ckpt_row_bytes(N);
  return NORM_OK;
}

int norm_ckpt_encode(const void* x, int64_t x_stride, void* ckpt, int64_t ckpt_stride, int format, int64_t M, int64_t N,
                     int dtype, gb300norm_stream_t stream) {
  RETURN_IF(check_shape(M, N, dtype));
  if (!fmt_ok(format)) return NORM_ERR_DTYPE;
  const int es = elem_size(dtype);
  const Mat mx{x, x_stride}, mq{ckpt, ckpt_stride};
  RETURN_IF(check_mat(mx, M, N, es, true));
  RETURN_IF(check_ckpt(mq, M, N, true));
  const Span sp[] = {mat_span(mx, M, N, es, false, 0), ckpt_span(mq, M, N, true)};
  RETURN_IF(check_overlaps(sp, 2));
  if (M == 0) return NORM_OK;
  DevInfo di;
  RETURN_IF(get_device(&di, nullptr));
  return launch_ckpt_encode(static_cast<const char*>(x), x_stride * es, static_cast<char*>(ckpt), ckpt_stride, M, N,
                            format, dtype, di, cs(stream));
}

int norm_ckpt_decode(const void* ckpt, int64_t ckpt_stride, int format, void* x, int64_t x_stride, int64_t M, int64_t N,
                     int dtype, gb300norm_stream_t stream) {
  RETURN_IF(check_shape(M, N, dtype));
  if (!fmt_ok(format)) return NORM_ERR_DTYPE;
  const int es = elem_size(dtype);
  const Mat mx{x, x_stride}, mq{ckpt, ckpt_stride};
  RETURN_IF(check_mat(mx, M, N, es, true));
  RETURN_IF(check_ckpt(mq, M, N, true));
  const Span sp[] = {mat_span(mx, M, N, es, true, 0), ckpt_span(mq, M, N, false)};
  RETURN_IF(check_overlaps(sp, 2));
  if (M == 0) return NORM_OK;
  DevInfo di;
  RETURN_IF(get_device(&di, nullptr));
  return launch_ckpt_decode(static_cast<const char*>(ckpt), ckpt_stride, static_cast<char*>(x), x_stride * es, M, N,
                            format, dtype, di, cs(stream));
}

int norm_rms_fwd_ckpt(const void* x, int64_t x_stride, const void* w, void* y, int64_t y_stride, float* rstd, void* ckpt,
                      int64_t ckpt_stride, int format, int64_t M, int64_t N, float offset, float eps, int dtype,
                      int w_dtype, gb300norm_stream_t stream) {
  return guarded([&] {
    return norm_fwd_ckpt(0, {x, x_stride}, {nullptr, 0}, w, nullptr, {y, y_stride}, {nullptr, 0}, nullptr, rstd,
                         {ckpt, ckpt_stride}, format, M, N, offset, eps, dtype, w_dtype, cs(stream));
  });
}

int norm_rms_bwd_ckpt(const void* dy, int64_t dy_stride, const void* ckpt, int64_t ckpt_stride, int format,
                      const void* w, const float* rstd, void* dx, int64_t dx_stride, void* dw, int dw_dtype,
                      void* workspace, size_t workspace_bytes, int64_t M, int64_t N, float offset, int dtype,
                      int w_dtype, gb300norm_stream_t stream) {
  return guarded([&] {
    return norm_bwd_ckpt(0, {dy, dy_stride}, {nullptr, 0}, {ckpt, ckpt_stride}, format, w, rstd,
                         {dx, dx_stride}, dw, nullptr, dw_dtype, workspace, workspace_bytes, M, N, offset, dtype, w_dtype,
                         cs(stream));
  });
}

int norm_ln_fwd_ckpt(const void* x, int64_t x_stride, const void* w, const void* b, void* y, int64_t y_stride,
                     float* mean, float* rstd, void* ckpt, int64_t ckpt_stride, int format, int64_t M, int64_t N,
                     float offset, float eps, int dtype, int w_dtype, gb300norm_stream_t stream) {
  return guarded([&] {
    return norm_fwd_ckpt(1, {x, x_stride}, {nullptr, 0}, w, b, {y, y_stride}, {nullptr, 0}, mean, rstd,
                         {ckpt, ckpt_stride}, format, M, N, offset, eps, dtype, w_dtype, cs(stream));
  });
}

int norm_ln_bwd_ckpt(const void* dy, int64_t dy_stride, const void* ckpt, int64_t ckpt_stride, int format, const void* w,
                     const float* rstd, void* dx, int64_t dx_stride, void* dw, void* db, int dw_dtype,
                     void* workspace, size_t workspace_bytes, int64_t M, int64_t N, float offset, int dtype, int w_dtype,
                     gb300norm_stream_t stream) {
  return guarded([&] {
    return norm_bwd_ckpt(1, {dy, dy_stride}, {nullptr, 0}, {ckpt, ckpt_stride}, format, w, rstd, {dx, dx_stride},
                         dw, db, dw_dtype, workspace, workspace_bytes, M, N, offset, dtype, w_dtype, cs(stream));
  });
}

int norm_fused_add_rms_fwd_ckpt(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                const void* w, void* y, int64_t y_stride, void* h_out, int64_t h_stride, float* rstd,
                                void* ckpt, int64_t ckpt_stride, int format, int64_t M, int64_t N, float offset,
                                float eps, int dtype, int w_dtype, gb300norm_stream_t stream) {
  return guarded([&] {
    return norm_fwd_ckpt(2, {x, x_stride}, {residual, residual_stride}, w, nullptr, {y, y_stride}, {h_out, h_stride},
                         nullptr, rstd, {ckpt, ckpt_stride}, format, M, N, offset, eps, dtype, w_dtype, cs(stream));
  });
}

int norm_fused_add_rms_bwd_ckpt(const void* dy, int64_t dy_stride, const void* dh_out, int64_t dh_stride,
                                const void* ckpt, int64_t ckpt_stride, int format, const void* w, const float* rstd,
                                void* dx, int64_t dx_stride, void* dw, int dw_dtype, void* workspace,
                                size_t workspace_bytes, int64_t M, int64_t N, float offset, int dtype, int w_dtype,
                                gb300norm_stream_t stream) {
  return guarded([&] {
    return norm_bwd_ckpt(2, {dy, dy_stride}, {dh_out, dh_stride}, {ckpt, ckpt_stride}, format, w, rstd,
                         {dx, dx_stride}, dw, nullptr, dw_dtype, workspace, workspace_bytes, M, N, offset, dtype, w_dtype,
                         cs(stream));
  });
}

int norm_block_bwd_workspace_bytes(int64_t M, int64_t N, int64_t gate_rows, int has_dw_post, int has_dw_pre,
                                   int has_dgate, size_t* bytes) {
  if (!bytes) return NORM_ERR_NULL;
  if (M < 0 || N <= 0 || N > INT32_MAX || (has_dgate && gate_rows < 1)) return NORM_ERR_SHAPE;
  const int64_t nbuf = block_ws_rows(gate_rows, M, has_dw_post, has_dw_pre, has_dgate);
  if (M == 0 || nbuf == 0) { *bytes = 0; return NORM_OK; }
  DevInfo di;
  RETURN_IF(get_device(&di, nullptr));
  *bytes = (size_t)(block_partial_rows(M, N, di.sms) * N * 4 * nbuf);
  return NORM_OK;
}

int norm_block_rms_fwd(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                       const void* w_post, const void* w_pre, const void* gate, int64_t gate_stride, int64_t gate_rows,
                       int64_t rows_per_gate, void* y, int64_t y_stride, void* h_out, int64_t h_stride, float* rstd_post,
                       float* rstd_pre, void* x_ckpt, void* h_ckpt, int64_t ckpt_stride, int ckpt_format, int64_t M,
                       int64_t N, float residual_scale, float block_scale, float offset, float eps, int dtype,
                       int w_dtype, int gate_dtype, gb300norm_stream_t stream) {
  return guarded([&]() -> int {
    RETURN_IF(check_common(M, N, offset, eps, dtype, w_dtype, w_post ? w_post : w_pre));
    RETURN_IF(check_w(w_pre, w_dtype));
    if (!finite(residual_scale) || !finite(block_scale)) return NORM_ERR_VALUE;
    if (N * elem_size(dtype) > kBlockMaxRowBytes) return NORM_ERR_TOO_LARGE;
    const bool q8 = x_ckpt || h_ckpt;
    if (q8 && ckpt_format == NORM_SAVED_FULL) return NORM_ERR_ARG;
    if (ckpt_format != NORM_SAVED_FULL && !fmt_ok(ckpt_format)) return NORM_ERR_DTYPE;
    if (M > 0 && ((w_pre != nullptr) != (y != nullptr) || (!y && !h_out))) return NORM_ERR_ARG;
    if ((rstd_post && !w_post) || (rstd_pre && !w_pre) || (h_ckpt && !w_pre) || (x_ckpt && !w_post && !gate))
      return NORM_ERR_ARG;
    const int es = elem_size(dtype), ews = elem_size(w_dtype), ges = elem_size(gate_dtype);
    const Mat mx{x, x_stride}, mr{residual, residual_stride}, my{y, y_stride}, mh{h_out, h_stride}, mg{gate, gate_stride};
    const Mat mqx{x_ckpt, ckpt_stride}, mqh{h_ckpt, ckpt_stride};
    int64_t used = 0;
    RETURN_IF(check_mat(mx, M, N, es, true));
    RETURN_IF(check_mat(mr, M, N, es, true));
    RETURN_IF(check_mat(my, M, N, es, false));
    RETURN_IF(check_mat(mh, M, N, es, false));
    RETURN_IF(check_gate(mg, gate_rows, rows_per_gate, M, N, gate_dtype, dtype, w_dtype, &used));
    RETURN_IF(check_ckpt(mqx, M, N, false));
    RETURN_IF(check_ckpt(mqh, M, N, false));
    RETURN_IF(check_vec_f32(rstd_post));
    RETURN_IF(check_vec_f32(rstd_pre));
    const Span sp[] = {mat_span(mx, M, N, es, false, 1), mat_span(mr, M, N, es, false, 1),
                       mat_span(my, M, N, es, true, 1), mat_span(mh, M, N, es, true, 1),
                       gate ? mat_span(mg, gate_rows, N, ges, false, 0) : Span(),
                       vec_span(w_post, N, ews, false), vec_span(w_pre, N, ews, false),
                       vec_span(rstd_post, M, 4, true), vec_span(rstd_pre, M, 4, true),
                       ckpt_span(mqx, M, N, true), ckpt_span(mqh, M, N, true)};
    RETURN_IF(check_overlaps(sp, 11));
    if (M == 0) return NORM_OK;
    DevInfo di;
    int* status = nullptr;
    RETURN_IF(get_device(&di, &status));
    BlockParams p = base(M, N, offset, eps, w_dtype, ckpt_format, status);
    p.alpha = residual_scale;
    p.beta = block_scale;
    set_stream(p, SX, mx, es);
    set_stream(p, SR, mr, es);
    BlockFlags f;
    f.grow = used > 1;
    if (f.grow) {
      set_stream(p, SG, mg, es);
      p.R = rows_per_gate;
      p.n_gates = gate_rows;
    } else if (used == 1) {
      p.gate = gate;
      p.gate_code = gate_dtype;
    }
    p.out_a = static_cast<char*>(h_out);
    p.a_stride = h_stride * es;
    p.out_b = static_cast<char*>(y);
    p.b_stride = y_stride * es;
    p.xq = static_cast<char*>(x_ckpt);
    p.hq = static_cast<char*>(h_ckpt);
    p.q_stride = ckpt_stride;
    p.w1 = w_post;
    p.w2 = w_pre;
    p.post = w_post != nullptr;
    p.pre = w_pre != nullptr;
    p.rs1_out = rstd_post;
    p.rs2_out = rstd_pre;
    f.q8 = q8;
    f.aligned = row16(mx, M, es) && row16(mr, M, es) && row16(my, M, es) && row16(mh, M, es) &&
                row16(mg, gate_rows, ges) && vec16(w_post) && vec16(w_pre);
    int G = 0;
    return launch_block_fwd(p, dtype, f, di, cs(stream), &G);
  });
}

int norm_block_rms_bwd(const void* dy, int64_t dy_stride, const void* dh_out, int64_t dh_stride, const void* x,
                       int64_t x_stride, const void* h, int64_t h_stride, int saved_format, const void* w_post,
                       const void* w_pre, const float* rstd_post, const float* rstd_pre, const void* gate,
                       int64_t gate_stride, int64_t gate_rows, int64_t rows_per_gate, void* dx, int64_t dx_stride,
                       void* dresidual, int64_t dresidual_stride, void* dgate, int64_t dgate_stride, void* dw_post,
                       void* dw_pre, int dw_dtype, void* workspace, size_t workspace_bytes, int64_t M, int64_t N,
                       float residual_scale, float block_scale, float offset, int dtype, int w_dtype, int gate_dtype,
                       gb300norm_stream_t stream) {
  return guarded([&]() -> int {
    RETURN_IF(check_common(M, N, offset, 0.f, dtype, w_dtype, w_post ? w_post : w_pre));
    RETURN_IF(check_w(w_pre, w_dtype));
    if (!finite(residual_scale) || !finite(block_scale)) return NORM_ERR_VALUE;
    if (N * elem_size(dtype) > kBlockMaxRowBytes) return NORM_ERR_TOO_LARGE;
    const bool q8 = saved_format != NORM_SAVED_FULL;
    if (q8 && !fmt_ok(saved_format)) return NORM_ERR_DTYPE;
    const bool need_x = w_post || dgate;
    if ((dw_post && !w_post) || (dw_pre && !w_pre) || (dgate && !gate)) return NORM_ERR_ARG;
    if (M > 0 && ((w_pre != nullptr) != (dy != nullptr))) return NORM_ERR_ARG;
    if (M > 0 && ((w_post && !rstd_post) || (w_pre && !rstd_pre) || (!w_pre && !dh_out))) return NORM_ERR_NULL;
    const int es = elem_size(dtype), ews = elem_size(w_dtype), ges = elem_size(gate_dtype);
    if ((dw_post || dw_pre) && dw_dtype != NORM_F32 && dw_dtype != w_dtype) return NORM_ERR_DTYPE;
    const int dws = dw_post || dw_pre ? elem_size(dw_dtype) : 4;
    for (const void* d : {dw_post, dw_pre})
      if (d && reinterpret_cast<uintptr_t>(d) % (uintptr_t)dws) return NORM_ERR_ALIGN;
    const Mat mdy{dy, dy_stride}, mdh{dh_out, dh_stride}, mx{need_x ? x : nullptr, x_stride},
        mh{w_pre ? h : nullptr, h_stride}, mg{gate, gate_stride}, mdx{dx, dx_stride}, mdr{dresidual, dresidual_stride},
        mdg{dgate, dgate_stride};
    int64_t used = 0;
    RETURN_IF(check_mat(mdy, M, N, es, false));
    RETURN_IF(check_mat(mdh, M, N, es, false));
    RETURN_IF(q8 ? check_ckpt(mx, M, N, need_x) : check_mat(mx, M, N, es, need_x));
    RETURN_IF(q8 ? check_ckpt(mh, M, N, w_pre != nullptr) : check_mat(mh, M, N, es, w_pre != nullptr));
    RETURN_IF(check_mat(mdx, M, N, es, false));
    RETURN_IF(check_mat(mdr, M, N, es, false));
    RETURN_IF(check_gate(mg, gate_rows, rows_per_gate, M, N, gate_dtype, dtype, w_dtype, &used));
    if (dgate) RETURN_IF(check_mat(mdg, gate_rows, N, ges, true));
    RETURN_IF(check_vec_f32(rstd_post));
    RETURN_IF(check_vec_f32(rstd_pre));
    const bool streamed = used > 1 && used == M;   // a gate row for every row
    const int64_t nbuf = block_ws_rows(used, M, dw_post != nullptr, dw_pre != nullptr, dgate != nullptr);
    DevInfo di;
    int* status = nullptr;
    int64_t rows = 0, need = 0;
    if (nbuf && M > 0) {
      RETURN_IF(check_workspace_ptr(workspace));
      RETURN_IF(get_device(&di, &status));
      rows = block_partial_rows(M, N, di.sms);
      need = rows * N * 4 * nbuf;
      RETURN_IF(check_workspace(workspace, workspace_bytes, need));
    }
    auto saved = [&](const Mat& m) { return q8 ? ckpt_span(m, M, N, false) : mat_span(m, M, N, es, false, 0); };
    const Span sp[] = {mat_span(mdy, M, N, es, false, 1), mat_span(mdh, M, N, es, false, 1), saved(mx), saved(mh),
                       vec_span(w_post, N, ews, false), vec_span(w_pre, N, ews, false),
                       vec_span(rstd_post, M, 4, false), vec_span(rstd_pre, M, 4, false),
                       gate ? mat_span(mg, gate_rows, N, ges, false, 0) : Span(), mat_span(mdx, M, N, es, true, 1),
                       mat_span(mdr, M, N, es, true, 1), dgate ? mat_span(mdg, gate_rows, N, ges, true, 0) : Span(),
                       vec_span(dw_post, N, dws, true), vec_span(dw_pre, N, dws, true),
                       vec_span(need ? workspace : nullptr, need, 1, true)};
    RETURN_IF(check_overlaps(sp, 15));
    if (!status) RETURN_IF(get_device(&di, &status));
    cudaStream_t st = cs(stream);
    BlockParams p = base(M, N, offset, 0.f, w_dtype, saved_format, status);
    p.dg = static_cast<char*>(dgate);
    p.dg_stride = dgate_stride * ges;
    p.gate_code = gate_dtype;
    p.n_gates = gate_rows;
    if (gate) p.R = rows_per_gate;
    int G = 0;
    if (M > 0) {
      di.max_partial_rows = rows;
      p.alpha = residual_scale;
      p.beta = block_scale;
      set_stream(p, SDY, mdy, es);
      set_stream(p, SR, mdh, es);
      set_stream(p, SX, mx, q8 ? 1 : es);
      set_stream(p, SH, mh, q8 ? 1 : es);
      p.room_x = gate != nullptr;   // x is read for its norm's gradients, else for the gate's alone
      if (streamed) {
        set_stream(p, SG, mg, es);
      } else {
        p.gate = gate;
        p.gate_stride = gate_stride;
        p.seg = used > 1;
      }
      p.out_a = static_cast<char*>(dresidual);
      p.a_stride = dresidual_stride * es;
      p.out_b = static_cast<char*>(dx);
      p.b_stride = dx_stride * es;
      p.w1 = w_post;
      p.w2 = w_pre;
      p.post = w_post != nullptr;
      p.pre = w_pre != nullptr;
      p.rs1 = rstd_post;
      p.rs2 = rstd_pre;
      float* wsf = static_cast<float*>(workspace);
      auto take = [&](bool want) {
        float* r = want ? wsf : nullptr;
        if (want) wsf += rows * N;
        return r;
      };
      p.ws1 = take(dw_post);
      p.ws2 = take(dw_pre);
      p.ws_head = take(dgate && !streamed);
      p.ws_tail = take(dgate && !streamed);
      BlockFlags f;
      f.grow = streamed;
      f.q8 = q8;
      f.acc = nbuf > 0;
      f.aligned = row16(mdy, M, es) && row16(mdh, M, es) && (q8 || (row16(mx, M, es) && row16(mh, M, es))) &&
                  row16(mdx, M, es) && row16(mdr, M, es) && row16(mg, gate_rows, ges) && row16(mdg, gate_rows, ges) &&
                  vec16(w_post) && vec16(w_pre);
      RETURN_IF(launch_block_bwd(p, dtype, f, di, st, &G));
    }
    // With a gate of fewer rows than M, its sums and the weights' in one launch
    // (8192 x 5120, a scale per channel: 2 us less than in two); without, the
    // weights' by the column reduction of the other norms, whose cluster form is
    // faster with many partial rows (backward 8192 x 2048: 45.2 against 49.0 us).
    // Neither which one nor the launch shape (room_x) depends on the gradients
    // wanted, so their bits do not (unless one of them, or the x read for it alone,
    // is all that is off 16 bytes: that takes the general form).
    const bool sum_gate = dgate && !streamed;
    if (!sum_gate) p.n_gates = 0;
    if (sum_gate || (gate && !streamed && (dw_post || dw_pre)))
      return launch_block_reduce(p, dw_post, dw_pre, dw_dtype, G, st);
    if (dw_post || dw_pre) return launch_colreduce(p.ws1, dw_post, p.ws2, dw_pre, G, (int)N, dw_dtype, st);
    return NORM_OK;
  });
}

}  // extern "C"
