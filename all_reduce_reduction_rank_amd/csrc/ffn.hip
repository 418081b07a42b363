// ffn.hip -- the gated feed-forward block of a tensor-parallel layer
// (ar_gated_ffn, ar_gated_ffn_backward): the work between the all-reduces
// that the collectives page describes (a column split of the gate and up
// projections, a row split of the down projection, partial sums left over).
//
// Forward, rank r:   g = x Wg^T, u = x Wu^T, h = act(g) u, out = h Wd^T.
//   One launch makes h: its tiles hold the same columns of g and u side by
//   side, so the activation and the product happen in registers.  One more
//   multiplies by Wd.
// Backward:  dh = dout Wd;  dg = dh u act'(g), du = dh act(g);
//            dx = dg Wg + du Wu;  dWg = dg^T x, dWu = du^T x, dWd = dout^T h.
//   dh never reaches memory: the tile that holds it writes dg, du and the
//   h that dWd needs (recomputed from g and u: one store instead of keeping h
//   from the forward pass).  dx is one product with two K segments.  dx and
//   the three weight gradients of every rank are one launch.
//
// Roundings to bf16 beside the stored results: h, dg and du, operands of the
// matrix cores; half a bf16 step of the value each, so that one rounding lies
// between the exact value and a product (none with up to 32 rows, where a
// second term holds what the first one's rounding left, fold_of).  g and u are kept for the backward
// pass in fp32: kept in bf16 they would put two more under every gradient
// (measured against fp64: 0.0035 relative instead of 0.0024, where the
// rounding of the result alone is 0.0017).  Every sum is fp32.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/ar.h"
#include "layer.hpp"
#include "products.hpp"

using namespace ar;

namespace {

struct FfnShape {
  uint64_t rows, hidden, inter, es, pitch;  // pitch: elements per row of h, dg, du (whole chunks)
  uint32_t fold;                            // h, dg, du: rows down to their second terms, 0: none
  uint64_t mid_bytes;                       // one rank's h (dg, du)
  // one rank's copies of x (dout), of w_gate (w_up), of w_down, where their
  // rows are not whole 16-byte chunks
  uint64_t pack_x, pack_up, pack_down;
  uint64_t share;  // one rank's shares of out (dx)
  uint64_t workspace(int n, bool backward) const {
    return (uint64_t)n * ((backward ? 3 : 1) * mid_bytes + share + (backward ? 2 : 1) * pack_x + 2 * pack_up + pack_down);
  }
};

FfnShape shape_of(int n, size_t rows, size_t hidden, size_t inter, int dtype) {
  FfnShape s;
  s.rows = rows, s.hidden = hidden, s.inter = inter;
  s.es = dtype == DT_BF16 ? 2 : 4;
  s.pitch = Packer::pitch(inter, s.es);
  s.fold = fold_of(rows, dtype);
  s.mid_bytes = layer_align((s.fold + s.rows) * s.pitch * s.es);
  s.share = share_bytes(n, rows, hidden);
  s.pack_x = Packer::bytes(rows, hidden, s.es);
  s.pack_up = Packer::bytes(inter, hidden, s.es);
  s.pack_down = Packer::bytes(hidden, inter, s.es);
  return s;
}

ar_status check_shape(int n, size_t rows, size_t hidden, size_t inter, int act, int dtype) {
  if (n < 1 || n > MAX_RANKS || dtype < 0 || dtype > 2 || act < 0 || act > 2) return AR_ERR_INVALID;
  if (hidden < 1 || inter < 1) return AR_ERR_INVALID;
  if (dtype == DT_I32) return AR_ERR_UNSUPPORTED;
  if (rows > LAYER_MAX_ROWS || hidden > LAYER_MAX_WIDTH || inter > LAYER_MAX_WIDTH) return AR_ERR_TOO_LARGE;
  return AR_OK;
}

}  // namespace

extern "C" {

size_t ar_gated_ffn_workspace(int nranks, size_t rows, size_t hidden, size_t inter, ar_dtype dtype, int backward) {
  if (check_shape(nranks, rows, hidden, inter, 0, (int)dtype) != AR_OK || rows == 0) return 0;
  return (size_t)shape_of(nranks, rows, hidden, inter, (int)dtype).workspace(nranks, backward != 0);
}

ar_status ar_gated_ffn(int nranks, const void* const* x, const void* const* w_gate, const void* const* w_up,
                       const void* const* w_down, void* const* out, void* const* gate, void* const* up, size_t rows,
                       size_t hidden, size_t inter, ar_act act, ar_dtype dtype, void* workspace,
                       size_t workspace_bytes, ar_stream_t stream) {
  const ar_status st = check_shape(nranks, rows, hidden, inter, (int)act, (int)dtype);
  if (st != AR_OK) return st;
  if (!x || !w_gate || !w_up || !w_down || !out || !gate != !up) return AR_ERR_INVALID;
  if (rows == 0) return AR_OK;
  const FfnShape s = shape_of(nranks, rows, hidden, inter, (int)dtype);
  const uint64_t xb = s.rows * s.hidden * s.es, wb = s.hidden * s.inter * s.es, gb = s.rows * s.inter * 4;
  const uint64_t need = s.workspace(nranks, false);
  LayerBuffers b;
  for (int r = 0; r < nranks; ++r) {
    b.in(x[r], xb);
    b.in(w_gate[r], wb);
    b.in(w_up[r], wb);
    b.in(w_down[r], wb);
    b.out(out[r], xb);
    if (gate) b.out(gate[r], gb);
    if (up) b.out(up[r], gb);
  }
  b.out(workspace, need);
  if (!b.ok()) return AR_ERR_INVALID;
  if (workspace_bytes < need) return AR_ERR_TOO_LARGE;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return AR_ERR_HIP;
  char* ws = (char*)workspace;
  auto h = [&](int r) { return ws + (uint64_t)r * s.mid_bytes; };

  ProductPlan up_plan, down_plan;
  up_plan.a.act = (int32_t)act;
  char* shares = ws + (uint64_t)nranks * s.mid_bytes;
  down_plan.may_share = s.share != 0;
  Packer pack(shares + (uint64_t)nranks * s.share, s.es);
  for (int r = 0; r < nranks; ++r) {
    const Packer::Rows px = pack.rows(x[r], s.rows, s.hidden), pg = pack.rows(w_gate[r], s.inter, s.hidden),
                       pu = pack.rows(w_up[r], s.inter, s.hidden), pd = pack.rows(w_down[r], s.hidden, s.inter);
    Problem* p = up_plan.add(s.rows, s.inter, s.hidden, px.ld, pg.ld, s.pitch);
    p->a[0] = px.p;
    p->b[0] = pg.p;
    p->b[1] = pu.p;
    p->fold = s.fold;
    p->c[0] = h(r);
    p->c[1] = gate ? (char*)gate[r] : nullptr;
    p->c[2] = up ? (char*)up[r] : nullptr;
    p = down_plan.add(s.fold + s.rows, s.hidden, s.inter, s.pitch, pd.ld, s.hidden);
    p->fold = s.fold;
    p->a[0] = h(r);
    p->b[0] = pd.p;
    p->c[0] = (char*)out[r];
    p->c[2] = shares + (uint64_t)r * s.share;
  }
  if (pack.launch((hipStream_t)stream) != hipSuccess) return AR_ERR_HIP;
  if (launch_products(PK_GATED, (int)dtype, up_plan, dev, (hipStream_t)stream) != hipSuccess) return AR_ERR_HIP;
  if (launch_products(PK_STORE_NT, (int)dtype, down_plan, dev, (hipStream_t)stream) != hipSuccess) return AR_ERR_HIP;
  return AR_OK;
}

ar_status ar_gated_ffn_backward(int nranks, const void* const* dout, const void* const* x, const void* const* w_gate,
                                const void* const* w_up, const void* const* w_down, const void* const* gate,
                                const void* const* up, void* const* dx, void* const* dw_gate, void* const* dw_up,
                                void* const* dw_down, size_t rows, size_t hidden, size_t inter, ar_act act,
                                ar_dtype dtype, void* workspace, size_t workspace_bytes, ar_stream_t stream) {
  const ar_status st = check_shape(nranks, rows, hidden, inter, (int)act, (int)dtype);
  if (st != AR_OK) return st;
  if (!dout || !x || !w_gate || !w_up || !w_down || !gate || !up || !dx || !dw_gate || !dw_up || !dw_down)
    return AR_ERR_INVALID;
  const FfnShape s = shape_of(nranks, rows, hidden, inter, (int)dtype);
  const uint64_t xb = s.rows * s.hidden * s.es, wb = s.hidden * s.inter * s.es, gb = s.rows * s.inter * 4;
  const uint64_t need = rows ? s.workspace(nranks, true) : 0;
  LayerBuffers b;
  for (int r = 0; r < nranks; ++r) {
    b.in(dout[r], xb);
    b.in(x[r], xb);
    b.in(w_gate[r], wb);
    b.in(w_up[r], wb);
    b.in(w_down[r], wb);
    b.in(gate[r], gb);
    b.in(up[r], gb);
    b.out(dx[r], xb);
    b.out(dw_gate[r], wb);
    b.out(dw_up[r], wb);
    b.out(dw_down[r], wb);
  }
  b.out(workspace, need);
  if (!b.ok()) return AR_ERR_INVALID;
  if (workspace_bytes < need) return AR_ERR_TOO_LARGE;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return AR_ERR_HIP;
  char* ws = (char*)workspace;
  auto mid = [&](int r, int i) { return ws + ((uint64_t)r * 3 + i) * s.mid_bytes; };  // dg, du, h

  ProductPlan mid_plan, grads;
  mid_plan.a.act = (int32_t)act;
  char* shares = ws + (uint64_t)nranks * 3 * s.mid_bytes;
  grads.may_share = s.share != 0;
  Packer pack(shares + (uint64_t)nranks * s.share, s.es);
  Packer::Rows px[MAX_RANKS], po[MAX_RANKS];
  for (int r = 0; r < nranks; ++r) {
    // (with no rows nothing is read, and nothing copied)
    const uint64_t some = rows ? 1 : 0;
    px[r] = pack.rows(x[r], s.rows, s.hidden);
    po[r] = pack.rows(dout[r], s.rows, s.hidden);
    const Packer::Rows pg = pack.rows(w_gate[r], some * s.inter, s.hidden),
                       pu = pack.rows(w_up[r], some * s.inter, s.hidden),
                       pd = pack.rows(w_down[r], some * s.hidden, s.inter);
    Problem* p = mid_plan.add(s.rows, s.inter, s.hidden, po[r].ld, pd.ld, s.pitch);
    p->a[0] = po[r].p;
    p->b[0] = pd.p;
    p->a[1] = (const char*)gate[r];
    p->b[1] = (const char*)up[r];
    for (int i = 0; i < 3; ++i) p->c[i] = mid(r, i);
    p->fold = s.fold;
    p = grads.add(s.fold + s.rows, s.hidden, s.inter, s.pitch, pg.ld, s.hidden);
    p->fold = s.fold;
    p->nseg = 2;
    p->a[0] = mid(r, 0);
    p->a[1] = mid(r, 1);
    p->b[0] = pg.p;
    p->b[1] = pu.p;
    p->c[0] = (char*)dx[r];
    p->c[2] = shares + (uint64_t)r * s.share;
  }
  grads.head = nranks;
  // With no rows every weight gradient is a product with k = 0: zeros.  The
  // second terms of dg, du and h, where there are any, are a second segment.
  const uint64_t low = s.fold * s.pitch * s.es;
  for (int r = 0; r < nranks; ++r) {
    Problem* p;
    for (int i = 0; i < 2; ++i) {
      p = grads.add(s.inter, s.hidden, s.rows, s.pitch, px[r].ld, s.hidden);
      p->nseg = s.fold ? 2 : 1;
      p->a[0] = mid(r, i);
      p->a[1] = mid(r, i) + low;
      p->b[0] = p->b[1] = px[r].p;
      p->c[0] = (char*)(i ? dw_up[r] : dw_gate[r]);
      p->mode = GRAD_TN;
    }
    p = grads.add(s.hidden, s.inter, s.rows, po[r].ld, s.pitch, s.inter);
    p->nseg = s.fold ? 2 : 1;
    p->a[0] = p->a[1] = po[r].p;
    p->b[0] = mid(r, 2);
    p->b[1] = mid(r, 2) + low;
    p->c[0] = (char*)dw_down[r];
    p->mode = GRAD_TN;
  }
  if (pack.launch((hipStream_t)stream) != hipSuccess ||
      launch_products(PK_GATED_BWD, (int)dtype, mid_plan, dev, (hipStream_t)stream) != hipSuccess ||
      launch_grads((int)dtype, grads, dev, (hipStream_t)stream) != hipSuccess)
    return AR_ERR_HIP;
  return AR_OK;
}

}  // extern "C"
