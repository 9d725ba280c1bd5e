// The operators around the state update: linear attention with one decay per head,
// RMS norm, products with 4-bit weights. C entry points (include/muir.h): each
// validates its arguments, sizes workspaces and launches the kernels.
#include "../../include/muir.h"
#include "host.h"
#include "lin_attn.cuh"
#include "lin_attn_tc.cuh"
#include "rms_norm.cuh"
#include "w4.cuh"

namespace muir_host {
bool take_layer_status(unsigned int* word) {
  const unsigned int zero = 0;
  return cudaMemcpyFromSymbol(word, muir::g_status, sizeof *word) == cudaSuccess &&
         cudaMemcpyToSymbol(muir::g_status, &zero, sizeof zero) == cudaSuccess;
}
}  // namespace muir_host

namespace {

using bf16 = __nv_bfloat16;
using muir_host::check_launch;
using muir_host::fail;
using muir_host::LaunchScope;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool dtype_ok(int t) { return t == MUIR_F32 || t == MUIR_BF16; }
constexpr int64_t kMaxBlocks = 0x7fffffff;
constexpr int kSMs = 148;

// Every pointer set and 16-byte aligned (optional ones may be NULL).
struct Ptr {
  const void* p;
  const char* name;
  bool optional = false;
};
template <size_t N>
int check_ptrs(const char* who, const Ptr (&ptrs)[N]) {
  for (const Ptr& q : ptrs) {
    if (!q.p && !q.optional) return fail(MUIR_ERR_INVALID_ARG, "%s: %s is NULL", who, q.name);
    if (!aligned(q.p, 16)) return fail(MUIR_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", who, q.name);
  }
  return MUIR_OK;
}

// ---- linear attention -----------------------------------------------------------

struct LinPlan {
  bool tc;  // the tensor-core pass
  int nseg;
  int64_t seglen;
};

// bf16 operands go to the tensor cores, fp32 ones to the CUDA cores (one bf16
// rounding of the weights would be all of fp32's accuracy). A box of the copies
// covers 64 channels, so a token row has at least that many. Few tokens are no
// exception, so that a short sequence's result is the same in every batch; they are no
// faster on the CUDA cores (in a graph, forward of 16 tokens, 16 heads of 64: 8.6 us on
// the CUDA cores, 8.5 on the tensor cores; of 128, 12.9 and 11.2; one token of 64, 8.1 and
// 8.5; a call outside a graph encodes four tensor maps for it, 14.9 and 15.4 us).
bool lin_use_tc(const muir_lin_args* a) {
  return a->dtype == MUIR_BF16 && a->T > 0 && (int64_t)a->H * a->dk >= 64 && (int64_t)a->H * a->dv >= 64;
}

// Segments of the sequence, for `outs` passes of outputs (in one launch) and `states`
// passes of segment states (in another, where there is more than one segment).
//
// Tensor cores, one CTA per SM: the split with the least cost, in times of a chunk of
// outputs: the waves of CTAs times their chunks and a start worth 2 chunks, a chunk
// of the segments' own states counting 0.55 (2.0 against 3.9 us at d = 128), and the
// walk over the segments. One sequence of 32768 tokens and 16 heads: 9 segments, one
// wave each, in the forward pass; the backward's 432 and 288 CTAs of 9 segments (3
// and 2 waves) take 130 units, 144 and 96 CTAs of 3 segments 137.
//
// CUDA cores: as many CTAs as fit beside one another, three for each SM up to 64
// channels and two for 128.
LinPlan lin_plan(const muir_lin_args* a, int outs, int states) {
  LinPlan pl{lin_use_tc(a), 1, 0};
  const int64_t run = pl.tc ? muir::kLtChunk : muir::kLinRun;
  const int64_t runs = a->T > 0 ? (a->T + run - 1) / run : 1;
  int64_t n = 1;
  if (pl.tc) {
    const int64_t units = a->B * a->H;
    double best = 0.0;
    for (int64_t c = 1; c <= runs && c <= 1024; ++c) {
      const double chunks = (double)((runs + c - 1) / c);
      const auto waves = [&](int passes) { return (double)((units * passes * c + kSMs - 1) / kSMs); };
      const double cost = waves(outs) * (chunks + 2.0) + (c > 1 ? waves(states) * (0.55 * chunks + 2.0) + 2.0 + 0.1 * (double)c : 0.0);
      if (c == 1 || cost < best) {
        best = cost;
        n = c;
      }
    }
  } else {
    const int dmin = a->dk < a->dv && outs > 1 ? a->dk : a->dv;
    const int64_t units = a->B * a->H * (dmin / 32) * outs;
    const int64_t fit = (a->dk > 64 || (outs > 1 && a->dv > 64) ? 2 : 3) * kSMs;
    n = (fit + units - 1) / units;
    if (n > runs) n = runs;
    if (n < 1) n = 1;
  }
  const int64_t per = (runs + n - 1) / n;
  pl.nseg = (int)((runs + per - 1) / per);
  pl.seglen = per * run;
  return pl;
}

int lin_validate(const muir_lin_args* a, const char* who) {
  if (!a) return fail(MUIR_ERR_INVALID_ARG, "%s: args is NULL", who);
  if (a->B < 0 || a->T < 0) return fail(MUIR_ERR_INVALID_ARG, "%s: negative size", who);
  if (a->H <= 0 || !dim_ok(a->dk) || !dim_ok(a->dv))
    return fail(MUIR_ERR_UNSUPPORTED, "%s: unsupported sizes H=%d dk=%d dv=%d", who, a->H, a->dk, a->dv);
  if (!dtype_ok(a->dtype)) return fail(MUIR_ERR_UNSUPPORTED, "%s: dtype %d", who, a->dtype);
  if (a->flags != 0) return fail(MUIR_ERR_INVALID_ARG, "%s: flags must be 0", who);
  if (a->T > (int64_t(1) << 30) || a->B > 65535 || a->H > 65535 || a->B * a->H > 65535)
    return fail(MUIR_ERR_UNSUPPORTED, "%s: B H must be at most 65535 and T at most 2^30", who);
  return MUIR_OK;
}
bool lin_empty(const muir_lin_args* a) { return a->B == 0; }
int lin_pointers(const muir_lin_args* a, const char* who) {
  const bool no_tokens = a->T == 0;
  const Ptr ptrs[] = {{a->q, "q", no_tokens}, {a->k, "k", no_tokens}, {a->v, "v", no_tokens},
                      {a->log_decay, "log_decay"}, {a->S0, "S0", true}};
  if (int rc = check_ptrs(who, ptrs)) return rc;
  if (!aligned(a->lengths, 4)) return fail(MUIR_ERR_INVALID_ARG, "%s: lengths is not 4-byte aligned", who);
  return MUIR_OK;
}
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
size_t lin_seg_bytes(const muir_lin_args* a, const LinPlan& pl) {
  return pl.nseg > 1 ? round256((size_t)a->B * a->H * pl.nseg * a->dk * a->dv * sizeof(float)) : 0;
}

template <typename K>
int set_smem(K kernel, size_t bytes) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
    return check_launch("cudaFuncSetAttribute");
  return MUIR_OK;
}

// CUDA-core passes: those with the same da share a launch.
template <int DA, typename T, bool OUT>
int lin_simt(const muir::LinSimtArgs& args, int n, const char* name, cudaStream_t s) {
  int64_t blocks = 0;
  for (int i = 0; i < n; ++i) {
    const muir::LinPass& p = args.p[i];
    const int64_t own = (int64_t)p.B * p.H * p.nseg * (p.dc / 32);
    blocks = own > blocks ? own : blocks;
  }
  if (blocks > kMaxBlocks) return fail(MUIR_ERR_UNSUPPORTED, "%s: too many blocks", name);
  if (int rc = set_smem(muir::lin_simt_kernel<DA, T, OUT>, sizeof(muir::LinSmem<DA>))) return rc;
  LaunchScope l(name, s);
  muir::lin_simt_kernel<DA, T, OUT><<<dim3((unsigned)blocks, (unsigned)n), 256, sizeof(muir::LinSmem<DA>), s>>>(args);
  return check_launch(name);
}
template <typename T, bool OUT>
int lin_simt_passes(const muir::LinPass* p, int n, const char* name, cudaStream_t s) {
  for (const int da : {32, 64, 128}) {
    muir::LinSimtArgs args{};
    int m = 0;
    for (int i = 0; i < n; ++i)
      if (p[i].da == da) args.p[m++] = p[i];
    if (m == 0) continue;
    const int rc = da == 32 ? lin_simt<32, T, OUT>(args, m, name, s)
                 : da == 64 ? lin_simt<64, T, OUT>(args, m, name, s) : lin_simt<128, T, OUT>(args, m, name, s);
    if (rc) return rc;
  }
  return MUIR_OK;
}
template <bool OUT>
int lin_simt_all(const muir::LinPass* p, int n, int dtype, const char* name, cudaStream_t s) {
  return dtype == MUIR_BF16 ? lin_simt_passes<bf16, OUT>(p, n, name, s) : lin_simt_passes<float, OUT>(p, n, name, s);
}

template <bool OUT, int PARTS>
int lin_tc(const muir::LinPass* p, int n, const char* name, cudaStream_t s) {
  muir::LinTcArgs args{};
  for (int i = 0; i < n; ++i) {
    const muir::LinPass& q = p[i];
    const uint64_t ra = (uint64_t)q.H * q.da, rc = (uint64_t)q.H * q.dc;
    if ((OUT && !muir_host::make_tmap_bf16_3d(&args.a[i], q.a, ra, (uint64_t)q.T, (uint64_t)q.B, muir::kLtChunk)) ||
        !muir_host::make_tmap_bf16_3d(&args.b[i], q.b, ra, (uint64_t)q.T, (uint64_t)q.B, muir::kLtChunk) ||
        !muir_host::make_tmap_bf16_3d(&args.c[i], q.c, rc, (uint64_t)q.T, (uint64_t)q.B, muir::kLtChunk) ||
        (OUT && q.dc >= 64 && !muir_host::make_tmap_bf16_3d(&args.o[i], q.out, rc, (uint64_t)q.T, (uint64_t)q.B, 32u)))
      return fail(MUIR_ERR_CUDA, "%s: tensor map encoding failed", name);
    args.p[i] = q;
  }
  const int64_t blocks = (int64_t)p->B * p->H * p->nseg;
  if (blocks > kMaxBlocks) return fail(MUIR_ERR_UNSUPPORTED, "%s: too many blocks", name);
  if (int rc = set_smem(muir::lin_tc_kernel<OUT, PARTS>, muir::kLtSmem)) return rc;
  LaunchScope l(name, s);
  muir::lin_tc_kernel<OUT, PARTS><<<dim3((unsigned)blocks, (unsigned)n), muir::kLtThreads, muir::kLtSmem, s>>>(args);
  return check_launch(name);
}

// `states`: the passes whose segment states are made and combined (none for one
// segment), `outs`: the passes that write outputs.
int lin_run(const LinPlan& pl, int dtype, const muir::LinPass* states, int ns, const muir::LinPass* outs, int no,
            const char* name, cudaStream_t s) {
  int rc = MUIR_OK;
  if (pl.nseg > 1) {
    rc = pl.tc ? lin_tc<false, 3>(states, ns, "lin_state", s) : lin_simt_all<false>(states, ns, dtype, "lin_state", s);
    if (rc) return rc;
    muir::LinCombineArgs ca{};
    for (int i = 0; i < ns; ++i) ca.p[i] = states[i];
    const muir::LinPass& p = states[0];
    LaunchScope l("lin_combine", s);
    muir::lin_combine_kernel<<<dim3((unsigned)((p.da * p.dc + 511) / 512), (unsigned)(p.B * p.H), (unsigned)ns), 128, 0, s>>>(ca);
    if ((rc = check_launch("lin_combine"))) return rc;
  }
  if (pl.tc) {
    // a final state comes from this launch only where there is one segment
    bool fin = false;
    for (int i = 0; i < no; ++i) fin = fin || (pl.nseg == 1 && outs[i].fin);
    return fin ? lin_tc<true, 3>(outs, no, name, s) : lin_tc<true, 2>(outs, no, name, s);
  }
  return lin_simt_all<true>(outs, no, dtype, name, s);
}

muir::LinPass lin_pass(const muir_lin_args* x, const LinPlan& pl, int da, int dc) {
  muir::LinPass p{};
  p.log_decay = x->log_decay;
  p.lengths = x->lengths;
  p.T = x->T;
  p.seglen = pl.seglen;
  p.nseg = pl.nseg;
  p.B = (int)x->B;
  p.H = x->H;
  p.da = da;
  p.dc = dc;
  return p;
}

}  // namespace

extern "C" {

size_t muir_lin_fwd_workspace(const muir_lin_args* a) {
  muir_host::clear_error();
  if (lin_validate(a, "lin_fwd") || lin_empty(a)) return 0;
  return lin_seg_bytes(a, lin_plan(a, 1, 1));
}

int muir_lin_fwd(const muir_lin_args* a, void* y, float* S_T, void* ws, size_t ws_bytes, void* stream) {
  muir_host::clear_error();
  int rc = lin_validate(a, "lin_fwd");
  if (rc) return rc;
  if (lin_empty(a)) return MUIR_OK;
  if ((rc = lin_pointers(a, "lin_fwd"))) return rc;
  const Ptr outs[] = {{y, "y", a->T == 0}, {S_T, "S_T", true}};
  if ((rc = check_ptrs("lin_fwd", outs))) return rc;
  const LinPlan pl = lin_plan(a, 1, 1);
  const size_t need = lin_seg_bytes(a, pl);
  if (need && (!ws || !aligned(ws, 256) || ws_bytes < need))
    return fail(MUIR_ERR_WORKSPACE, "lin_fwd: workspace needs %zu bytes, 256-byte aligned", need);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  muir::LinPass p = lin_pass(a, pl, a->dk, a->dv);
  p.a = a->q;
  p.b = a->k;
  p.c = a->v;
  p.out = y;
  p.init = a->S0;
  p.fin = S_T;
  p.seg = need ? static_cast<float*>(ws) : nullptr;
  p.p_scale = p.o_scale = a->scale;
  p.u_scale = 1.f;
  return lin_run(pl, a->dtype, &p, 1, &p, 1, "lin_fwd", s);
}

size_t muir_lin_bwd_workspace(const muir_lin_args* a) {
  muir_host::clear_error();
  if (lin_validate(a, "lin_bwd") || lin_empty(a)) return 0;
  const LinPlan pl = lin_plan(a, 3, 2);
  return 2 * lin_seg_bytes(a, pl);
}

int muir_lin_bwd(const muir_lin_args* a, const muir_lin_grads* g, void* ws, size_t ws_bytes, void* stream) {
  muir_host::clear_error();
  int rc = lin_validate(a, "lin_bwd");
  if (rc) return rc;
  if (!g) return fail(MUIR_ERR_INVALID_ARG, "lin_bwd: grads is NULL");
  if (lin_empty(a)) return MUIR_OK;
  if ((rc = lin_pointers(a, "lin_bwd"))) return rc;
  const bool no_tokens = a->T == 0;
  const Ptr ptrs[] = {{g->dy, "dy", no_tokens}, {g->dq, "dq", no_tokens}, {g->dk, "dk", no_tokens}, {g->dv, "dv", no_tokens},
                      {g->dS_T, "dS_T", true}, {g->dS0, "dS0", true}};
  if ((rc = check_ptrs("lin_bwd", ptrs))) return rc;
  // the passes run side by side: one may still read these while dS0 is written
  if (g->dS0 && (g->dS0 == g->dS_T || g->dS0 == a->S0))
    return fail(MUIR_ERR_INVALID_ARG, "lin_bwd: dS0 must not be dS_T's or S0's buffer");
  const LinPlan pl = lin_plan(a, 3, 2);
  const size_t seg = lin_seg_bytes(a, pl);
  if (seg && (!ws || !aligned(ws, 256) || ws_bytes < 2 * seg))
    return fail(MUIR_ERR_WORKSPACE, "lin_bwd: workspace needs %zu bytes, 256-byte aligned", 2 * seg);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* S = seg ? static_cast<float*>(ws) : nullptr;
  float* dS = seg ? reinterpret_cast<float*>(static_cast<char*>(ws) + seg) : nullptr;

  // the gradients with the longest walk back first; states of dv's and dk's pass, and of dq's
  muir::LinPass p[3], st[2];
  // dv: keys against queries, cotangents summed, from the last token to the first
  p[0] = lin_pass(a, pl, a->dk, a->dv);
  p[0].a = a->k;
  p[0].b = a->q;
  p[0].c = g->dy;
  p[0].out = g->dv;
  p[0].init = g->dS_T;
  p[0].fin = g->dS0;
  p[0].seg = dS;
  p[0].reverse = 1;
  p[0].p_scale = p[0].u_scale = a->scale;
  p[0].o_scale = 1.f;
  st[0] = p[0];
  // dk: values against cotangents, queries summed; the state is dS^T
  p[1] = lin_pass(a, pl, a->dv, a->dk);
  p[1].a = a->v;
  p[1].b = g->dy;
  p[1].c = a->q;
  p[1].out = g->dk;
  p[1].init = g->dS_T;
  p[1].init_t = 1;
  p[1].seg = dS;
  p[1].seg_t = 1;
  p[1].reverse = 1;
  p[1].p_scale = p[1].u_scale = a->scale;
  p[1].o_scale = 1.f;
  // dq: cotangents against values, keys summed, forward; the state is S^T
  p[2] = lin_pass(a, pl, a->dv, a->dk);
  p[2].a = g->dy;
  p[2].b = a->v;
  p[2].c = a->k;
  p[2].out = g->dq;
  p[2].init = a->S0;
  p[2].init_t = 1;
  p[2].seg = S;
  p[2].seg_t = 1;
  p[2].p_scale = p[2].o_scale = a->scale;
  p[2].u_scale = 1.f;
  st[1] = lin_pass(a, pl, a->dk, a->dv);
  st[1].b = a->k;
  st[1].c = a->v;
  st[1].init = a->S0;
  st[1].seg = S;
  st[1].u_scale = 1.f;
  return lin_run(pl, a->dtype, st, 2, p, 3, "lin_bwd", s);
}

int muir_lin_step(const muir_lin_step_args* a, void* stream) {
  muir_host::clear_error();
  if (!a) return fail(MUIR_ERR_INVALID_ARG, "lin_step: args is NULL");
  if (a->n_seq < 0) return fail(MUIR_ERR_INVALID_ARG, "lin_step: n_seq < 0");
  if (a->H <= 0 || !dim_ok(a->dk) || !dim_ok(a->dv))
    return fail(MUIR_ERR_UNSUPPORTED, "lin_step: unsupported sizes H=%d dk=%d dv=%d", a->H, a->dk, a->dv);
  if (!dtype_ok(a->dtype)) return fail(MUIR_ERR_UNSUPPORTED, "lin_step: dtype %d", a->dtype);
  if (a->n_seq == 0) return MUIR_OK;
  const Ptr ptrs[] = {{a->S, "S"}, {a->q, "q"}, {a->k, "k"}, {a->v, "v"}, {a->log_decay, "log_decay"}, {a->y, "y"}};
  if (int rc = check_ptrs("lin_step", ptrs)) return rc;
  if (a->n_seq > kMaxBlocks / a->H / (a->dv / 32)) return fail(MUIR_ERR_UNSUPPORTED, "lin_step: too many rows");
  const unsigned blocks = (unsigned)(a->n_seq * a->H * (a->dv / 32));
  const muir::LinStepParams p{a->S, a->q, a->k, a->v, a->log_decay, a->y, a->H, a->dv, a->scale};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope l("lin_step", s);
#define MUIR_STEP(DK)                                                   \
  if (a->dtype == MUIR_BF16)                                            \
    muir::lin_step_kernel<DK, bf16><<<blocks, 128, 0, s>>>(p);          \
  else                                                                  \
    muir::lin_step_kernel<DK, float><<<blocks, 128, 0, s>>>(p)
  switch (a->dk) {
    case 32: MUIR_STEP(32); break;
    case 64: MUIR_STEP(64); break;
    default: MUIR_STEP(128); break;
  }
#undef MUIR_STEP
  return check_launch("lin_step launch");
}

}  // extern "C"

// ---- RMS norm ---------------------------------------------------------------------

namespace {

constexpr int kNormMaxD = 16384;

int norm_validate(const char* who, int64_t n, int32_t d, int32_t dtype, bool need_eps, float eps) {
  if (n < 0) return fail(MUIR_ERR_INVALID_ARG, "%s: n < 0", who);
  if (d <= 0 || d % 8 || d > kNormMaxD)
    return fail(MUIR_ERR_UNSUPPORTED, "%s: d must be a multiple of 8 up to %d (got %d)", who, kNormMaxD, d);
  if (!dtype_ok(dtype)) return fail(MUIR_ERR_UNSUPPORTED, "%s: dtype %d", who, dtype);
  if (need_eps && !(eps >= 0.f)) return fail(MUIR_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
  if (n > kMaxBlocks) return fail(MUIR_ERR_UNSUPPORTED, "%s: too many rows", who);
  return MUIR_OK;
}

template <typename T, int NT, int V, bool QUANT>
void norm_go(const muir::NormParams& p, cudaStream_t s) {
  if (NT > 32) muir::rms_norm_kernel<T, NT, V, QUANT><<<(unsigned)p.n, NT, 0, s>>>(p);
  else muir::rms_norm_kernel<T, NT, V, QUANT><<<(unsigned)((p.n + 7) / 8), 256, 0, s>>>(p);
}
// Threads per row: a warp up to 1024 elements; above that two pieces of 8 per thread
// (32768 x 2048 bf16 with the residual, before the loads were moved ahead of the
// stores: 88 us with 128 threads, 94 with 256 and one piece, 101 with 64 and four).
template <typename T, bool QUANT>
void norm_dispatch(const muir::NormParams& p, cudaStream_t s) {
  if (p.d <= 256) norm_go<T, 32, 1, QUANT>(p, s);
  else if (p.d <= 512) norm_go<T, 32, 2, QUANT>(p, s);
  else if (p.d <= 1024) norm_go<T, 32, 4, QUANT>(p, s);
  else if (p.d <= 2048) norm_go<T, 128, 2, QUANT>(p, s);
  else if (p.d <= 4096) norm_go<T, 256, 2, QUANT>(p, s);
  else if (p.d <= 8192) norm_go<T, 512, 2, QUANT>(p, s);
  else norm_go<T, 1024, 2, QUANT>(p, s);
}

int norm_fwd(const char* who, muir::NormParams p, int32_t dtype, bool quant, void* stream) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope l(who, s);
  if (dtype == MUIR_BF16) quant ? norm_dispatch<bf16, true>(p, s) : norm_dispatch<bf16, false>(p, s);
  else quant ? norm_dispatch<float, true>(p, s) : norm_dispatch<float, false>(p, s);
  return check_launch(who);
}

// CTAs of the backward: rows are walked in strides of the grid, so that dweight's
// partial sums are few. Above 1024 columns as many CTAs as stay resident; below, where
// CTAs are smaller, four for each SM as well, which leaves narrow rows waiting for memory
// with few loads in flight (524288 x 128 bf16: 731 us, 62 at the copy rate).
int norm_bwd_blocks(int64_t n, int32_t d) {
  const int64_t most = kSMs * (d <= 2048 ? 4 : d <= 4096 ? 2 : 1);
  return (int)(n < most ? n : most);
}

template <typename T>
void norm_bwd_dispatch(const muir::NormBwdParams& p, unsigned blocks, cudaStream_t s) {
  if (p.d <= 256) muir::rms_norm_bwd_kernel<T, 32, 1><<<blocks, 32, 0, s>>>(p);
  else if (p.d <= 1024) muir::rms_norm_bwd_kernel<T, 128, 1><<<blocks, 128, 0, s>>>(p);
  else if (p.d <= 2048) muir::rms_norm_bwd_kernel<T, 256, 1><<<blocks, 256, 0, s>>>(p);
  else if (p.d <= 4096) muir::rms_norm_bwd_kernel<T, 512, 1><<<blocks, 512, 0, s>>>(p);
  else if (p.d <= 8192) muir::rms_norm_bwd_kernel<T, 1024, 1><<<blocks, 1024, 0, s>>>(p);
  else muir::rms_norm_bwd_kernel<T, 1024, 2><<<blocks, 1024, 0, s>>>(p);
}

}  // namespace

extern "C" {

int muir_rms_norm(const void* x, const void* residual, const float* weight, void* y, void* h, float* rstd, int64_t n,
                  int32_t d, float eps, int32_t dtype, void* stream) {
  muir_host::clear_error();
  int rc = norm_validate("rms_norm", n, d, dtype, true, eps);
  if (rc || n == 0) return rc;
  const Ptr ptrs[] = {{x, "x"}, {residual, "residual", true}, {weight, "weight"}, {y, "y"}, {h, "h", residual == nullptr}};
  if ((rc = check_ptrs("rms_norm", ptrs))) return rc;
  if (!aligned(rstd, 4)) return fail(MUIR_ERR_INVALID_ARG, "rms_norm: rstd is not 4-byte aligned");
  return norm_fwd("rms_norm", muir::NormParams{x, residual, weight, y, h, nullptr, nullptr, rstd, n, d, eps}, dtype, false,
                  stream);
}

int muir_rms_norm_quant(const void* x, const void* residual, const float* weight, void* q, float* scale, void* h, float* rstd,
                        int64_t n, int32_t d, float eps, int32_t dtype, void* stream) {
  muir_host::clear_error();
  int rc = norm_validate("rms_norm_quant", n, d, dtype, true, eps);
  if (rc || n == 0) return rc;
  const Ptr ptrs[] = {{x, "x"}, {residual, "residual", true}, {weight, "weight"}, {q, "q"}, {h, "h", residual == nullptr}};
  if ((rc = check_ptrs("rms_norm_quant", ptrs))) return rc;
  if (!scale) return fail(MUIR_ERR_INVALID_ARG, "rms_norm_quant: scale is NULL");
  if (!aligned(rstd, 4) || !aligned(scale, 4)) return fail(MUIR_ERR_INVALID_ARG, "rms_norm_quant: rstd or scale misaligned");
  return norm_fwd("rms_norm_quant",
                  muir::NormParams{x, residual, weight, nullptr, h, static_cast<uint8_t*>(q), scale, rstd, n, d, eps}, dtype,
                  true, stream);
}

size_t muir_rms_norm_bwd_workspace(int64_t n, int32_t d) {
  muir_host::clear_error();
  if (norm_validate("rms_norm_bwd", n, d, MUIR_F32, false, 0.f) || n == 0) return 0;
  return round256((size_t)norm_bwd_blocks(n, d) * d * sizeof(float));
}

int muir_rms_norm_bwd(const void* dy, const void* h, const float* weight, const float* rstd, const void* dh, void* dx,
                      float* dweight, int64_t n, int32_t d, int32_t dtype, void* ws, size_t ws_bytes, void* stream) {
  muir_host::clear_error();
  int rc = norm_validate("rms_norm_bwd", n, d, dtype, false, 0.f);
  if (rc) return rc;
  const bool none = n == 0;
  const Ptr ptrs[] = {{dy, "dy", none}, {h, "h", none}, {weight, "weight", none}, {dh, "dh", true}, {dx, "dx", none},
                      {dweight, "dweight"}};
  if ((rc = check_ptrs("rms_norm_bwd", ptrs))) return rc;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (none) {  // the sum over no rows
    if (cudaMemsetAsync(dweight, 0, (size_t)d * sizeof(float), s) != cudaSuccess) return check_launch("rms_norm_bwd");
    return MUIR_OK;
  }
  if (!rstd || !aligned(rstd, 4)) return fail(MUIR_ERR_INVALID_ARG, "rms_norm_bwd: rstd is NULL or misaligned");
  const size_t need = muir_rms_norm_bwd_workspace(n, d);
  if (!ws || !aligned(ws, 256) || ws_bytes < need)
    return fail(MUIR_ERR_WORKSPACE, "rms_norm_bwd: workspace needs %zu bytes, 256-byte aligned", need);
  const unsigned blocks = (unsigned)norm_bwd_blocks(n, d);
  const muir::NormBwdParams p{dy, h, dh, weight, rstd, dx, dweight, static_cast<float*>(ws), n, d};
  {
    LaunchScope l("rms_norm_bwd", s);
    dtype == MUIR_BF16 ? norm_bwd_dispatch<bf16>(p, blocks, s) : norm_bwd_dispatch<float>(p, blocks, s);
  }
  if ((rc = check_launch("rms_norm_bwd"))) return rc;
  LaunchScope l("rms_norm_dw", s);
  muir::rms_norm_dw_kernel<<<(unsigned)((d + 31) / 32), 1024, 0, s>>>(p.part, dweight, (int)blocks, d);
  return check_launch("rms_norm_dw");
}

}  // extern "C"

// ---- 4-bit weights ------------------------------------------------------------------

namespace {

int w4_validate(const char* who, int32_t K, int32_t O, int32_t group) {
  if (K <= 0 || K % 128 || O <= 0)
    return fail(MUIR_ERR_UNSUPPORTED, "%s: K must be a multiple of 128 and O positive (got %d, %d)", who, K, O);
  if (O > kMaxBlocks - 15) return fail(MUIR_ERR_UNSUPPORTED, "%s: O must be at most 2^31 - 16", who);  // whole tiles, in 32 bits
  if (group != 32 && group != 64 && group != 128) return fail(MUIR_ERR_UNSUPPORTED, "%s: group %d", who, group);
  return MUIR_OK;
}

template <typename X, typename Y, int NB, int RT>
void w4_launch(const muir::W4Params& p, int group, cudaStream_t s) {
  const int tiles = (p.O + 15) / 16;
  const dim3 grid((unsigned)((tiles + RT - 1) / RT), (unsigned)((p.n + 8 * NB - 1) / (8 * NB)));
  if (group == 32) muir::w4_matvec_kernel<X, Y, NB, 4, RT><<<grid, 32 * muir::kW4Warps, 0, s>>>(p);
  else if (group == 64) muir::w4_matvec_kernel<X, Y, NB, 2, RT><<<grid, 32 * muir::kW4Warps, 0, s>>>(p);
  else muir::w4_matvec_kernel<X, Y, NB, 1, RT><<<grid, 32 * muir::kW4Warps, 0, s>>>(p);
}
// Two tiles of outputs per CTA where that still makes eight CTAs for each SM: x is
// then fetched and converted half as often. K = 2048, two tiles against one: 50257
// outputs of eight e4m3 rows 17.4 against 18.8 us, 30000 12.9 both, 16384 7.2 against
// 6.9, 6144 of one bf16 row 4.5 against 3.8. More than 16 rows take one tile (registers).
template <typename X, typename Y, int NB>
void w4_go(const muir::W4Params& p, int group, cudaStream_t s) {
  if constexpr (NB <= 2) {
    if ((p.O + 15) / 16 >= 16 * kSMs) return w4_launch<X, Y, NB, 2>(p, group, s);
  }
  w4_launch<X, Y, NB, 1>(p, group, s);
}
template <typename X, typename Y>
void w4_rows(const muir::W4Params& p, int group, cudaStream_t s) {
  if (p.n <= 8) w4_go<X, Y, 1>(p, group, s);
  else if (p.n <= 16) w4_go<X, Y, 2>(p, group, s);
  else w4_go<X, Y, 4>(p, group, s);
}

}  // namespace

extern "C" {

size_t muir_w4_bytes(int32_t K, int32_t O, int32_t group, size_t* scale_bytes) {
  muir_host::clear_error();
  if (scale_bytes) *scale_bytes = 0;
  if (w4_validate("w4_bytes", K, O, group)) return 0;
  const size_t rows = ((size_t)O + 15) / 16 * 16;
  if (scale_bytes) *scale_bytes = rows * (K / group) * 2;
  return rows * K / 2;
}

int muir_w4_quantize(const void* w, void* codes, void* scales, int32_t K, int32_t O, int32_t group, int32_t dtype,
                     void* stream) {
  muir_host::clear_error();
  int rc = w4_validate("w4_quantize", K, O, group);
  if (rc) return rc;
  if (!dtype_ok(dtype)) return fail(MUIR_ERR_UNSUPPORTED, "w4_quantize: dtype %d", dtype);
  const Ptr ptrs[] = {{w, "w"}, {codes, "codes"}, {scales, "scales"}};
  if ((rc = check_ptrs("w4_quantize", ptrs))) return rc;
  const int64_t groups = (int64_t)O * (K / group), need = (groups + 7) / 8;
  const unsigned blocks = (unsigned)(need < 32 * kSMs ? need : 32 * kSMs);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope l("w4_quantize", s);
  if (dtype == MUIR_BF16)
    muir::w4_quantize_kernel<bf16><<<blocks, 256, 0, s>>>(static_cast<const bf16*>(w), static_cast<uint8_t*>(codes),
                                                          static_cast<bf16*>(scales), groups, group);
  else
    muir::w4_quantize_kernel<float><<<blocks, 256, 0, s>>>(static_cast<const float*>(w), static_cast<uint8_t*>(codes),
                                                           static_cast<bf16*>(scales), groups, group);
  return check_launch("w4_quantize");
}

int muir_w4_pack(const void* codes, const void* scales, void* wq, void* ws, int32_t K, int32_t O, int32_t group,
                 void* stream) {
  muir_host::clear_error();
  int rc = w4_validate("w4_pack", K, O, group);
  if (rc) return rc;
  const Ptr ptrs[] = {{codes, "codes"}, {scales, "scales"}, {wq, "wq"}, {ws, "ws"}};
  if ((rc = check_ptrs("w4_pack", ptrs))) return rc;
  size_t sb = 0;
  const int64_t words = (int64_t)(muir_w4_bytes(K, O, group, &sb) / 4), nscales = (int64_t)(sb / 2);
  const int64_t need = (words + nscales + 255) / 256;
  const unsigned blocks = (unsigned)(need < 32 * kSMs ? need : 32 * kSMs);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope l("w4_pack", s);
  muir::w4_pack_kernel<<<blocks, 256, 0, s>>>(static_cast<const uint8_t*>(codes), static_cast<const bf16*>(scales),
                                              static_cast<uint32_t*>(wq), static_cast<bf16*>(ws), K, O, 128 / group, words,
                                              nscales);
  return check_launch("w4_pack");
}

int muir_w4_matvec(const void* x, const float* x_scale, const void* wq, const void* ws, void* y, int64_t n, int32_t K,
                   int32_t O, int32_t group, int32_t x_dtype, int32_t y_dtype, void* stream) {
  muir_host::clear_error();
  int rc = w4_validate("w4_matvec", K, O, group);
  if (rc) return rc;
  if (!dtype_ok(y_dtype) || (x_dtype != MUIR_E4M3 && x_dtype != y_dtype))
    return fail(MUIR_ERR_UNSUPPORTED, "w4_matvec: x dtype %d with y dtype %d", x_dtype, y_dtype);
  if (n < 0) return fail(MUIR_ERR_INVALID_ARG, "w4_matvec: n < 0");
  if (n > 65535 * 32) return fail(MUIR_ERR_UNSUPPORTED, "w4_matvec: too many rows");
  if (n == 0) return MUIR_OK;
  const Ptr ptrs[] = {{x, "x"}, {wq, "wq"}, {ws, "ws"}, {y, "y"}};
  if ((rc = check_ptrs("w4_matvec", ptrs))) return rc;
  if (!aligned(x_scale, 4)) return fail(MUIR_ERR_INVALID_ARG, "w4_matvec: x_scale is not 4-byte aligned");
  if (x_scale && x_dtype != MUIR_E4M3) return fail(MUIR_ERR_INVALID_ARG, "w4_matvec: x_scale belongs to 8-bit rows");
  const muir::W4Params p{x, x_scale, static_cast<const uint8_t*>(wq), static_cast<const bf16*>(ws), y, n, K, O};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  LaunchScope l("w4_matvec", s);
  if (x_dtype == MUIR_BF16) w4_rows<bf16, bf16>(p, group, s);
  else if (x_dtype == MUIR_F32) w4_rows<float, float>(p, group, s);
  else if (y_dtype == MUIR_BF16) w4_rows<__nv_fp8_e4m3, bf16>(p, group, s);
  else w4_rows<__nv_fp8_e4m3, float>(p, group, s);
  return check_launch("w4_matvec");
}

}  // extern "C"
