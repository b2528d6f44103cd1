// C ABI of linear attention with a decay for each head (include/delta_linear.h): argument validation,
// workspace layout and the order of the launches.  Nothing here throws or allocates.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "../../include/delta_linear.h"
#include "abi_common.h"
#include "linear.h"

using delta::LinChain;
using delta::LinDecode;
using delta::LinGates;
using delta::LinRole;
using namespace delta::abi;

static_assert((int)DELTA_LIN_GATE_TOKEN == (int)delta::LIN_GATE_TOKEN && (int)DELTA_LIN_GATE_HEAD == (int)delta::LIN_GATE_HEAD,
              "gate kinds");

namespace {

struct Lin {
  int B, L, H, Hk, dk, dv, gate, NT, P, NS;
  int most;  // segments that a sequence of up to this length is cut into
  bool bf16;
  float scale;
  size_t nqk, nv, ng, state;  // bytes of q, of v, of the gates, of the states
};

int lin_shape(const delta_shape* s, int32_t qk_heads, int32_t gate, bool backward, Lin& n) {
  const int rc = check_shape(s);
  if (rc) return rc;
  if (s->n_h != 1 || qk_heads < 1 || s->H % qk_heads != 0 || s->L > (1 << 30)) return DELTA_ERR_BAD_SHAPE;
  if (gate != DELTA_LIN_GATE_NONE && gate != DELTA_LIN_GATE_TOKEN && gate != DELTA_LIN_GATE_HEAD) return DELTA_ERR_UNSUPPORTED_DIM;
  if ((long long)s->H * (s->dk > s->dv ? s->dk : s->dv) > (1LL << 20)) return DELTA_ERR_BAD_SHAPE;
  // a launch has fewer than 2^32 threads: up to 1024 for a sequence and head, one for four elements of a state
  const long long heads = (long long)s->B * s->H;
  if (heads > (1LL << 20) || heads * s->dk * s->dv > (1LL << 33)) return DELTA_ERR_BAD_SHAPE;
  n.B = s->B, n.L = s->L, n.H = s->H, n.Hk = qk_heads, n.dk = s->dk, n.dv = s->dv, n.gate = gate;
  n.bf16 = s->dtype == DELTA_BF16, n.scale = s->scale;
  delta::lin_split(n.B, n.L, n.H, n.dv, n.bf16, backward, n.NT, n.P, n.NS, n.most);
  const size_t tokens = (size_t)n.B * n.L, e = esize(s->dtype);
  n.nqk = n.H ? tokens * n.Hk * n.dk * e : 0, n.nv = tokens * n.H * n.dv * e;
  n.ng = 4 * (gate == DELTA_LIN_GATE_TOKEN ? tokens * n.H : gate == DELTA_LIN_GATE_HEAD ? (size_t)n.H : 0);
  n.state = (size_t)n.B * n.H * n.dk * n.dv * 4;
  return DELTA_OK;
}

// Regions of a workspace, each on its own 256 bytes; with a null base only their total is formed.  A longer sequence may
// have fewer segments than a shorter one; there is room for the most of any up to this length, so that a workspace
// for the longest serves all.
struct Carve {
  char* base;
  size_t used = 0;
  template <typename T>
  T* take(size_t bytes) {
    T* p = base && bytes ? reinterpret_cast<T*>(base + used) : nullptr;
    used += align_up(bytes);
    return p;
  }
};

struct FwdSpace {
  float* segs;
  double* decay;
};
size_t carve(const Lin& n, void* base, FwdSpace& w) {
  Carve c{static_cast<char*>(base)};
  const size_t segments = n.most > 1 ? (size_t)n.B * n.H * n.most : 0;
  w.segs = c.take<float>(segments * n.dk * n.dv * 4);
  w.decay = c.take<double>(segments * 8);
  return c.used;
}

struct BwdSpace {
  float *segs, *gsegs;
  double *decay, *gdecay, *part;
  float *e, *f, *pair, *edge, *states, *wait_q, *wait_k, *wait_v, *dq, *dk;
};
size_t carve(const Lin& n, bool gates, void* base, BwdSpace& w) {
  Carve c{static_cast<char*>(base)};
  const bool halves = gates && n.dv <= 128;
  const size_t heads = (size_t)n.B * n.H, chunks = heads * n.NT, tokens = chunks * delta::lin_chunk(n.bf16) * 4;
  const size_t qk_state = delta::lin_state_bytes(n.dv, n.dk), v_state = delta::lin_state_bytes(n.dk, n.dv);
  const size_t segments = n.most > 1 ? heads * n.most : 0, parts = heads * n.most;
  w.segs = c.take<float>(segments * n.dk * n.dv * 4);
  w.gsegs = c.take<float>(segments * n.dk * n.dv * 4);
  w.decay = c.take<double>(segments * 8);
  w.gdecay = c.take<double>(segments * 8);
  w.part = c.take<double>(gates && n.gate == DELTA_LIN_GATE_HEAD ? heads * ((n.NT + delta::LIN_GATE_CHUNKS - 1) / delta::LIN_GATE_CHUNKS) * 8 : 0);
  w.e = c.take<float>(gates ? tokens : 0);
  w.f = c.take<float>(gates ? tokens : 0);
  w.pair = c.take<float>(gates ? tokens : 0);
  w.edge = c.take<float>(gates ? chunks * 4 : 0);
  w.states = c.take<float>(gates ? chunks * qk_state : 0);
  w.wait_q = c.take<float>(halves ? parts * qk_state : 0);
  w.wait_k = c.take<float>(halves ? parts * qk_state : 0);
  w.wait_v = c.take<float>(halves ? parts * v_state : 0);
  w.dq = c.take<float>(n.H != n.Hk ? heads * n.L * n.dk * 4 : 0);  // parts of the heads that share
  w.dk = c.take<float>(n.H != n.Hk ? heads * n.L * n.dk * 4 : 0);
  return c.used;
}

// Pointers that have to be there, and every alignment.
template <int N>
int check_pointers(const void* const (&needed)[N], bool work) {
  for (const void* p : needed)
    if (work && !p) return DELTA_ERR_NULL_ARG;
  return DELTA_OK;
}
template <int N>
int check_aligned(const void* const (&ptrs)[N], const float* g, const float* dg) {
  for (const void* p : ptrs)
    if (!aligned16(p)) return DELTA_ERR_MISALIGNED;
  return aligned(g, 4) && aligned(dg, 4) ? DELTA_OK : DELTA_ERR_MISALIGNED;
}

Range span(const void* p, size_t bytes) { return range(p, p ? bytes : 0); }

LinChain chain_of(const Lin& n, const float* g) {
  LinChain c;
  memset(&c, 0, sizeof(c));
  c.B = n.B, c.L = n.L, c.H = n.H, c.NT = n.NT, c.P = n.P, c.NS = n.NS, c.run = n.P;
  c.g = g, c.gate = n.gate;
  c.outer = c.inner = c.write = 1.f;
  return c;
}

}  // namespace

extern "C" {

int delta_fwd_lin_workspace_bytes(const delta_shape* s, int32_t qk_heads, size_t* bytes) {
  Lin n;
  const int rc = lin_shape(s, qk_heads, DELTA_LIN_GATE_NONE, false, n);
  if (rc) return rc;
  if (!bytes) return DELTA_ERR_NULL_ARG;
  FwdSpace w;
  *bytes = carve(n, nullptr, w);
  return DELTA_OK;
}

int delta_fwd_lin(const delta_shape* s, int32_t qk_heads, int32_t gate, const void* q, const void* k, const void* v,
                  const float* g_log, const float* S0, void* O, float* S_final, void* workspace, size_t workspace_bytes,
                  void* stream) {
  Lin n;
  int rc = lin_shape(s, qk_heads, gate, false, n);
  if (rc) return rc;
  if ((rc = check_pointers({q, k, v, O}, n.nv > 0))) return rc;
  if ((gate == DELTA_LIN_GATE_NONE) != (g_log == nullptr) && (g_log || n.nv > 0)) return DELTA_ERR_NULL_ARG;
  FwdSpace w;
  const size_t need = carve(n, nullptr, w);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DELTA_ERR_WORKSPACE;
  if ((rc = check_aligned({q, k, v, S0, O, S_final, workspace}, g_log, nullptr))) return rc;
  const bool in_place = S0 && S0 == S_final;
  const Range in[] = {span(q, n.nqk), span(k, n.nqk), span(v, n.nv), span(g_log, n.ng), span(in_place ? nullptr : S0, n.state)};
  const Range out[] = {span(O, n.nv), span(S_final, n.state), span(workspace, need)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  if (n.state == 0 || (n.L == 0 && !S_final)) return DELTA_OK;
  if ((rc = launch_guard())) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (g_log && validate_on() && (rc = validate_gates(g_log, n.ng / 4, st))) return rc;
  carve(n, workspace, w);
  LinChain c = chain_of(n, g_log);
  c.x = LinRole{q, n.Hk, n.dk}, c.y = LinRole{k, n.Hk, n.dk}, c.z = LinRole{v, n.H, n.dv};
  c.start = S0, c.end = S_final, c.segs = w.segs, c.decay = w.decay;
  c.outer = c.inner = n.scale;
  c.out = O, c.out_f32 = !n.bf16;
  if (n.P != 1) {  // P = 0: no tokens, the state as it is
    c.run = S_final ? n.P : n.P - 1;
    if (n.P > 0 && (rc = hip_status(delta::launch_lin_summary(c, nullptr, n.bf16, st)))) return rc;
    if ((rc = hip_status(delta::launch_lin_combine(&c, nullptr, st))) || n.P == 0) return rc;
    c.run = n.P;
  }
  return hip_status(delta::launch_lin_chain(c, n.bf16, false, n.P == 1 && S_final ? delta::LIN_STATE : delta::LIN_PLAIN, st));
}

int delta_bwd_lin_workspace_bytes(const delta_shape* s, int32_t qk_heads, int32_t gate, size_t* bytes) {
  Lin n;
  const int rc = lin_shape(s, qk_heads, gate, true, n);
  if (rc) return rc;
  if (!bytes) return DELTA_ERR_NULL_ARG;
  BwdSpace w;
  *bytes = carve(n, gate != DELTA_LIN_GATE_NONE, nullptr, w);
  return DELTA_OK;
}

int delta_bwd_lin(const delta_shape* s, int32_t qk_heads, int32_t gate, const void* q, const void* k, const void* v,
                  const float* g_log, const float* S0, const void* dO, const float* dS_final, void* dq, void* dk, void* dv,
                  float* dg_log, float* dS0, void* workspace, size_t workspace_bytes, void* stream) {
  Lin n;
  int rc = lin_shape(s, qk_heads, gate, true, n);
  if (rc) return rc;
  if ((rc = check_pointers({q, k, v, dO, dq, dk, dv}, n.nv > 0))) return rc;
  if ((gate == DELTA_LIN_GATE_NONE) != (g_log == nullptr) && (g_log || n.nv > 0)) return DELTA_ERR_NULL_ARG;
  if (gate == DELTA_LIN_GATE_NONE && dg_log) return DELTA_ERR_UNSUPPORTED_DIM;
  BwdSpace w;
  const size_t need = carve(n, dg_log != nullptr, nullptr, w);
  if (need > 0 && (!workspace || workspace_bytes < need)) return DELTA_ERR_WORKSPACE;
  if ((rc = check_aligned({q, k, v, S0, dO, dS_final, dq, dk, dv, dS0, workspace}, g_log, dg_log))) return rc;
  const Range in[] = {span(q, n.nqk),    span(k, n.nqk),   span(v, n.nv),           span(g_log, n.ng),
                      span(S0, n.state), span(dO, n.nv), span(dS_final, n.state)};
  const Range out[] = {span(dq, n.nqk), span(dk, n.nqk), span(dv, n.nv), span(dg_log, n.ng), span(dS0, n.state), span(workspace, need)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  const bool sum_only = gate == DELTA_LIN_GATE_HEAD && dg_log && n.H > 0;  // no tokens, and a gradient to clear
  if ((n.state == 0 || (n.L == 0 && !dS0)) && !sum_only) return DELTA_OK;
  if ((rc = launch_guard())) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (g_log && validate_on() && (rc = validate_gates(g_log, n.ng / 4, st))) return rc;
  carve(n, dg_log != nullptr, workspace, w);

  LinGates gp;
  memset(&gp, 0, sizeof(gp));
  gp.B = n.B, gp.L = n.L, gp.H = n.H, gp.C = delta::lin_chunk(n.bf16), gp.NT = n.NT;
  gp.e = w.e, gp.f = w.f, gp.pair = w.pair, gp.edge = w.edge;
  gp.g = g_log, gp.gate = gate, gp.dg = dg_log, gp.part = w.part;
  if (n.state == 0 || n.L == 0) {
    if (n.state > 0 && dS0) {
      LinChain c = chain_of(n, g_log);
      c.y.width = n.dk, c.z.width = n.dv, c.start = dS_final, c.end = dS0;
      if ((rc = hip_status(delta::launch_lin_combine(nullptr, &c, st)))) return rc;
    }
    gp.B = 0;
    return sum_only ? hip_status(delta::launch_lin_gates(gp, st)) : DELTA_OK;
  }

  const LinRole rq{q, n.Hk, n.dk}, rk{k, n.Hk, n.dk}, rv{v, n.H, n.dv}, ro{dO, n.H, n.dv};
  const bool shared = n.H != n.Hk;
  const long rows = (long)n.B * n.L;
  // S: the states from the start on; dq = scale chain(dO, v, k) with them transposed.  G: their gradients from the end on;
  // dv = chain(k, q, dO), and dk = chain(v, dO, q) with them transposed.
  LinChain dqc = chain_of(n, g_log), dvc = dqc;
  dqc.y = rk, dqc.z = rv, dqc.segs = w.segs, dqc.decay = w.decay, dqc.start = S0;
  dvc.y = rq, dvc.z = ro, dvc.segs = w.gsegs, dvc.decay = w.gdecay, dvc.start = dS_final, dvc.end = dS0;
  dvc.write = dvc.inner = n.scale;
  if (n.P > 1) {
    dqc.run = n.P - 1, dvc.run = dS0 ? n.P : n.P - 1;
    if ((rc = hip_status(delta::launch_lin_summary(dqc, &dvc, n.bf16, st)))) return rc;
    if ((rc = hip_status(delta::launch_lin_combine(&dqc, &dvc, st)))) return rc;
    dqc.run = dvc.run = n.P;
  }
  LinChain dkc = dvc;
  dqc.x = ro, dqc.y = rv, dqc.z = rk, dqc.w = rq, dqc.flip = true, dqc.outer = dqc.inner = n.scale, dqc.tok = w.e;
  dkc.x = rv, dkc.y = ro, dkc.z = rq, dkc.w = rk, dkc.flip = true, dkc.end = nullptr, dkc.tok = w.f;
  dvc.x = rk;
  dqc.out = shared ? w.dq : dq, dkc.out = shared ? w.dk : dk, dvc.out = dv;
  dqc.out_f32 = dkc.out_f32 = shared || !n.bf16, dvc.out_f32 = !n.bf16;
  const bool state = n.P == 1 && dS0;
  dqc.pair = w.pair, dqc.states = dkc.states = w.states, dqc.edge = dkc.edge = w.edge;
  if (!dg_log && n.dv <= 128) {
    if ((rc = hip_status(delta::launch_lin_backward(dqc, dvc, dkc, false, state, n.bf16, st)))) return rc;
  } else if (n.dv <= 128) {
    // S and G meet at every chunk: in a first launch dq walks a segment's first half from the front and dk the other from
    // the back, each leaving its states, and in a second each meets the other's.  dv goes in halves beside them, or whole in
    // the first launch, by which of the two takes fewer rounds of half walks on what the card holds at once: 256 workgroups
    // of each chain in bf16 (2 x 16 heads of 8K tokens, 8 segments) three rounds, dv in halves four; 160 in float32 four, dv
    // whole five.
    dqc.wait = w.wait_q, dkc.wait = w.wait_k, dvc.wait = w.wait_v;
    const long units = (long)n.B * n.H * n.P, card = n.bf16 ? 512 : 256;
    auto rounds = [card](long halves) { return (halves + card - 1) / card; };
    const bool halves = 2 * rounds(3 * units) < std::max(2L, rounds(4 * units)) + rounds(2 * units);
    for (int part = 1; part <= 2; ++part) {
      dqc.part = dkc.part = part, dvc.part = halves ? part : 0;
      if (part == 2 && !halves) dvc.run = 0;
      if ((rc = hip_status(delta::launch_lin_backward(dqc, dvc, dkc, true, state, n.bf16, st)))) return rc;
    }
  } else {  // dq leaves all states, dk meets them
    if ((rc = hip_status(delta::launch_lin_chain(dqc, n.bf16, false, dg_log ? delta::LIN_PAIRS : delta::LIN_PLAIN, st)))) return rc;
    if ((rc = hip_status(delta::launch_lin_chain(dvc, n.bf16, true, state ? delta::LIN_STATE : delta::LIN_PLAIN, st)))) return rc;
    if ((rc = hip_status(delta::launch_lin_chain(dkc, n.bf16, true, dg_log ? delta::LIN_SUMS : delta::LIN_PLAIN, st)))) return rc;
  }
  if (shared && (rc = hip_status(delta::launch_lin_share(w.dq, w.dk, dq, dk, rows, n.Hk, n.H / n.Hk, n.dk, n.bf16, st)))) return rc;
  return dg_log ? hip_status(delta::launch_lin_gates(gp, st)) : DELTA_OK;
}

int delta_decode_lin(const delta_shape* s, int32_t qk_heads, int32_t gate, const void* q, const void* k, const void* v,
                     const float* g_log, float* S, void* O, void* stream) {
  Lin n;
  int rc = lin_shape(s, qk_heads, gate, false, n);
  if (rc) return rc;
  if (s->L != 1) return DELTA_ERR_BAD_SHAPE;
  if ((rc = check_pointers({q, k, v, S, O}, n.nv > 0))) return rc;
  if ((gate == DELTA_LIN_GATE_NONE) != (g_log == nullptr) && (g_log || n.nv > 0)) return DELTA_ERR_NULL_ARG;
  if ((rc = check_aligned({q, k, v, S, O}, g_log, nullptr))) return rc;
  const Range in[] = {span(q, n.nqk), span(k, n.nqk), span(v, n.nv), span(g_log, n.ng)};
  const Range out[] = {span(S, n.state), span(O, n.nv)};
  if (any_overlap(in, out)) return DELTA_ERR_ALIAS;
  if (n.state == 0) return DELTA_OK;
  if ((rc = launch_guard())) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (g_log && validate_on() && (rc = validate_gates(g_log, n.ng / 4, st))) return rc;
  const LinDecode p{n.B, n.H, n.Hk, n.dk, n.dv, gate, n.scale, q, k, v, g_log, S, O};
  return hip_status(delta::launch_lin_decode(p, n.bf16, st));
}

}  // extern "C"
