// C-ABI layer of the gated delta rule: argument checks (host only, before any HIP
// call), the split into segments, workspace carving and the kernel sequence.
#include "zm_ttt.h"

#include <math.h>

#include <initializer_list>

#include "api_util.h"
#include "delta_rule.h"

using namespace zm;

namespace {

constexpr int64_t kMaxDeltaTokens = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxDeltaBlocks = ((int64_t)1 << 24) - 1;  // of 256 threads: a launch's grid
constexpr int64_t kMaxDeltaLd = (int64_t)1 << 24;
constexpr int kMaxDeltaHeads = 64;

int check_delta(const zm_delta_desc* d) {
  if (!d || d->heads < 1 || d->heads_k < 1 || d->d_head < 1 || d->n_seq < 0) return ZM_ERR_INVALID_ARG;
  if (d->io_dtype != ZM_BF16 && d->io_dtype != ZM_F32) return ZM_ERR_INVALID_ARG;
  if (d->heads % d->heads_k != 0 || !isfinite(d->scale)) return ZM_ERR_INVALID_ARG;
  const int64_t wk = (int64_t)d->heads_k * d->d_head, wv = (int64_t)d->heads * d->d_head;
  if (d->ld_q < wk || d->ld_k < wk || d->ld_v < wv || d->ld_o < wv) return ZM_ERR_INVALID_ARG;
  if (d->ld_q % 8 || d->ld_k % 8 || d->ld_v % 8 || d->ld_o % 8) return ZM_ERR_INVALID_ARG;
  if (d->ld_q > kMaxDeltaLd || d->ld_k > kMaxDeltaLd || d->ld_v > kMaxDeltaLd || d->ld_o > kMaxDeltaLd)
    return ZM_ERR_INVALID_ARG;
  if (d->heads > kMaxDeltaHeads || (d->d_head != 64 && d->d_head != 128)) return ZM_ERR_UNSUPPORTED;
  return ZM_OK;
}

int check_ptr(const void* p, size_t align) { return p && aligned(p, align) ? ZM_OK : ZM_ERR_INVALID_ARG; }

struct DeltaPlan {
  int n_chunks, n_segs, seg_chunks;
  int seg_room;  // segments the workspace has place for: at least n_segs, never fewer for more tokens
  bool split;    // sequences in several segments
};

// Upper bounds over every way n tokens can fall into n_seq sequences.
DeltaPlan delta_plan(const zm_delta_desc* d, int64_t n) {
  DeltaPlan p;
  p.n_chunks = (int)((n + (int64_t)(kChunk - 1) * d->n_seq) / kChunk);
  // One workgroup goes through a whole sequence of one head while these are enough
  // for half the compute units, or while the sequences are short; else a workgroup to
  // each segment of at least kMinSegChunks chunks, about kTargetWgs of them.
  // Measured with 8 heads of 128, us whole / in segments: bf16 384 tokens 43 / 50, 512
  // 54 / 52, 1560 150 / 71 (1374 in segments of 8 chunks 128, of 2 72); fp32 256 tokens
  // 70 / 71, 384 96 / 74; backward bf16 384 tokens 113 / 120, 1560 346 / 169.
  constexpr int kMinSegChunks = 2;
  const int64_t split_chunks = d->io_dtype == ZM_F32 ? 5 : 8;
  const int64_t units = (int64_t)d->n_seq * d->heads;
  int64_t seg = p.n_chunks > 0 ? p.n_chunks : 1;
  if (units < kTargetWgs / 2 && p.n_chunks >= split_chunks * d->n_seq) {
    seg = ceil_div((int64_t)p.n_chunks * d->heads, kTargetWgs);
    if (seg < kMinSegChunks) seg = kMinSegChunks;
  }
  p.seg_chunks = (int)seg;
  p.n_segs = (int)(p.n_chunks / seg) + d->n_seq;
  p.split = p.n_chunks > seg;
  if (!p.split) p.n_segs = d->n_seq;
  // n_segs falls where seg steps up; of chunks / seg neither chunks / kMinSegChunks nor
  // kTargetWgs / heads is ever passed
  const int64_t most = kTargetWgs / d->heads, room = p.n_chunks / kMinSegChunks;
  p.seg_room = p.split ? (int)(room < most ? room : most) + d->n_seq : d->n_seq;
  return p;
}

// Bump allocator over the workspace; with base null it only counts.
struct Carve {
  char* base;
  size_t at = 0;
  template <typename T>
  T* take(size_t count) {
    T* const p = base ? (T*)(base + at) : nullptr;
    at += round_up(count * sizeof(T), 256);
    return p;
  }
};

DeltaSeqs seqs(const zm_delta_desc* d, const DeltaPlan& p, int64_t n, const int* offsets, Carve& c) {
  DeltaSeqs s{};
  s.offsets = offsets;
  s.n = (int)n;
  s.n_seq = d->n_seq;
  s.n_chunks = p.n_chunks;
  s.n_segs = p.n_segs;
  s.seg_chunks = p.seg_chunks;
  // With more workgroups than compute units the long ones start first, so that they do
  // not end last: 61 sequences of 6 to 24 chunks, 16 heads, 510 -> 430 us.
  s.longest_first = !p.split && d->n_seq > 1 && d->n_seq <= kTableLds &&
                    (int64_t)d->n_seq * d->heads > kTargetWgs;
  if (d->n_seq > 1) {
    s.chunks = c.take<int4>(p.n_chunks);
    s.segs = c.take<int4>(p.seg_room);
    s.first_chunk = c.take<int>(d->n_seq + 1);
    s.begin = c.take<int>(d->n_seq + 1);
  }
  return s;
}

struct ForwardWs {
  DeltaArgs a;
  float* trans;
  float* starts;
  size_t bytes;
};

ForwardWs forward_ws(const zm_delta_desc* d, const DeltaPlan& p, int64_t n, const int* offsets, void* ws) {
  ForwardWs f{};
  Carve c{(char*)ws};
  f.a.sq = seqs(d, p, n, offsets, c);
  const size_t slots = (size_t)p.n_chunks * d->heads, tile = (size_t)kTriFrags * kFragElems;
  if (d->io_dtype == ZM_F32) {
    f.a.t_frags = c.take<uint16_t>(slots * 3 * tile);
    f.a.p_frags = c.take<uint16_t>(slots * 3 * tile);
    f.a.rows = c.take<float>(slots * 3 * kChunk);
  }
  if (p.split) {
    const size_t states = (size_t)p.seg_room * d->heads * d->d_head * d->d_head;
    f.trans = c.take<float>(2 * states);
    f.starts = c.take<float>(states);
  }
  f.bytes = c.at;
  f.a.heads = d->heads;
  f.a.heads_k = d->heads_k;
  f.a.d = d->d_head;
  f.a.scale = d->scale;
  f.a.f32 = d->io_dtype == ZM_F32;
  return f;
}

struct BackwardWs {
  DeltaArgs a;
  float *trans, *starts, *ends, *e;   // segments
  float *m_in, *d_m, *u, *x, *dq, *dk;
  size_t bytes;
};

BackwardWs backward_ws(const zm_delta_desc* d, const DeltaPlan& p, int64_t n, const int* offsets, void* ws) {
  BackwardWs f{};
  Carve c{(char*)ws};
  f.a.sq = seqs(d, p, n, offsets, c);
  const size_t slots = (size_t)p.n_chunks * d->heads, tile = (size_t)kTriFrags * kFragElems;
  const size_t dd = (size_t)d->d_head * d->d_head, rows = (size_t)n * d->heads * d->d_head;
  if (d->io_dtype == ZM_F32) f.a.t_frags = c.take<uint16_t>(slots * 3 * tile);
  f.a.tt_frags = c.take<uint16_t>(slots * 3 * tile);
  f.a.pt_frags = c.take<uint16_t>(slots * 3 * tile);
  f.a.rows = c.take<float>(slots * 3 * kChunk);
  if (p.split) {
    const size_t states = (size_t)p.seg_room * d->heads * dd;
    f.trans = c.take<float>(3 * states);
    f.starts = c.take<float>(states);
    f.ends = c.take<float>(states);
    f.e = c.take<float>(states);
  }
  f.m_in = c.take<float>(slots * dd);
  f.d_m = c.take<float>(slots * dd);
  f.u = c.take<float>(slots * kChunk * d->d_head);
  f.x = c.take<float>(slots * kChunk * d->d_head);
  if (d->heads != d->heads_k) {
    f.dq = c.take<float>(rows);
    f.dk = c.take<float>(rows);
  }
  f.bytes = c.at;
  f.a.heads = d->heads;
  f.a.heads_k = d->heads_k;
  f.a.d = d->d_head;
  f.a.scale = d->scale;
  f.a.f32 = d->io_dtype == ZM_F32;
  return f;
}

int check_counts(const zm_delta_desc* d, int64_t n) {
  if (n < 0 || n > kMaxDeltaTokens || (d->n_seq == 0 && n > 0)) return ZM_ERR_INVALID_ARG;
  const int64_t chunks = (n + (int64_t)(kChunk - 1) * d->n_seq) / kChunk;
  // a block to each (chunk or segment, head), of 768 threads at most (segments: a sequence
  // has one, and takes part in both terms) or of 512; the join has few
  if ((chunks + d->n_seq) * d->heads * 2 > kMaxDeltaBlocks) return ZM_ERR_UNSUPPORTED;
  return ZM_OK;
}

// The pointers of n tokens; offsets is optional for a single sequence.
int check_inputs(const zm_delta_desc* d, int64_t n, const int* offsets, const void* q, const void* k,
                 const void* v, const float* g, const float* beta) {
  if (d->n_seq > 1 || offsets) ZM_TRY(check_ptr(offsets, 4));
  if (n == 0) return ZM_OK;
  ZM_TRY(check_ptr(q, 16));
  ZM_TRY(check_ptr(k, 16));
  ZM_TRY(check_ptr(v, 16));
  ZM_TRY(check_ptr(g, 4));
  return check_ptr(beta, 4);
}

// An output in an input's place would be read after it is written (by other heads'
// workgroups, or by the second pass over segments), and of two outputs in one place one
// would be lost.  Null pointers are not arrays.
int check_apart(const void* out, std::initializer_list<const void*> others) {
  if (out)
    for (const void* p : others)
      if (p == out) return ZM_ERR_INVALID_ARG;
  return ZM_OK;
}

void set_inputs(DeltaArgs& a, const zm_delta_desc* d, const void* q, const void* k, const void* v,
                const float* g, const float* beta) {
  a.q = DeltaTokens{q, d->ld_q};
  a.k = DeltaTokens{k, d->ld_k};
  a.v = DeltaTokens{v, d->ld_v};
  a.g = g;
  a.beta = beta;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return ZM_OK;
  if (!ws) return ZM_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return ZM_ERR_INVALID_ARG;
  return have < need ? ZM_ERR_WORKSPACE : ZM_OK;
}

}  // namespace

extern "C" {

int zm_delta_rule_workspace_size(const zm_delta_desc* desc, int64_t n, size_t* bytes) {
  if (!bytes) return ZM_ERR_INVALID_ARG;
  ZM_TRY(check_delta(desc));
  ZM_TRY(check_counts(desc, n));
  *bytes = forward_ws(desc, delta_plan(desc, n), n, nullptr, nullptr).bytes;
  return ZM_OK;
}

int zm_delta_rule(const zm_delta_desc* desc, int64_t n, const int32_t* offsets, const void* q,
                  const void* k, const void* v, const float* g, const float* beta,
                  const float* state_in, float* state_out, void* o, void* workspace,
                  size_t workspace_bytes, void* stream) {
  ZM_TRY(check_delta(desc));
  ZM_TRY(check_counts(desc, n));
  ZM_TRY(check_inputs(desc, n, offsets, q, k, v, g, beta));
  if (n > 0) ZM_TRY(check_ptr(o, 16));
  if (n > 0) ZM_TRY(check_apart(o, {q, k, v, g, beta, offsets, state_in, state_out}));
  if (!aligned(state_in, 16) || !aligned(state_out, 16)) return ZM_ERR_INVALID_ARG;
  const DeltaPlan p = delta_plan(desc, n);
  ForwardWs f = forward_ws(desc, p, n, offsets, workspace);
  ZM_TRY(check_workspace(workspace, workspace_bytes, f.bytes));
  if (n > 0) ZM_TRY(check_apart(state_out, {q, k, v, g, beta, offsets}));  // it may be state_in
  if (desc->n_seq == 0) return ZM_OK;
  set_inputs(f.a, desc, q, k, v, g, beta);
  const hipStream_t st = (hipStream_t)stream;
  if (f.a.sq.chunks) ZM_HIP(launch_delta_table(f.a.sq, st));
  const auto scan = f.a.f32 ? launch_delta_scan : launch_delta_fused;
  if (f.a.f32) ZM_HIP(launch_delta_prep(f.a, false, st));
  DeltaScanArgs s{};
  s.state_in = state_in;
  s.state_out = state_out;
  s.o = o;
  s.ld_o = desc->ld_o;
  if (p.split) {
    s.trans = f.trans;
    ZM_HIP(scan(f.a, s, st));
    ZM_HIP(launch_delta_join(f.a, DeltaJoinArgs{state_in, f.trans, 2, nullptr, f.starts}, st));
    s.trans = nullptr;
    s.seg_start = f.starts;
  }
  ZM_HIP(scan(f.a, s, st));
  return ZM_OK;
}

int zm_delta_rule_step(const zm_delta_desc* desc, const void* q, const void* k, const void* v,
                       const float* g, const float* beta, float* state, void* o, void* stream) {
  ZM_TRY(check_delta(desc));
  if ((int64_t)desc->n_seq * desc->heads > kMaxDeltaBlocks) return ZM_ERR_UNSUPPORTED;
  if (desc->n_seq == 0) return ZM_OK;
  ZM_TRY(check_inputs(desc, desc->n_seq, (const int*)256, q, k, v, g, beta));
  ZM_TRY(check_ptr(state, 16));
  ZM_TRY(check_ptr(o, 16));
  ZM_TRY(check_apart(o, {q, k, v, g, beta, state}));
  DeltaStepArgs a{};
  a.q = DeltaTokens{q, desc->ld_q};
  a.k = DeltaTokens{k, desc->ld_k};
  a.v = DeltaTokens{v, desc->ld_v};
  a.g = g;
  a.beta = beta;
  a.state = state;
  a.o = o;
  a.ld_o = desc->ld_o;
  a.n_seq = desc->n_seq;
  a.heads = desc->heads;
  a.heads_k = desc->heads_k;
  a.d = desc->d_head;
  a.scale = desc->scale;
  a.f32 = desc->io_dtype == ZM_F32;
  ZM_HIP(launch_delta_step(a, (hipStream_t)stream));
  return ZM_OK;
}

int zm_delta_rule_backward_workspace_size(const zm_delta_desc* desc, int64_t n, size_t* bytes) {
  if (!bytes) return ZM_ERR_INVALID_ARG;
  ZM_TRY(check_delta(desc));
  ZM_TRY(check_counts(desc, n));
  *bytes = backward_ws(desc, delta_plan(desc, n), n, nullptr, nullptr).bytes;
  return ZM_OK;
}

int zm_delta_rule_backward(const zm_delta_desc* desc, int64_t n, const int32_t* offsets, const void* d_o,
                           const void* q, const void* k, const void* v, const float* g, const float* beta,
                           const float* state_in, const float* dstate_out, void* dq, int64_t ld_dq,
                           void* dk, int64_t ld_dk, void* dv, int64_t ld_dv, float* dg, float* dbeta,
                           float* dstate_in, void* workspace, size_t workspace_bytes, void* stream) {
  ZM_TRY(check_delta(desc));
  ZM_TRY(check_counts(desc, n));
  ZM_TRY(check_inputs(desc, n, offsets, q, k, v, g, beta));
  const int64_t wk = (int64_t)desc->heads_k * desc->d_head, wv = (int64_t)desc->heads * desc->d_head;
  if (ld_dq < wk || ld_dk < wk || ld_dv < wv || ld_dq % 8 || ld_dk % 8 || ld_dv % 8) return ZM_ERR_INVALID_ARG;
  if (ld_dq > kMaxDeltaLd || ld_dk > kMaxDeltaLd || ld_dv > kMaxDeltaLd) return ZM_ERR_INVALID_ARG;
  if (n > 0) {
    ZM_TRY(check_ptr(d_o, 16));
    ZM_TRY(check_ptr(dq, 16));
    ZM_TRY(check_ptr(dk, 16));
    ZM_TRY(check_ptr(dv, 16));
    ZM_TRY(check_ptr(dg, 4));
    ZM_TRY(check_ptr(dbeta, 4));
    ZM_TRY(check_apart(dq, {q, k, v, d_o, dk, dv}));
    ZM_TRY(check_apart(dk, {q, k, v, d_o, dv}));
    ZM_TRY(check_apart(dv, {q, k, v, d_o}));
  }
  if (!aligned(state_in, 16) || !aligned(dstate_out, 16) || !aligned(dstate_in, 16)) return ZM_ERR_INVALID_ARG;
  const DeltaPlan p = delta_plan(desc, n);
  BackwardWs f = backward_ws(desc, p, n, offsets, workspace);
  ZM_TRY(check_workspace(workspace, workspace_bytes, f.bytes));
  ZM_TRY(check_apart(dstate_in, {state_in}));  // dstate_in may be dstate_out
  if (n > 0) {
    const auto apart = [&](const void* out, std::initializer_list<const void*> others) {
      ZM_TRY(check_apart(out, {q, k, v, d_o, g, beta, offsets}));
      return check_apart(out, others);
    };
    for (const void* out : {(const void*)dq, (const void*)dk, (const void*)dv})
      ZM_TRY(apart(out, {dg, dbeta, dstate_in, dstate_out, state_in}));
    ZM_TRY(apart(dg, {dbeta, dstate_in, dstate_out, state_in}));
    ZM_TRY(apart(dbeta, {dstate_in, dstate_out, state_in}));
    ZM_TRY(apart(dstate_in, {}));
  }
  if (desc->n_seq == 0) return ZM_OK;
  set_inputs(f.a, desc, q, k, v, g, beta);
  const hipStream_t st = (hipStream_t)stream;
  if (f.a.sq.chunks) ZM_HIP(launch_delta_table(f.a.sq, st));
  ZM_HIP(launch_delta_prep(f.a, true, st));
  const auto scan = f.a.f32 ? launch_delta_scan : launch_delta_fused;
  DeltaScanArgs s{};
  s.state_in = state_in;
  DeltaGradArgs r{};
  r.d_o = DeltaTokens{d_o, desc->ld_o};
  r.dstate_out = dstate_out;
  if (p.split) {
    s.trans = f.trans;
    s.both = true;
    ZM_HIP(scan(f.a, s, st));
    ZM_HIP(launch_delta_join(f.a, DeltaJoinArgs{state_in, f.trans, 3, nullptr, f.starts}, st));
    s.trans = nullptr;
    s.seg_start = f.starts;
    r.e_out = f.e;
    ZM_HIP(launch_delta_reverse(f.a, r, st));
    ZM_HIP(launch_delta_join(f.a, DeltaJoinArgs{dstate_out, f.trans, 3, f.e, f.ends}, st));
    r.e_out = nullptr;
    r.seg_end = f.ends;
  }
  s.m_out = f.m_in;
  s.u_out = f.u;
  ZM_HIP(scan(f.a, s, st));
  r.dstate_in = dstate_in;
  r.m_in = f.m_in;
  r.d_m = f.d_m;
  r.u = f.u;
  r.x = f.x;
  r.dv = dv;
  r.ld_dv = ld_dv;
  r.dq = dq;
  r.dk = dk;
  r.ld_dq = ld_dq;
  r.ld_dk = ld_dk;
  r.dq_part = f.dq;
  r.dk_part = f.dk;
  r.dg = dg;
  r.dbeta = dbeta;
  ZM_HIP(launch_delta_reverse(f.a, r, st));
  ZM_HIP(launch_delta_grads(f.a, r, st));
  return ZM_OK;
}

}  // extern "C"
