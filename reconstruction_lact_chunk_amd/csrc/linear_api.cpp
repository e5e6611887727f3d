// C-ABI layer of linear attention with decays: argument checks (host only, before any HIP
// call), the split into segments, workspace carving and the kernel sequence.
#include "zm_ttt.h"

#include <math.h>

#include <initializer_list>

#include "api_util.h"
#include "linear_attn.h"

using namespace zm;

namespace {

constexpr int64_t kMaxLinTokens = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxLinBlocks = ((int64_t)1 << 24) - 1;  // of 256 threads: a launch's grid
constexpr int64_t kMaxLinLd = (int64_t)1 << 24;
constexpr int kMaxLinHeads = 64;

int check_stride(int64_t ld, int64_t width) {
  return ld < width || ld % 8 || ld > kMaxLinLd ? ZM_ERR_INVALID_ARG : ZM_OK;
}

int check_desc(const zm_linear_desc* d) {
  if (!d || d->heads < 1 || d->heads_k < 1 || d->d_head < 1 || d->n_seq < 0) return ZM_ERR_INVALID_ARG;
  if (d->io_dtype != ZM_BF16 && d->io_dtype != ZM_F32) return ZM_ERR_INVALID_ARG;
  if (d->heads % d->heads_k != 0 || !isfinite(d->scale)) return ZM_ERR_INVALID_ARG;
  const int64_t wk = (int64_t)d->heads_k * d->d_head, wv = (int64_t)d->heads * d->d_head;
  ZM_TRY(check_stride(d->ld_q, wk));
  ZM_TRY(check_stride(d->ld_k, wk));
  ZM_TRY(check_stride(d->ld_v, wv));
  ZM_TRY(check_stride(d->ld_o, wv));
  if (d->ld_g != 0 && (d->ld_g < d->heads || d->ld_g > kMaxLinLd)) return ZM_ERR_INVALID_ARG;
  if (d->heads > kMaxLinHeads || (d->d_head != 64 && d->d_head != 128)) return ZM_ERR_UNSUPPORTED;
  return ZM_OK;
}

int check_ptr(const void* p, size_t align) { return p && aligned(p, align) ? ZM_OK : ZM_ERR_INVALID_ARG; }

struct LinPlan {
  int64_t n_chunks;
  int n_segs, n_slots, n_split, seg_chunks, chunk;
  int64_t slots;      // states of segments that the workspace has place for
  int64_t splits;     // sequences of several segments, the same
  bool split;         // a sequence can have several segments
};

// Upper bounds over every way n tokens can fall into n_seq sequences.
LinPlan lin_plan(const zm_linear_desc* d, int64_t n) {
  LinPlan p;
  p.chunk = d->io_dtype == ZM_F32 ? 32 : 64;
  const int64_t ragged = (int64_t)(p.chunk - 1) * d->n_seq;
  p.n_chunks = (n + ragged) / p.chunk;
  // About this many workgroups in all, two to a compute unit.  8 heads of 128, bf16, us at
  // 256 / 512 / 1024: 10992 tokens 69 / 67 / 80, 40000 tokens 187 / 156 / 183.
  const int64_t target = 2 * kTargetWgs;
  int64_t seg = ceil_div(p.n_chunks * d->heads, target);
  // Segments of one chunk make the join long: 3000 tokens (47 chunks) of 8 heads 42 us, in
  // segments of two 35; 10000 of 2 heads 54 and 42; of fewer chunks one is better: 1374 tokens of 8 heads 31 and 34.
  const int64_t each = d->n_seq > 0 ? p.n_chunks / d->n_seq : 0;
  if (seg < 2 && each > 32) seg = 2;
  // The same of two in longer ones of one head: 33,000 tokens (516 chunks) 68 us, of three 58, their
  // gradient 137 and 114; 20,000 (313) 50 either way, 90 and 95.  No more than that where 512 workgroups take
  // fewer: 137,400 of one head in segments of 5 chunks 123 us, of 16 143.
  if (seg < 3 && each > 400) seg = 3;
  // Two chunks one after the other take less than two launches more: 128 tokens 17 us against
  // 21, 256 tokens (four chunks) 27 against 22.
  if (n <= 2 * p.chunk) seg = p.n_chunks;
  if (seg < 1) seg = 1;
  p.seg_chunks = (int)seg;
  const int64_t tokens = seg * p.chunk;
  // every segment but a sequence's last is full
  const int64_t full = n / tokens;
  p.split = n > tokens;
  p.n_segs = (int)((p.split ? full : 0) + d->n_seq);
  p.n_split = p.split ? (int)(full < d->n_seq ? full : d->n_seq) : 0;
  p.n_slots = p.split ? (int)full + p.n_split : 0;
  // Place for the full segments and one more of each sequence that has some.  full falls
  // where seg steps up, and with it split can; neither n / chunk nor target / heads is
  // passed, and split needs n (target - heads) > heads (ragged - chunk + 1), so that the
  // workspace never decreases with n.
  p.slots = p.splits = 0;
  if (n > p.chunk && n * (target - d->heads) > d->heads * (ragged - p.chunk + 1)) {
    const int64_t most = target / d->heads, all = n / p.chunk, room = all < most ? all : most;
    p.splits = room < d->n_seq ? room : d->n_seq;
    p.slots = room + p.splits;
  }
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

// The table, and what segments add; ways: 2 with the gradients.
void common_ws(LinArgs& a, Carve& c, const zm_linear_desc* d, const LinPlan& p, int64_t n, const int* offsets, int ways) {
  LinSeqs& s = a.sq;
  s.offsets = offsets;
  s.n = (int)n;
  s.n_seq = d->n_seq;
  s.n_segs = p.n_segs;
  s.n_slots = p.n_slots;
  s.n_split = p.n_split;
  // 70 sequences of 4 to 24 chunks, 16 heads: 303 us, in the order of the tokens 318
  s.longest_first = (int64_t)p.n_segs * d->heads > 2 * kTargetWgs && p.n_segs <= kLinSorted;
  s.seg_tokens = p.seg_chunks * p.chunk;
  s.chunk = p.chunk;
  if (d->n_seq > kLinWaveSeqs) {
    s.segs = c.take<LinSeg>(p.slots + d->n_seq);
    s.by_slot = c.take<int>(p.slots);
    s.by_split = c.take<int>(p.splits);
    s.all = c.take<int4>(1);
  }
  for (int i = 0; i < ways && p.slots > 0; ++i) {
    a.part[i] = c.take<float>((size_t)p.slots * d->heads * d->d_head * d->d_head);
    a.decay[i] = c.take<float2>((size_t)p.slots * d->heads);
  }
  a.heads = d->heads;
  a.heads_k = d->heads_k;
  a.scale = d->scale;
  a.ld_g = d->ld_g;
}

size_t forward_ws(LinArgs& a, const zm_linear_desc* d, const LinPlan& p, int64_t n, const int* offsets, void* ws) {
  Carve c{(char*)ws};
  common_ws(a, c, d, p, n, offsets, 1);
  return c.at;
}

// What dg alone needs comes last.
size_t backward_ws(LinArgs& a, const zm_linear_desc* d, const LinPlan& p, int64_t n, const int* offsets, void* ws,
                   bool dg, float** sums) {
  Carve c{(char*)ws};
  common_ws(a, c, d, p, n, offsets, 2);
  const size_t dd = (size_t)d->d_head * d->d_head, rows = (size_t)n * d->heads * d->d_head;
  if (d->heads != d->heads_k) {
    a.o_part = c.take<float>(rows);
    a.dk_part = c.take<float>(rows);
  }
  *sums = nullptr;
  if (!dg) return c.at;
  a.flow = c.take<float>((size_t)n * d->heads);
  a.d_dump = c.take<float>((size_t)p.n_chunks * d->heads * dd);
  a.d_exp = c.take<double>((size_t)p.n_chunks * d->heads);
  if (d->ld_g == 0) *sums = c.take<float>((size_t)p.n_chunks * d->heads);
  return c.at;
}

int check_counts(const zm_linear_desc* d, int64_t n) {
  if (n < 0 || n > kMaxLinTokens || (d->n_seq == 0 && n > 0)) return ZM_ERR_INVALID_ARG;
  // the largest grid: a block of 512 threads to each segment and head (the join's
  // 128 waves to a split sequence and head are at most 128 times 512)
  if (d->n_seq > kMaxLinBlocks || (int64_t)lin_plan(d, n).n_segs * d->heads * 2 > kMaxLinBlocks) return ZM_ERR_UNSUPPORTED;
  return ZM_OK;
}

// The pointers of n tokens; offsets is optional for a single sequence, g always.
int check_inputs(const zm_linear_desc* d, int64_t n, const int* offsets, const void* q, const void* k, const void* v,
                 const float* g) {
  if (d->n_seq > 1 || offsets) ZM_TRY(check_ptr(offsets, 4));
  if (!aligned(g, 4)) return ZM_ERR_INVALID_ARG;
  if (n == 0) return ZM_OK;
  ZM_TRY(check_ptr(q, 16));
  ZM_TRY(check_ptr(k, 16));
  return check_ptr(v, 16);
}

// An output in an input's place would be read after it is written, and of two outputs in
// one place one would be lost.  Null pointers are not arrays.
int check_apart(const void* out, std::initializer_list<const void*> others) {
  if (out)
    for (const void* p : others)
      if (p == out) return ZM_ERR_INVALID_ARG;
  return ZM_OK;
}

int backward_size(const zm_linear_desc* d, int64_t n, bool dg, size_t* bytes) {
  if (!bytes) return ZM_ERR_INVALID_ARG;
  ZM_TRY(check_desc(d));
  ZM_TRY(check_counts(d, n));
  LinArgs a{};
  float* sums;
  *bytes = backward_ws(a, d, lin_plan(d, n), n, nullptr, nullptr, dg, &sums);
  return ZM_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return ZM_OK;
  if (!ws) return ZM_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return ZM_ERR_INVALID_ARG;
  return have < need ? ZM_ERR_WORKSPACE : ZM_OK;
}

}  // namespace

extern "C" {

int zm_linear_attention_workspace_size(const zm_linear_desc* desc, int64_t n, size_t* bytes) {
  if (!bytes) return ZM_ERR_INVALID_ARG;
  ZM_TRY(check_desc(desc));
  ZM_TRY(check_counts(desc, n));
  LinArgs a{};
  *bytes = forward_ws(a, desc, lin_plan(desc, n), n, nullptr, nullptr);
  return ZM_OK;
}

int zm_linear_attention(const zm_linear_desc* desc, int64_t n, const int32_t* offsets, const void* q, const void* k,
                        const void* v, const float* g, const float* state_in, float* state_out, void* o,
                        void* workspace, size_t workspace_bytes, void* stream) {
  ZM_TRY(check_desc(desc));
  ZM_TRY(check_counts(desc, n));
  ZM_TRY(check_inputs(desc, n, offsets, q, k, v, g));
  if (!aligned(state_in, 16) || !aligned(state_out, 16)) return ZM_ERR_INVALID_ARG;
  if (n > 0) {
    ZM_TRY(check_ptr(o, 16));
    ZM_TRY(check_apart(o, {q, k, v, g, offsets, state_in, state_out}));
    ZM_TRY(check_apart(state_out, {q, k, v, g, offsets}));  // it may be state_in
  }
  const LinPlan p = lin_plan(desc, n);
  LinArgs a{};
  ZM_TRY(check_workspace(workspace, workspace_bytes, forward_ws(a, desc, p, n, offsets, workspace)));
  if (desc->n_seq == 0) return ZM_OK;
  a.q = LinTokens{q, desc->ld_q};
  a.k = LinTokens{k, desc->ld_k};
  a.v = LinTokens{v, desc->ld_v};
  a.g = g;
  a.state_in = state_in;
  a.state_out = state_out;
  a.o = o;
  a.ld_o = desc->ld_o;
  const hipStream_t st = (hipStream_t)stream;
  const bool f32 = desc->io_dtype == ZM_F32;
  if (a.sq.segs) ZM_HIP(launch_linear_table(a.sq, st));
  if (p.split) {
    ZM_HIP(launch_linear_states(a, desc->d_head, f32, st));
    ZM_HIP(launch_linear_join(a, desc->d_head, false, st));
  }
  ZM_HIP(launch_linear_out(a, desc->d_head, f32, st));
  return ZM_OK;
}

int zm_linear_attention_step(const zm_linear_desc* desc, const void* q, const void* k, const void* v, const float* g,
                             float* state, void* o, void* stream) {
  ZM_TRY(check_desc(desc));
  if ((int64_t)desc->n_seq * desc->heads > kMaxLinBlocks) return ZM_ERR_UNSUPPORTED;
  if (desc->n_seq == 0) return ZM_OK;
  ZM_TRY(check_inputs(desc, desc->n_seq, (const int*)256, q, k, v, g));
  ZM_TRY(check_ptr(state, 16));
  ZM_TRY(check_ptr(o, 16));
  ZM_TRY(check_apart(o, {q, k, v, g, state}));
  ZM_TRY(check_apart(state, {q, k, v, g}));
  LinStepArgs a{};
  a.q = LinTokens{q, desc->ld_q};
  a.k = LinTokens{k, desc->ld_k};
  a.v = LinTokens{v, desc->ld_v};
  a.g = g;
  a.ld_g = desc->ld_g;
  a.state = state;
  a.o = o;
  a.ld_o = desc->ld_o;
  a.n_seq = desc->n_seq;
  a.heads = desc->heads;
  a.heads_k = desc->heads_k;
  a.scale = desc->scale;
  ZM_HIP(launch_linear_step(a, desc->d_head, desc->io_dtype == ZM_F32, (hipStream_t)stream));
  return ZM_OK;
}

int zm_linear_attention_backward_workspace_size(const zm_linear_desc* desc, int64_t n, size_t* bytes) {
  return backward_size(desc, n, true, bytes);
}

int zm_linear_attention_backward_workspace_size_no_dg(const zm_linear_desc* desc, int64_t n, size_t* bytes) {
  return backward_size(desc, n, false, bytes);
}

int zm_linear_attention_backward(const zm_linear_desc* desc, int64_t n, const int32_t* offsets, const void* d_o,
                                 const void* q, const void* k, const void* v, const float* g, const float* state_in,
                                 const float* dstate_out, void* dq, int64_t ld_dq, void* dk, int64_t ld_dk, void* dv,
                                 int64_t ld_dv, float* dg, float* dstate_in, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  ZM_TRY(check_desc(desc));
  ZM_TRY(check_counts(desc, n));
  ZM_TRY(check_inputs(desc, n, offsets, q, k, v, g));
  const int64_t wk = (int64_t)desc->heads_k * desc->d_head, wv = (int64_t)desc->heads * desc->d_head;
  ZM_TRY(check_stride(ld_dq, wk));
  ZM_TRY(check_stride(ld_dk, wk));
  ZM_TRY(check_stride(ld_dv, wv));
  if (!aligned(state_in, 16) || !aligned(dstate_out, 16) || !aligned(dstate_in, 16) || !aligned(dg, 4))
    return ZM_ERR_INVALID_ARG;
  if (dg && !g) return ZM_ERR_INVALID_ARG;
  const bool one = desc->ld_g == 0;  // dg [heads] is written whatever n
  if (n > 0) {
    for (const void* p : {d_o, (const void*)dq, (const void*)dk, (const void*)dv}) ZM_TRY(check_ptr(p, 16));
    const void* const outs[] = {dq, dk, dv, dg, dstate_in};
    for (int i = 0; i < 5; ++i) {
      ZM_TRY(check_apart(outs[i], {q, k, v, d_o, g, offsets, state_in}));
      if (outs[i] != dstate_in) ZM_TRY(check_apart(outs[i], {dstate_out}));  // dstate_in may be dstate_out
      for (int j = 0; j < i; ++j) ZM_TRY(check_apart(outs[i], {outs[j]}));
    }
  }
  ZM_TRY(check_apart(dstate_in, {state_in}));
  const LinPlan p = lin_plan(desc, n);
  LinArgs a{};
  float* sums;
  const size_t need = backward_ws(a, desc, p, n, offsets, workspace, dg != nullptr, &sums);
  ZM_TRY(check_workspace(workspace, workspace_bytes, need));
  const hipStream_t st = (hipStream_t)stream;
  const bool f32 = desc->io_dtype == ZM_F32;
  const int d = desc->d_head;
  if (desc->n_seq > 0) {
    a.q = LinTokens{q, desc->ld_q};
    a.k = LinTokens{k, desc->ld_k};
    a.v = LinTokens{v, desc->ld_v};
    a.d_o = LinTokens{d_o, desc->ld_o};
    a.g = g;
    a.state_in = state_in;
    a.dstate_out = dstate_out;
    a.dstate_in = dstate_in;
    a.o = dq;
    a.ld_o = ld_dq;
    a.dk = dk;
    a.ld_dk = ld_dk;
    a.dv = dv;
    a.ld_dv = ld_dv;
    a.dg = one ? sums : dg;
    if (a.sq.segs) ZM_HIP(launch_linear_table(a.sq, st));
    if (p.split || a.flow) ZM_HIP(launch_linear_grad_states(a, d, f32, st));
    if (p.split) ZM_HIP(launch_linear_join(a, d, true, st));
    ZM_HIP(launch_linear_dkdv(a, d, f32, st));
    if (n > 0) ZM_HIP(launch_linear_dq(a, d, f32, st));
    if (n > 0 && a.o_part) {
      ZM_HIP(launch_linear_groups(a, d, f32, one ? dg : nullptr, st));
      return ZM_OK;
    }
  }
  if (dg && one) ZM_HIP(launch_linear_decay_sum(sums, a.sq, desc->heads, dg, st));
  return ZM_OK;
}

}  // extern "C"
