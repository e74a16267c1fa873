// C ABI of the gated delta rule: argument validation and dispatch. Every check runs on the host
// before anything is enqueued; a failing call launches nothing.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "buffer_checks.h"
#include "delta_internal.h"
#include "scan_internal.h"
#include "ssm_delta.h"

namespace {

using ssm::aligned;
using ssm::Buf;
using ssm::check_buffers;

constexpr int64_t kMaxThreads = 0xffffffff;  // of a launch, along one dimension

// A tensor of up to three outer dimensions and an innermost one of stride 1.
struct Shape {
  int64_t n[4];
  int64_t s[3];
};

// Largest element offset + 1, or -1 on overflow.
int64_t extent(const Shape& t) {
  int64_t e = t.n[3];
  for (int i = 0; i < 4; ++i)
    if (t.n[i] == 0) return 0;
  for (int i = 0; i < 3; ++i) {
    int64_t x;
    if (__builtin_mul_overflow(t.n[i] - 1, t.s[i], &x) || __builtin_add_overflow(e, x, &e)) return -1;
  }
  int64_t bytes;
  return __builtin_mul_overflow(e, (int64_t)4, &bytes) ? -1 : e;
}

// True when no two indices share an element: taken by increasing stride, every dimension of size
// > 1 steps past the whole extent of the ones below it.
bool disjoint(const Shape& t) {
  int at[3], k = 0;
  for (int i = 0; i < 3; ++i) {
    if (t.n[i] == 0) return true;
    if (t.n[i] > 1) at[k++] = i;
  }
  for (int i = 1; i < k; ++i)
    for (int j = i; j > 0 && t.s[at[j]] < t.s[at[j - 1]]; --j) {
      const int x = at[j]; at[j] = at[j - 1]; at[j - 1] = x;
    }
  int64_t e = t.n[3];
  for (int i = 0; i < k; ++i) {
    if (t.s[at[i]] < e) return false;
    e += (t.n[at[i]] - 1) * t.s[at[i]];
  }
  return true;
}

Shape shape_q(const ssm_delta_desc& d) { return {{d.batch, d.seqlen, d.ngroups, d.dstate}, {d.q_stride_batch, d.q_stride_step, d.q_stride_group}}; }
Shape shape_k(const ssm_delta_desc& d) { return {{d.batch, d.seqlen, d.ngroups, d.dstate}, {d.k_stride_batch, d.k_stride_step, d.k_stride_group}}; }
Shape shape_v(const ssm_delta_desc& d) { return {{d.batch, d.seqlen, d.nheads, d.headdim}, {d.v_stride_batch, d.v_stride_step, d.v_stride_head}}; }
Shape shape_y(const ssm_delta_desc& d) { return {{d.batch, d.seqlen, d.nheads, d.headdim}, {d.y_stride_batch, d.y_stride_step, d.y_stride_head}}; }
Shape shape_g(const ssm_delta_desc& d) { return {{d.batch, d.seqlen, d.nheads, 1}, {d.g_stride_batch, d.g_stride_step, d.g_stride_head}}; }
Shape shape_beta(const ssm_delta_desc& d) { return {{d.batch, d.seqlen, d.nheads, 1}, {d.beta_stride_batch, d.beta_stride_step, d.beta_stride_head}}; }

int64_t chunks(const ssm_delta_desc& d) { return (d.seqlen + ssm::kDeltaChunk - 1) / ssm::kDeltaChunk; }
int64_t esize(const ssm_delta_desc& d) { return d.io_dtype == SSM_DTYPE_BF16 ? 2 : 4; }

int check_desc(const ssm_delta_desc* d) {
  if (!d) return SSM_ERR_NULL_ARG;
  if (d->io_dtype != SSM_DTYPE_F32 && d->io_dtype != SSM_DTYPE_BF16) return SSM_ERR_BAD_DTYPE;
  if (d->operands != SSM_DELTA_OPERANDS_24 && d->operands != SSM_DELTA_OPERANDS_16) return SSM_ERR_BAD_DTYPE;
  if (d->batch < 0 || d->seqlen < 0 || d->nheads < 1 || d->ngroups < 1 || d->nheads % d->ngroups ||
      d->dstate < 1 || d->dstate > SSM_DELTA_MAX_DSTATE || d->headdim < 1)
    return SSM_ERR_BAD_SHAPE;
  // room for every buffer of the passes, in bytes: a step of one head of one entry each way takes up
  // to 1400 (records 608, images 384, copies 320, a split's matrices 48)
  int64_t t = 4096, u;
  for (int64_t n : {d->batch, d->nheads, d->headdim, d->dstate})
    if (__builtin_mul_overflow(t, n > 0 ? n : 1, &t)) return SSM_ERR_BAD_SHAPE;
  if (__builtin_mul_overflow(t, d->seqlen + 64, &u)) return SSM_ERR_BAD_SHAPE;
  for (const Shape& s : {shape_q(*d), shape_k(*d), shape_v(*d), shape_g(*d), shape_beta(*d), shape_y(*d)}) {
    for (int64_t st : s.s)
      if (st < 0) return SSM_ERR_BAD_STRIDE;
    if (extent(s) < 0) return SSM_ERR_BAD_SHAPE;
  }
  return disjoint(shape_y(*d)) ? SSM_OK : SSM_ERR_BAD_STRIDE;
}

size_t state_bytes(const ssm_delta_desc& d) {
  return (size_t)d.batch * d.nheads * d.headdim * d.dstate * sizeof(float);
}

// 16-byte access to rows of `n` entries with the given base and strides, `n` a multiple of 8, and 64
// of them within 2 GB
bool row_access(const ssm_delta_desc& d, int64_t n, const void* base, const int64_t (&s)[3]) {
  const int64_t per = 16 / esize(d);
  return n % 8 == 0 && aligned(base, 16) && s[0] % per == 0 && s[1] % per == 0 && s[2] % per == 0 &&
         s[1] < ((int64_t)1 << 31) / (ssm::kDeltaChunk * esize(d));
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
int64_t value_pad(const ssm_delta_desc& d) { return (d.headdim + 7) / 8 * 8; }

// Room for a copy of q or k, and of v or dy (see DeltaPack), in whole chunks as the rest.
size_t key_copy(const ssm_delta_desc& d) {
  return align256((size_t)d.batch * d.ngroups * chunks(d) * ssm::kDeltaChunk * ssm::delta_pad_key(d.dstate) * esize(d));
}
size_t value_copy(const ssm_delta_desc& d) {
  return align256((size_t)d.batch * d.nheads * chunks(d) * ssm::kDeltaChunk * value_pad(d) * esize(d));
}

// Adds the copy of a tensor (n entries a row, `pad` in the copy) to the list if the kernels cannot
// take it as it is, and points base and strides at it.
void pack(const ssm_delta_desc& d, int64_t heads, int64_t n, int64_t pad, const void** base,
          int64_t* sb, int64_t* st, int64_t* sh, uint8_t* room, ssm::DeltaPack* list) {
  const int64_t s[3] = {*sb, *st, *sh};
  if (n == pad && row_access(d, n, *base, s)) return;
  ssm::DeltaPack::Item& t = list->item[list->count++];
  t = {*base, room, *sb, *st, *sh, heads, n, pad};
  *base = room;
  *st = pad;
  *sh = d.seqlen * pad;
  *sb = heads * d.seqlen * pad;
}
void pack_inputs(const ssm_delta_desc& d, ssm::DeltaParams* p, uint8_t* room, ssm::DeltaPack* list) {
  memset(list, 0, sizeof(*list));
  list->batch = d.batch;
  list->L = d.seqlen;
  list->bf16 = p->bf16;
  const int64_t key = ssm::delta_pad_key(d.dstate);
  pack(d, d.ngroups, d.dstate, key, &p->q, &p->q_sb, &p->q_st, &p->q_sg, room, list);
  pack(d, d.ngroups, d.dstate, key, &p->k, &p->k_sb, &p->k_st, &p->k_sg, room + key_copy(d), list);
  pack(d, d.nheads, d.headdim, value_pad(d), &p->v, &p->v_sb, &p->v_st, &p->v_sh, room + 2 * key_copy(d), list);
}

void fill(const ssm_delta_desc& d, const void* q, const void* k, const void* v, const void* g,
          const void* beta, float scale, ssm::DeltaParams* p) {
  memset(p, 0, sizeof(*p));
  p->q = q; p->k = k; p->v = v; p->g = g; p->beta = beta; p->scale = scale;
  p->batch = d.batch; p->L = d.seqlen; p->nheads = d.nheads; p->ngroups = d.ngroups;
  p->dk = d.dstate; p->dv = d.headdim; p->rep = d.nheads / d.ngroups;
  p->q_sb = d.q_stride_batch; p->q_st = d.q_stride_step; p->q_sg = d.q_stride_group;
  p->k_sb = d.k_stride_batch; p->k_st = d.k_stride_step; p->k_sg = d.k_stride_group;
  p->v_sb = d.v_stride_batch; p->v_st = d.v_stride_step; p->v_sh = d.v_stride_head;
  p->y_sb = d.y_stride_batch; p->y_st = d.y_stride_step; p->y_sh = d.y_stride_head;
  p->g_sb = d.g_stride_batch; p->g_st = d.g_stride_step; p->g_sh = d.g_stride_head;
  p->be_sb = d.beta_stride_batch; p->be_st = d.beta_stride_step; p->be_sh = d.beta_stride_head;
  p->nchunks = chunks(d);
  p->bf16 = d.io_dtype == SSM_DTYPE_BF16;
  p->terms = d.operands == SSM_DELTA_OPERANDS_16 ? 2 : 3;
  p->nseg = 1;
  p->seg_chunks = p->nchunks;
  p->v_cols = value_pad(d);
}

void set_split(int64_t nseg, int64_t seg_chunks, const ssm::DeltaSplitLayout& l, uint8_t* at, ssm::DeltaParams* p) {
  p->nseg = nseg;
  p->seg_chunks = seg_chunks;
  if (nseg <= 1) return;
  p->local = reinterpret_cast<float*>(at + l.local);
  p->trans = at + l.trans;
  p->starts = reinterpret_cast<float*>(at + l.starts);
}

// Workspace of the forward pass: records, what a split sequence takes, copies of inputs.
struct FwdLayout {
  int64_t nseg, seg_chunks;
  ssm::DeltaSplitLayout split;
  size_t records, copies, total;
};
FwdLayout fwd_layout(const ssm_delta_desc& d) {
  ssm::DeltaParams p;
  fill(d, nullptr, nullptr, nullptr, nullptr, nullptr, 0.0f, &p);
  ssm::delta_plan(&p);
  FwdLayout l;
  l.nseg = p.nseg;
  l.seg_chunks = p.seg_chunks;
  l.split = ssm::delta_split_layout(p);
  l.records = align256((size_t)d.batch * d.nheads * p.nchunks * ssm::delta_record_bytes(p.bf16, false));
  l.copies = l.records + l.split.total;
  l.total = l.copies + 2 * key_copy(d) + value_copy(d);
  return l;
}

// Workspace of the backward pass: records, the forward image, the backward image, what a split
// sequence takes, copies of inputs.
struct BwdLayout {
  int64_t nseg, seg_chunks;
  ssm::DeltaSplitLayout split;
  size_t image, image_b, split_at, copies, total;
};
BwdLayout bwd_layout(const ssm_delta_desc& d) {
  ssm::DeltaParams p;
  fill(d, nullptr, nullptr, nullptr, nullptr, nullptr, 0.0f, &p);
  ssm::delta_plan(&p);
  const size_t items = (size_t)d.batch * d.nheads * p.nchunks;
  const size_t img = items * ssm::delta_image_bytes(d.dstate, d.headdim);
  BwdLayout l;
  l.nseg = p.nseg;
  l.seg_chunks = p.seg_chunks;
  l.split = ssm::delta_split_layout(p);
  l.image = align256(items * ssm::delta_record_bytes(p.bf16, true));
  l.image_b = l.image + img;
  l.split_at = align256(l.image_b + img);
  l.copies = l.split_at + l.split.total;
  l.total = l.copies + 2 * key_copy(d) + 2 * value_copy(d);
  return l;
}

// Every launch of a pass that is not split (a split one has few heads) has a 32-bit number of threads.
bool launchable(const ssm::DeltaParams& p, bool bwd) {
  const int64_t heads = p.batch * p.nheads, columns = 16 * ssm::delta_scan_waves(p);
  return p.nchunks <= kMaxThreads / 256 && heads * ((p.dv + columns - 1) / columns) <= kMaxThreads / (4 * columns) &&
         (!bwd || p.batch * p.ngroups * p.nchunks <= kMaxThreads / 512);
}

int run_status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

}  // namespace

extern "C" {

int ssm_delta_desc_init_contiguous(ssm_delta_desc* d, int64_t batch, int64_t seqlen,
                                   int64_t nheads, int64_t ngroups, int64_t dstate,
                                   int64_t headdim, int32_t io_dtype) {
  if (!d) return SSM_ERR_NULL_ARG;
  memset(d, 0, sizeof(*d));
  d->batch = batch; d->seqlen = seqlen; d->nheads = nheads; d->ngroups = ngroups;
  d->dstate = dstate; d->headdim = headdim; d->io_dtype = io_dtype;
  d->q_stride_group = d->k_stride_group = dstate;
  d->q_stride_step = d->k_stride_step = ngroups * dstate;
  d->q_stride_batch = d->k_stride_batch = seqlen * ngroups * dstate;
  d->v_stride_head = d->y_stride_head = headdim;
  d->v_stride_step = d->y_stride_step = nheads * headdim;
  d->v_stride_batch = d->y_stride_batch = seqlen * nheads * headdim;
  d->g_stride_head = d->beta_stride_head = 1;
  d->g_stride_step = d->beta_stride_step = nheads;
  d->g_stride_batch = d->beta_stride_batch = seqlen * nheads;
  return SSM_OK;
}

int ssm_gated_delta_workspace_size(const ssm_delta_desc* desc, size_t* bytes) {
  if (!bytes) return SSM_ERR_NULL_ARG;
  const int rc = check_desc(desc);
  if (rc != SSM_OK) return rc;
  *bytes = fwd_layout(*desc).total;
  return SSM_OK;
}

int ssm_gated_delta_fwd(const ssm_delta_desc* desc, const void* q, const void* k, const void* v,
                        const void* g, const void* beta, float scale, const float* s0, void* y,
                        float* s_final, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int rc = ssm_gated_delta_workspace_size(desc, &need);
  if (rc != SSM_OK) return rc;
  const ssm_delta_desc& d = *desc;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  const size_t es = esize(d), sb = state_bytes(d);
  if (d.batch == 0) return SSM_OK;
  const bool steps = d.seqlen > 0;
  if (steps && (!q || !k || !v || !g || !beta || !y)) return SSM_ERR_NULL_ARG;
  const Buf in[] = {{q, extent(shape_q(d)) * es, es}, {k, extent(shape_k(d)) * es, es},
                    {v, extent(shape_v(d)) * es, es}, {g, extent(shape_g(d)) * es, es},
                    {beta, extent(shape_beta(d)) * es, es}, {s0, sb, 4}};
  const Buf out[] = {{steps ? y : nullptr, extent(shape_y(d)) * es, es}, {s_final, sb, 4},
                     {steps ? workspace : nullptr, need, 16}};
  if (steps && (!workspace || workspace_bytes < need)) return SSM_ERR_WORKSPACE;
  rc = check_buffers(in, 6, out, 3);
  if (rc != SSM_OK) return rc;
  if (!steps)
    return s_final ? run_status(ssm::launch_state_copy(s0, s_final, (int64_t)(sb / 4), hs)) : SSM_OK;
  ssm::DeltaParams p;
  fill(d, q, k, v, g, beta, scale, &p);
  if (!launchable(p, false)) return SSM_ERR_UNSUPPORTED;
  p.y = y; p.s0 = s0; p.s_final = s_final;
  // (row_access asks more of y than its 8-byte stores need)
  p.vec_y = row_access(d, d.headdim, y, shape_y(d).s);
  p.vec_state = d.dstate % 4 == 0 && aligned(s0, 16) && aligned(s_final, 16);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const FwdLayout lay = fwd_layout(d);
  p.rec = ws;
  set_split(lay.nseg, lay.seg_chunks, lay.split, ws + lay.records, &p);
  ssm::DeltaPack list;
  pack_inputs(d, &p, ws + lay.copies, &list);
  hipError_t e = ssm::launch_delta_pack(list, hs);
  if (e == hipSuccess) e = ssm::launch_delta_fwd(p, hs);
  return run_status(e);
}

int ssm_gated_delta_update(const ssm_delta_desc* desc, float* state, const void* q, const void* k,
                           const void* v, const void* g, const void* beta, float scale, void* y,
                           void* stream) {
  int rc = check_desc(desc);
  if (rc != SSM_OK) return rc;
  const ssm_delta_desc& d = *desc;
  if (d.seqlen != 1) return SSM_ERR_BAD_SHAPE;
  if (d.batch == 0) return SSM_OK;
  if (!state || !q || !k || !v || !g || !beta || !y) return SSM_ERR_NULL_ARG;
  const size_t es = esize(d);
  const Buf in[] = {{q, extent(shape_q(d)) * es, es}, {k, extent(shape_k(d)) * es, es},
                    {v, extent(shape_v(d)) * es, es}, {g, extent(shape_g(d)) * es, es},
                    {beta, extent(shape_beta(d)) * es, es}};
  const Buf out[] = {{y, extent(shape_y(d)) * es, es}, {state, state_bytes(d), 4}};
  rc = check_buffers(in, 5, out, 2);
  if (rc != SSM_OK) return rc;
  // (with more heads than that, a wavefront takes 32 rows)
  if (d.batch * d.nheads * ((d.headdim + 31) / 32) > kMaxThreads / 256 * 4) return SSM_ERR_UNSUPPORTED;
  ssm::DeltaParams p;
  fill(d, q, k, v, g, beta, scale, &p);
  p.y = y;
  // 4 entries of q and k in one load, 16-byte pieces of the state
  bool vec = d.dstate % 4 == 0 && aligned(q, 4 * es) && aligned(k, 4 * es) && aligned(state, 16);
  for (int64_t s : {d.q_stride_batch, d.q_stride_group, d.k_stride_batch, d.k_stride_group})
    vec = vec && s % 4 == 0;
  return run_status(ssm::launch_delta_update(p, state, vec, static_cast<hipStream_t>(stream)));
}

int ssm_gated_delta_bwd_workspace_size(const ssm_delta_desc* desc, size_t* bytes) {
  if (!bytes) return SSM_ERR_NULL_ARG;
  const int rc = check_desc(desc);
  if (rc != SSM_OK) return rc;
  *bytes = bwd_layout(*desc).total;
  return SSM_OK;
}

int ssm_gated_delta_bwd(const ssm_delta_desc* desc, const void* q, const void* k, const void* v,
                        const void* g, const void* beta, float scale, const float* s0,
                        const void* dy, const float* ds_final, void* dq, void* dk, void* dv,
                        void* dg, void* dbeta, float* ds0, void* workspace,
                        size_t workspace_bytes, void* stream) {
  int rc = check_desc(desc);
  if (rc != SSM_OK) return rc;
  const ssm_delta_desc& d = *desc;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  if (d.batch == 0) return SSM_OK;
  const size_t es = esize(d), sb = state_bytes(d);
  const bool steps = d.seqlen > 0;
  if (steps && (!q || !k || !v || !g || !beta || !dy || !dq || !dk || !dv || !dg || !dbeta))
    return SSM_ERR_NULL_ARG;
  const BwdLayout lay = bwd_layout(d);
  if (steps && (!workspace || workspace_bytes < lay.total)) return SSM_ERR_WORKSPACE;
  const size_t per_step = (size_t)d.batch * d.seqlen * es;
  const size_t qk_bytes = per_step * d.ngroups * d.dstate, g_bytes = per_step * d.nheads;
  const Buf in[] = {{q, extent(shape_q(d)) * es, es}, {k, extent(shape_k(d)) * es, es},
                    {v, extent(shape_v(d)) * es, es}, {g, extent(shape_g(d)) * es, es},
                    {beta, extent(shape_beta(d)) * es, es}, {dy, extent(shape_y(d)) * es, es},
                    {s0, sb, 4}, {ds_final, sb, 4}};
  const Buf out[] = {{dq, qk_bytes, es}, {dk, qk_bytes, es}, {dv, g_bytes * d.headdim, es},
                     {dg, g_bytes, es}, {dbeta, g_bytes, es}, {ds0, sb, 4},
                     {steps ? workspace : nullptr, lay.total, 16}};
  rc = check_buffers(in, 8, out, 7);
  if (rc != SSM_OK) return rc;
  if (!steps)
    return ds0 ? run_status(ssm::launch_state_copy(ds_final, ds0, (int64_t)(sb / 4), hs)) : SSM_OK;
  ssm::DeltaBwdParams p;
  memset(&p, 0, sizeof(p));
  fill(d, q, k, v, g, beta, scale, &p.f);
  if (!launchable(p.f, true)) return SSM_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.f.s0 = s0;
  p.f.rec = ws; p.f.image = ws + lay.image; p.image_b = ws + lay.image_b;
  set_split(lay.nseg, lay.seg_chunks, lay.split, ws + lay.split_at, &p.f);
  p.dy = dy; p.ds_final = ds_final;
  p.dq = dq; p.dk = dk; p.dv = dv; p.dg = dg; p.dbeta = dbeta; p.ds0 = ds0;
  p.vec_dv = d.headdim % 4 == 0 && aligned(dv, 8);
  p.vec_out = d.dstate % 8 == 0 && aligned(dq, 16) && aligned(dk, 16);
  p.f.vec_state = d.dstate % 4 == 0 && aligned(s0, 16) && aligned(ds_final, 16) && aligned(ds0, 16);
  ssm::DeltaPack list;
  uint8_t* room = ws + lay.copies;
  pack_inputs(d, &p.f, room, &list);
  pack(d, d.nheads, d.headdim, value_pad(d), &p.dy, &p.f.y_sb, &p.f.y_st, &p.f.y_sh,
       room + 2 * key_copy(d) + value_copy(d), &list);
  hipError_t e = ssm::launch_delta_pack(list, hs);
  if (e == hipSuccess) e = ssm::launch_delta_bwd(p, hs);
  return run_status(e);
}

}  // extern "C"
