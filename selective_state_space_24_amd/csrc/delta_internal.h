// Launch parameters shared by the host dispatch and the gfx950 kernels of the gated delta rule.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

constexpr int kDeltaChunk = 64;      // steps per chunk
constexpr int kDeltaMaxKey = 128;    // largest dstate (entries of a key)

// What the kernels take of q, k, v and dy: rows that allow 16-byte access, 64 of which reach over
// less than 2 GB; q and k of exactly delta_pad_key(dk) entries, v and dy of v_cols. An input that
// is not so is copied into the workspace, padded with zeros, first.
struct DeltaPack {
  struct Item {
    const void* src;
    void* dst;              // (batch, heads, L, pad)
    int64_t sb, st, sh;     // strides of src (batch, L, heads, n)
    int64_t heads, n, pad;  // pad a multiple of 8
  } item[4];
  int64_t batch, L;
  int32_t count, bf16;
};

struct DeltaParams {
  const void* q;
  const void* k;
  const void* v;
  const void* g;
  const void* beta;
  void* y;
  const float* s0;   // nullable: (batch, nheads, headdim, dstate) fp32
  float* s_final;    // nullable
  float scale;
  int64_t batch, L, nheads, ngroups, dk, dv;
  int64_t rep;       // heads of a group, nheads / ngroups
  int64_t q_sb, q_st, q_sg, k_sb, k_st, k_sg, v_sb, v_st, v_sh, y_sb, y_st, y_sh;
  int64_t g_sb, g_st, g_sh, be_sb, be_st, be_sh;
  int64_t nchunks;   // ceil(L / kDeltaChunk)
  uint8_t* rec;      // workspace: one record per (batch, head, chunk), see delta_common.h
  // a sequence split into nseg segments of seg_chunks chunks (nseg 1: none of the buffers)
  int64_t nseg, seg_chunks;
  float* local;      // (batch, head, segment, dv, dk): the state a segment makes from zeros, and
                     // then, in the backward pass, the gradient before it of zeros after it
  uint8_t* trans;    // (batch, head, segment): the matrix it multiplies its initial state by, in
                     // image fragments
  float* starts;     // (batch, head, segment, dv, dk): the state each segment starts from, and then
                     // the gradient of the state after it
  uint8_t* image;    // backward workspace: the states and U, see delta_common.h
  int64_t v_cols;    // entries of a row of v (and dy) there are to read: dv rounded up to 8
  int32_t vec_y;     // rows of y (dv) allow 8-byte access and dv is a multiple of 4
  int32_t vec_state; // states allow 16-byte access and dk is a multiple of 4
  int32_t bf16;
  int32_t terms;     // bf16 terms of a computed operand: 3, or 2 where the caller chose 16 bits
};

// The backward pass: the forward's arguments (y's strides are dy's) and the gradients, written
// contiguous. The workspace holds f.rec, f.image and image_b.
struct DeltaBwdParams {
  DeltaParams f;
  const void* dy;
  const float* ds_final;  // nullable
  void* dq;
  void* dk;
  void* dv;
  void* dg;
  void* dbeta;
  float* ds0;             // nullable
  uint8_t* image_b;       // dS and dR
  int32_t vec_dv;         // rows of dv allow 8-byte access (and dv is a multiple of 4)
  int32_t vec_out;        // dq and dk allow 16-byte access and dk is a multiple of 8
};

// The padded key length: dk rounded up to 32, 64 or 128.
inline int delta_pad_key(int64_t dk) { return dk <= 32 ? 32 : (dk <= 64 ? 64 : 128); }
// Segments of a pass (sets nseg, seg_chunks), and the workspace they take beside the rest.
void delta_plan(DeltaParams* p);
struct DeltaSplitLayout {
  size_t local, trans, starts, total;
};
DeltaSplitLayout delta_split_layout(const DeltaParams& p);
// Bytes of one record of the forward or the backward pass, and of an image per (batch, head,
// chunk).
size_t delta_record_bytes(bool bf16, bool bwd);
size_t delta_image_bytes(int64_t dk, int64_t dv);
// Wavefronts (16 columns of v each) per workgroup of the scans: 4 or 8.
int delta_scan_waves(const DeltaParams& p);

hipError_t launch_delta_pack(const DeltaPack& p, hipStream_t stream);
hipError_t launch_delta_fwd(const DeltaParams& p, hipStream_t stream);
// the backward pass's forward half: records, states and U
hipError_t launch_delta_states(const DeltaParams& p, hipStream_t stream);
// the gradients of the states after the segments, from the last one to the first
hipError_t launch_delta_combine_back(const DeltaBwdParams& p, hipStream_t stream);
hipError_t launch_delta_bwd(const DeltaBwdParams& p, hipStream_t stream);
hipError_t launch_delta_update(const DeltaParams& p, float* state, int32_t vec, hipStream_t stream);

}  // namespace ssm
