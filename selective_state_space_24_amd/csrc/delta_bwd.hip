// gfx950 kernels of the gated delta rule's backward pass (formulas and tile layouts in
// delta_common.h). After the forward half has made T, P, the state S before each chunk and U:
//
// 1. The reverse scan, last chunk first, with dS the gradient of the state after the chunk:
//      dU = e^{G_63 - G} (K dS) + P^T dY,  dR = T^T dU,  dV = beta dR
//      dS' = e^{G_63} dS + Q^T (scale e^G dY) - K^T (beta e^G dR)
//    Columns of v are on their own, as in the forward scan, and the layout is the same. dS and dR
//    go to the second image.
// 2. The gradient kernel, every chunk at once. With E_ts = dY_t . U_s, N_ts = -dR_t . U_s:
//      dQ_t = scale e^{G_t} S dY_t + sum_{s <= t} scale D_ts E_ts K_s
//      dK_s = sum_{t >= s} scale D_ts E_ts Q_t + sum_x M_xs K_x - beta_s e^{G_s} S dR_s
//             + e^{G_63 - G_s} dS U_s,    M_ts = M_st = beta_t D_ts N_ts (s < t)
//      dbeta_t = dR_t . V_t - e^{G_t} K_t . (S dR_t) + sum_{s < t} N_ts D_ts K_t . K_s
//      dG_x = sum_{s < x} (E.P + N.A)_xs - sum_{t > x} (E.P + N.A)_tx + Q_x . (scale e^{G_x} S dY_x)
//             - K_x . (beta_x e^{G_x} S dR_x) - K_x . (e^{G_63 - G_x} dS U_x)
//             (at 63 instead of the last: + sum_{s < 63} K_s . (e^{G_63 - G_s} dS U_s) + e^{G_63} <S, dS>)
//      dg_t = sum_{x >= t} dG_x
#include "delta_common.h"

namespace ssm {

using namespace delta;

namespace {

// --- reverse scan ------------------------------------------------------------------------------
template <class P, int KK, int NW>
struct BackLds {
  typedef Record<P, true> Rec;
  typedef Mover<P, KK, NW, 2> Move;
  static constexpr int kK = 0;
  static constexpr int kQ = 4 * KK * P::kFrag;
  static constexpr int kRec = 2 * kQ;
  static constexpr int kRows = kRec + Rec::kRows;
  static constexpr int kBytes = kRec + Rec::kBytes;
  static constexpr Buffers kBuf = buffers(kBytes, Move::kTileBytes);  // tiles of dY
  static constexpr int kAll = kBuf.n * kBytes + kBuf.tiles * Move::kTileBytes;
};

// Four products to the forward scan's five, with T and P transposed on the way out of LDS: 740 us for
// batch 4, 8192 steps of 64 heads, 128 x 64 in bf16 (680 with 16-bit operands), of which 1.6 GB of
// image written take 330 us at a copy's rate. There 256 workgroups of four wavefronts leave one to a
// SIMD, which spends 27 % of the time in matrix and 24 % in other vector instructions; the LDS is busy
// 43 % of it, 29 % with the bank conflicts of the transposed reads.
//
// dV leaves a chunk late, as the forward scan's y does. Where the sequence is split, a first run
// (LOCAL) makes what each segment but the first adds to the gradient of the state before it, from
// zeros after it; dS passes from segment to segment by M^T; and every segment then runs from its own.
template <class P, int KK, int NW, bool LOCAL>
__global__ void __launch_bounds__(64 * NW) delta_back_kernel(const DeltaBwdParams q) {
  typedef typename P::IO IO;
  typedef BackLds<P, KK, NW> Lds;
  typedef typename Lds::Rec Rec;
  constexpr int NT = P::kTerms;
  constexpr int NBUF = Lds::kBuf.n, YBUF = Lds::kBuf.tiles;
  const DeltaParams& p = q.f;
  __shared__ __attribute__((aligned(16))) uint8_t smem[Lds::kAll];
  lds_u8* const sm = (lds_u8*)smem;
  auto tile_at = [&](int buf) { return sm + NBUF * Lds::kBytes + (YBUF == 2 ? buf : 0) * Lds::Move::kTileBytes; };
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // 32-bit arithmetic: there are fewer than 2^31 items
  const uint32_t slices = (uint32_t)((p.dv + 16 * NW - 1) / (16 * NW));
  const uint32_t item = (uint32_t)die_item(blockIdx.x, gridDim.x);
  const uint32_t segs = (uint32_t)p.nseg - LOCAL, runs = item / slices;
  const int64_t bh = runs / segs, seg = runs - (uint32_t)bh * segs + LOCAL, bhs = bh * p.nseg + seg;
  const uint32_t b = (uint32_t)bh / (uint32_t)p.nheads, h = (uint32_t)bh - b * (uint32_t)p.nheads;
  const uint32_t grp = h / (uint32_t)p.rep;
  const int64_t slice0 = (int64_t)(item % slices) * (16 * NW);
  const int64_t col = slice0 + 16 * w + c;
  const bool live = col < p.dv;
  const int dk = (int)p.dk;
  const int64_t L = p.L, nch = p.nchunks;
  const int64_t c0 = seg * p.seg_chunks, c1 = c0 + p.seg_chunks < nch ? c0 + p.seg_chunks : nch;
  const IO* Kp = static_cast<const IO*>(p.k) + b * p.k_sb + grp * p.k_sg;
  const IO* Qp = static_cast<const IO*>(p.q) + b * p.q_sb + grp * p.q_sg;
  const IO* DYp = static_cast<const IO*>(q.dy) + b * p.y_sb + h * p.y_sh;
  IO* DVp = static_cast<IO*>(q.dv) + (b * L * p.nheads + h) * p.dv;
  const int64_t dv_st = p.nheads * p.dv;
  const uint8_t* rec = p.rec + bh * nch * (int64_t)Rec::kBytes;
  const int64_t tile = (slice0 >> 4) + w, img_slices = (p.dv + 31) / 32;
  const int64_t img_chunk = img_slices * Image<P, KK>::kBytes;
  uint8_t* const image = !LOCAL && tile < 2 * img_slices
                             ? q.image_b + bh * nch * img_chunk + (tile >> 1) * Image<P, KK>::kBytes : nullptr;
  const int img_s = (int)(tile & 1) * KK * Image<P, KK>::kFrag, img_u = (int)(tile & 1) * 2 * Image<P, KK>::kFrag;

  typename Lds::Move mv;
  auto place = [&](int rows) {
    const int64_t st[2] = {p.k_st, p.q_st};
    mv.place(w, lane, rows, st, p.y_st, p.v_cols - slice0);
  };
  // the loads of a chunk in parts, as in the forward scan
  constexpr int kPoints = KK + 4;
  constexpr int kFragN = Lds::Move::kFragSteps, kTileN = YBUF == NBUF ? Lds::Move::kTileSteps : 0;
  constexpr int kSteps = kFragN + kTileN + (Rec::kBytes / 1024 + NW - 1) / NW;
  auto load_part = [&](int64_t ch, int buf, int first, int last) {
    lds_u8* const to = sm + buf * Lds::kBytes;
    const int64_t t0 = ch * kC;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s < first * kSteps / kPoints || s >= last * kSteps / kPoints) continue;
      if (s < kFragN) mv.frag_step(s, w, Kp + t0 * p.k_st, Qp + t0 * p.q_st, to + Lds::kK);
      else if (s < kFragN + kTileN) mv.row_step(s - kFragN, w, DYp + t0 * p.y_st + slice0, tile_at(buf));
      else
        Lds::Move::template run_step<Rec::kBytes / 1024>(s - kFragN - kTileN, w, lane,
                                                         rec + ch * (int64_t)Rec::kBytes, to + Lds::kRec);
    }
  };
  auto load_late_tile = [&](int64_t ch) {
    if constexpr (YBUF != NBUF) {
#pragma unroll
      for (int i = 0; i < Lds::Move::kTileSteps; ++i) mv.row_step(i, w, DYp + ch * kC * p.y_st + slice0, tile_at(0));
    }
  };

  f32x4 S[2 * KK];  // dS, laid out as the forward scan's S
#pragma unroll
  for (int a = 0; a < 2 * KK; ++a) S[a] = f32x4{0, 0, 0, 0};
  const float* after = LOCAL ? nullptr : seg + 1 < p.nseg ? p.starts + bhs * (p.dv * p.dk)
                               : q.ds_final ? q.ds_final + bh * (p.dv * p.dk) : nullptr;
  if (after && live) load_state<KK>(after + col * p.dk, dk, p.vec_state, g, S);
  RowStore<P> late;  // dV of the chunk after
  auto store_late = [&](int64_t ch) {
    const int64_t left = L - ch * kC;
    late.store(DVp + ch * kC * dv_st, dv_st, left < kC ? (int)left : kC, slice0 + 16 * w, p.dv, q.vec_dv, lane);
  };
  place((int)(L - (c1 - 1) * kC < kC ? L - (c1 - 1) * kC : kC));
  load_part(c1 - 1, 0, 0, kPoints);
  load_late_tile(c1 - 1);
  place(kC);
  wait_vmem_all();
  sync_lds();

  for (int64_t ch = c1 - 1; ch >= c0; --ch) {
    const int buf = NBUF == 2 ? (int)((c1 - 1 - ch) & 1) : 0;
    lds_u8* const B = sm + buf * Lds::kBytes;
    const lds_u8* const rows = B + Lds::kRows;
    f32x4 d[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const f32x4 on = lds16f(rows + Rec::kOn + tile_row4(a, g) * 4);
      d[a] = P::template load_col4<Lds::Move::kPitch>(tile_at(buf), tile_row4(a, g), 16 * w, c);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[a][i] = live && on[i] != 0.0f ? d[a][i] : 0.0f;
    }
    const bool more = ch > c0;
    auto point = [&](int i) {
      if constexpr (NBUF == 2) {
        if (more) load_part(ch - 1, buf ^ 1, i, i + 1);
      }
    };
    if (image) {
      uint8_t* im = image + ch * img_chunk + Image<P, KK>::kS + img_s;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) P::put_kept(im + kk * Image<P, KK>::kFrag, lane, S[2 * kk], S[2 * kk + 1]);
    }
    if constexpr (!LOCAL) {
      if (ch + 1 < c1) store_late(ch + 1);
    }
    typedef typename P::Exact Exact;
    typedef typename P::template Terms<NT> TermsT;
    auto get_rows = [&](Exact (&f)[4], int kk) {
#pragma unroll
      for (int a = 0; a < 4; ++a) f[a] = P::load_frag(B + Lds::kK + (a * KK + kk) * P::kFrag, lane);
    };
    // the transposes of T and P, rows of tiles a0 and a0 + 1
    auto get_tt = [&](TermsT (&t)[2], int mat, int block, int kk, int a0) {
#pragma unroll
      for (int a = 0; a < 2; ++a)
        P::load_terms_t(B + Lds::kRec + mat + tri_block(2 * kk, a0 >> 1) * block,
                        B + Lds::kRec + mat + tri_block(2 * kk + 1, a0 >> 1) * block, a0 + a, lane, t[a]);
    };
    // dU
    f32x4 du[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) du[a] = f32x4{0, 0, 0, 0};
    Exact fk[2][4];
    TermsT tp[2];
    get_rows(fk[0], 0);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      if (kk + 1 < KK) get_rows(fk[(kk + 1) & 1], kk + 1);
      else get_tt(tp, Rec::kP, Rec::kPBlock, 0, 0);
      TermsT s;
      P::split(S[2 * kk], S[2 * kk + 1], s);
      point(kk);
      __builtin_amdgcn_sched_barrier(0);
      P::template mma_rows<NT>(fk[kk & 1], s, du);
    }
    if constexpr (YBUF != NBUF) {
      if (more) {
        sync_lds();  // every wavefront has read its columns of dY
        load_late_tile(ch - 1);
      }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const f32x4 dec = lds16f(rows + Rec::kDecay + tile_row4(a, g) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) du[a][i] *= dec[i];
    }
    TermsT tt[2];
#pragma unroll
    for (int n3 = 0; n3 < 3; ++n3) {  // (kk, a0): (0, 0), (1, 0), (1, 2)
      const Exact e = P::exact(d[n3 ? 2 : 0], d[n3 ? 3 : 1]);
      TermsT now[2] = {tp[0], tp[1]};
      if (n3 < 2) get_tt(tp, Rec::kP, Rec::kPBlock, 1, 2 * n3);
      else get_tt(tt, Rec::kT, Rec::kTBlock, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      const int a0 = n3 == 2 ? 2 : 0;
#pragma unroll
      for (int a = 0; a < 2; ++a) du[a0 + a] = P::mma_te(now[a], e, du[a0 + a]);
    }
    // dR
    f32x4 dr[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) dr[a] = f32x4{0, 0, 0, 0};
    {
      TermsT e;
      P::split(du[0], du[1], e);
      point(KK);
#pragma unroll
      for (int n3 = 0; n3 < 3; ++n3) {
        TermsT now[2] = {tt[0], tt[1]};
        if (n3 < 2) get_tt(tt, Rec::kT, Rec::kTBlock, 1, 2 * n3);
        if (n3 == 1) {
          P::split(du[2], du[3], e);
          point(KK + 1);
        }
        __builtin_amdgcn_sched_barrier(0);
        P::mma_tt_rows(now, e, dr + (n3 == 2 ? 2 : 0));
      }
    }
    if (image) {
      uint8_t* im = image + ch * img_chunk + Image<P, KK>::kU + img_u;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) P::put_kept(im + kk * Image<P, KK>::kFrag, lane, dr[2 * kk], dr[2 * kk + 1]);
    }
    // dV, and the weighted rows of dY and dR
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = tile_row4(a, g) * 4;
      const f32x4 eg = lds16f(rows + Rec::kGrow + r), be = lds16f(rows + Rec::kBeta + r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dr[a][i] *= be[i];
        d[a][i] *= p.scale * eg[i];
      }
    }
    if constexpr (!LOCAL) late.take(dr, c);
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const f32x4 eg = lds16f(rows + Rec::kGrow + tile_row4(a, g) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) dr[a][i] *= -eg[i];
    }
    const float last = lds4f(rows + Rec::kGrow + (kC - 1) * 4);
#pragma unroll
    for (int a = 0; a < 2 * KK; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[a][i] *= last;
    constexpr int kRows = KK > 1 ? 4 : 2, kGroups = 2 * KK / kRows;
    auto get_t = [&](Exact (&x)[kRows], int kk, int grp2) {  // group grp2 / 2 of Q^T or K^T
      const lds_u8* const m = B + (grp2 & 1 ? Lds::kK : Lds::kQ);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int a = (grp2 >> 1) * kRows + r;
        x[r] = P::load_frag_t(m + (2 * kk * KK + (a >> 1)) * P::kFrag, m + ((2 * kk + 1) * KK + (a >> 1)) * P::kFrag, a, lane);
      }
    };
    Exact xt[2][kRows];
    get_t(xt[0], 0, 0);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      TermsT e, f;
      P::split(d[2 * kk], d[2 * kk + 1], e);
      P::split(dr[2 * kk], dr[2 * kk + 1], f);
      point(KK + 2 + kk);
#pragma unroll
      for (int i = 0; i < 2 * kGroups; ++i) {
        const int n4 = kk * 2 * kGroups + i;
        if (n4 + 1 < 4 * kGroups) get_t(xt[(n4 + 1) & 1], (n4 + 1) / (2 * kGroups), (n4 + 1) % (2 * kGroups));
        __builtin_amdgcn_sched_barrier(0);
        P::template mma_rows<NT>(xt[n4 & 1], i & 1 ? f : e, S + (i >> 1) * kRows);
      }
    }
    if constexpr (NBUF == 1) {
      if (more) {
        sync_lds();
        load_part(ch - 1, 0, 0, kPoints);
      }
    }
    if (more) {
      wait_vmem_all();
      sync_lds();
    }
  }
  float* before = nullptr;
  if constexpr (LOCAL) {
    before = p.local + bhs * (p.dv * p.dk);
  } else {
    store_late(c0);
    if (q.ds0 && seg == 0) before = q.ds0 + bh * (p.dv * p.dk);
  }
  if (before && live) store_state<KK>(before + col * p.dk, dk, p.vec_state, g, S);
}

// --- gradients -----------------------------------------------------------------------------------
// One workgroup of eight wavefronts per (batch, group, chunk): the heads of the group in turn, dQ
// and dK summed over them in registers (a fixed order, no atomics). Wavefronts w and w + 4 own
// steps [16w, 16w + 16) as columns: with x a row of a tile and y = 16w + c its column, the first
// makes the tiles E both ways round (x = s, y = t and x = t, y = s) and the second N; they hand
// each other the weighted tiles through LDS, and each makes half the rows of its columns of dQ^T
// and dK^T from them. The sums over v go in slices of 32 columns, brought into LDS one ahead. Images
// kept in fp32 (bf16 io, three terms) come in staged: S and dS into a strip of LDS, U and dR into
// registers, and each wavefront makes terms of its share once when the slice before has been read.
// That is 24 values a lane; terms made by every wavefront of what it reads would be a hundred, and
// terms kept in memory half as many bytes again to move.
//
// Bound by latency within the CU: the LDS (153 KB with keys of 128, three terms; 145 KB with two)
// leaves room for one workgroup on each. Batch 4, 8192 steps of 64 heads (16 of keys), 128 x 64 in
// bf16: 1.8-1.9 ms, with 16-bit operands 1.4 ms (5 % less if the same slice is read every time).
// The SIMDs spend 27 % of the time in matrix and 37 % in other vector instructions.
template <class P, int KK>
struct GradLds {
  typedef Image<P, KK> Img;
  static constexpr int kK = 0;
  static constexpr int kQ = 4 * KK * P::kFrag;
  static constexpr int kSlice = 2 * kQ;
  // a slice: the image (S, U), the second one (dS, dR), dY
  static constexpr int kFrag = P::template kImageFrag<P::kTerms>;
  static constexpr int kS = 0, kU = 2 * KK * kFrag, kImg = kU + 4 * kFrag;
  static constexpr int kDYBytes = 4 * P::kFrag;
  static constexpr int kSliceBytes = 2 * kImg + (P::kStaged ? 0 : kDYBytes);
  static constexpr int kTerms = kFrag;      // a right operand handed over
  // the tiles are handed over in the buffer of the slice before
  static constexpr int kHandBytes = 4 * 6 * kTerms;
  static constexpr int kBuffer = kSliceBytes > kHandBytes ? kSliceBytes : kHandBytes;
  // staged: the next slice's S and dS in fp32, its U and dR in registers, and two slots for dY
  static constexpr int kStage = P::kStaged ? 2 * 2 * KK * Img::kFrag : 0;
  static constexpr int kRest = 2 * 8 * kC * 4 + (6 * kC + 8) * 4;  // rows of two heads, sums
  static constexpr int kBufs = !P::kStaged && kSlice + 2 * kBuffer + kRest <= 160 * 1024 ? 2 : 1;
  static constexpr int kStageAt = kSlice + kBufs * kBuffer;
  static constexpr int kDYAt = kStageAt + kStage;
  static constexpr int kRows = kDYAt + (P::kStaged ? 2 * kDYBytes : 0);
  static constexpr int kSums = kRows + 2 * 8 * kC * 4;
  static constexpr int kBytes = kRows + kRest;
};

// sum over the four lane groups
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

template <class P, int KK>
__global__ void __launch_bounds__(512) delta_grad_kernel(const DeltaBwdParams q) {
  typedef typename P::IO IO;
  typedef typename P::Exact Exact;
  constexpr int NT = P::kTerms;
  typedef typename P::template Terms<NT> TermsT;
  typedef GradLds<P, KK> Lds;
  typedef Record<P, true> Rec;
  typedef Image<P, KK> Img;
  typedef Mover<P, KK, 8, 1> Move;
  constexpr int NBUF = Lds::kBufs;
  constexpr int kTiles = KK > 1 ? KK : 2;  // row tiles of dQ^T and dK^T to a wavefront
  const DeltaParams& p = q.f;
  __shared__ __attribute__((aligned(128))) uint8_t smem[Lds::kBytes];
  lds_u8* const sm = (lds_u8*)smem;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3, part = wave >> 2;
  const int a0 = part * kTiles;            // the first of its row tiles
  const bool has = a0 < 2 * KK;
  const uint32_t item = (uint32_t)die_item(blockIdx.x, gridDim.x), nch = (uint32_t)p.nchunks;
  const uint32_t bg = item / nch, ch = item - bg * nch;
  const uint32_t b = bg / (uint32_t)p.ngroups, grp = bg - b * (uint32_t)p.ngroups;
  const int rep = (int)p.rep;
  const int64_t L = p.L, t0 = (int64_t)ch * kC;
  const int n = (int)(L - t0 < kC ? L - t0 : kC);
  const int dk = (int)p.dk, cols = (int)p.v_cols;
  const int slices = (int)((p.dv + 31) / 32);
  const bool direct_y = cols % 32 == 0;

  // K and Q once
  {
    const IO* Kp = static_cast<const IO*>(p.k) + b * p.k_sb + grp * p.k_sg;
    const IO* Qp = static_cast<const IO*>(p.q) + b * p.q_sb + grp * p.q_sg;
    for (int f = wave; f < 8 * KK; f += 8) {
      const int mat = f / (4 * KK), fb = f % (4 * KK), a = fb / KK, kk = fb % KK;
      const int r = tile_row(a, c);
      const int64_t t = t0 + (r < n ? r : n - 1);
      const IO* row = mat ? Qp + t * p.q_st : Kp + t * p.k_st;
      P::store_frag(sm + f * P::kFrag, lane, P::load8(row + 32 * kk + 8 * g));
    }
  }
  // Slice sl of the r-th head of the group, with the first of a head the rows of its record: into
  // buffer `buf`; or, staged, to where the wavefront that will make terms of it finds its part, and dY
  // into slot `buf`.
  f32x4 raw_a, raw_b;  // a fragment of U (first wavefronts) or dR
  auto load_slice = [&](int r, int sl, int buf) {
    lds_u8* const to = sm + Lds::kSlice + buf * Lds::kBuffer;
    lds_u8* const dy_at = P::kStaged ? sm + Lds::kDYAt + buf * Lds::kDYBytes : to + 2 * Lds::kImg;
    const int64_t h = (int64_t)grp * rep + r, bhc = (b * p.nheads + h) * nch + ch;
    const int64_t at = (bhc * slices + sl) * Img::kBytes;
    if constexpr (P::kStaged) {
      if (wave < 2 * KK) {
        const int f = wave * Img::kFrag;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t unit = (uint32_t)(uintptr_t)(sm + Lds::kStageAt + 2 * f + half * 1024);
          dma16(p.image + at + Img::kS + f, half * 1024 + lane * 16, unit);
          dma16(q.image_b + at + Img::kS + f, half * 1024 + lane * 16, unit + Img::kFrag);
        }
      }
    } else {
      Move::template run<Img::kBytes / 1024>(wave, lane, p.image + at, to);
      Move::template run<Img::kBytes / 1024>(wave, lane, q.image_b + at, to + Lds::kImg);
    }
    if (sl == 0)
      Move::template run<2>(wave, lane, p.rec + bhc * (int64_t)Rec::kBytes + Rec::kRows,
                            sm + Lds::kRows + (r & 1) * 2048);
    if (wave < 4) {
      const int x = tile_row(w, c);
      const IO* row = static_cast<const IO*>(q.dy) + b * p.y_sb + h * p.y_sh + (t0 + (x < n ? x : n - 1)) * p.y_st;
      lds_u8* const f = dy_at + w * P::kFrag;
      if (direct_y) {
#pragma unroll
        for (int half = 0; half < P::kFrag / 1024; ++half)
          dma16(row + sl * 32 + 8 * g + 4 * half, (uint32_t)(uintptr_t)(f + half * 1024));
      } else {
        P::store_frag(f, lane, sl * 32 + 8 * g < cols ? P::load8(row + sl * 32 + 8 * g) : Exact{});
      }
    }
    if constexpr (P::kStaged) {
      const uint8_t* f = (part ? q.image_b : p.image) + at + Img::kU + w * Img::kFrag + lane * 16;
      raw_a = *reinterpret_cast<const f32x4*>(f);
      raw_b = *reinterpret_cast<const f32x4*>(f + 1024);
    }
  };
  // staged: the wavefront's fragments as terms into the buffer; returns its share of <S, dS>
  auto make_terms = [&]() {
    float dot = 0.0f;
    if constexpr (P::kStaged) {
      lds_u8* const to = sm + Lds::kSlice;
      if (wave < 2 * KK) {
        const lds_u8* const from = sm + Lds::kStageAt + 2 * wave * Img::kFrag + lane * 16;
        const f32x4 sa = lds16f(from), sb = lds16f(from + 1024);
        const f32x4 da = lds16f(from + Img::kFrag), db = lds16f(from + Img::kFrag + 1024);
#pragma unroll
        for (int i = 0; i < 4; ++i) dot = fmaf(sa[i], da[i], fmaf(sb[i], db[i], dot));
        P::template put_image<NT>(to + Lds::kS + wave * Lds::kFrag, lane, sa, sb);
        P::template put_image<NT>(to + Lds::kImg + Lds::kS + wave * Lds::kFrag, lane, da, db);
      }
      P::template put_image<NT>(to + part * Lds::kImg + Lds::kU + w * Lds::kFrag, lane, raw_a, raw_b);
    }
    return dot;
  };
  // lane (g, c)'s fragment of row y = 16w + c
  const int a_y = row_tile(16 * w + c), l_y = g * 16 + row_slot(16 * w + c);
  const int y = 16 * w + c;
  const int64_t ty = t0 + (y < n ? y : n - 1);
  auto frag_y = [&](int mat, int kk) { return P::load_frag(sm + mat + (a_y * KK + kk) * P::kFrag, l_y); };
  auto sums = [&](int i) { return reinterpret_cast<__attribute__((address_space(3))) float*>(sm + Lds::kSums + 4 * i); };

  f32x4 dq[kTiles], dkk[kTiles];
#pragma unroll
  for (int a = 0; a < kTiles; ++a) dq[a] = dkk[a] = f32x4{0, 0, 0, 0};

  int buf = 0;
  load_slice(0, 0, 0);
  for (int r = 0; r < rep; ++r) {
    const int64_t h = (int64_t)grp * rep + r;
    const IO* vrow = static_cast<const IO*>(p.v) + b * p.v_sb + h * p.v_sh + ty * p.v_st;

    // E (first wavefronts) or N (second): rows s, and rows t
    f32x4 m1[4], m2[4];
    f32x4 sy[kTiles], sr[kTiles], su[kTiles];      // S dY, S dR, dS U
#pragma unroll
    for (int a = 0; a < 4; ++a) m1[a] = m2[a] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int a = 0; a < kTiles; ++a) sy[a] = sr[a] = su[a] = f32x4{0, 0, 0, 0};
    float rv = 0.0f, ss = 0.0f;  // dR . V; this wavefront's share of <S, dS>
    for (int sl = 0; sl < slices; ++sl) {
      wait_vmem_all();
      sync_lds();
      if constexpr (P::kStaged) {
        ss += make_terms();
        sync_lds();
      }
      const lds_u8* const B = sm + Lds::kSlice + (NBUF == 2 ? buf : 0) * Lds::kBuffer;
      const lds_u8* const iY = P::kStaged ? sm + Lds::kDYAt + buf * Lds::kDYBytes : B + 2 * Lds::kImg;
      Exact vv = {};
      if (part == 0 && sl * 32 + 8 * g < cols) vv = P::load8(vrow + sl * 32 + 8 * g);
      if constexpr (NBUF == 2 || P::kStaged) {
        if (sl + 1 < slices) load_slice(r, sl + 1, buf ^ 1);
        else if (r + 1 < rep) load_slice(r + 1, 0, buf ^ 1);
      }

      const lds_u8 *const iS = B + Lds::kS, *const iU = B + Lds::kU;
      const lds_u8 *const iD = B + Lds::kImg + Lds::kS, *const iR = B + Lds::kImg + Lds::kU;
      const Exact yb = P::load_frag(iY + a_y * P::kFrag, l_y);
      TermsT ub, rb;
      P::load_image_block(iU, 2, w, lane, ub);
      P::load_image_block(iR, 2, w, lane, rb);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        if ((a >> 1) <= (w >> 1)) {
          TermsT ua;
          P::load_image_tile(iU, 2, a, lane, ua);
          if (part == 0) m1[a] = P::mma_te(ua, yb, m1[a]);
          else m1[a] = P::mma_tt(ua, rb, m1[a]);
        }
        if ((a >> 1) >= (w >> 1)) {
          if (part == 0) {
            m2[a] = P::template mma<NT>(P::load_frag(iY + a * P::kFrag, lane), ub, m2[a]);
          } else {
            TermsT ra;
            P::load_image_tile(iR, 2, a, lane, ra);
            m2[a] = P::mma_tt(ra, ub, m2[a]);
          }
        }
      }
      if (has) {
#pragma unroll
        for (int a = 0; a < kTiles; ++a) {
          TermsT s, d;
          P::load_image_tile(iS, KK, a0 + a, lane, s);
          P::load_image_tile(iD, KK, a0 + a, lane, d);
          sy[a] = P::mma_te(s, yb, sy[a]);
          sr[a] = P::mma_tt(s, rb, sr[a]);
          su[a] = P::mma_tt(d, ub, su[a]);
        }
      }
      float x[8], z[8];
      if (part == 0) {
        P::floats(rb, x);
        P::floats(vv, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) rv = fmaf(x[e], z[e], rv);
      }
      if constexpr (!P::kStaged) {
        for (int f = wave; f < 2 * KK; f += 8) {
          P::image_floats(iS + f * Lds::kFrag, lane, x);
          P::image_floats(iD + f * Lds::kFrag, lane, z);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], z[e], ss);
        }
      }
      if constexpr (NBUF == 1 && !P::kStaged) {
        if (sl + 1 < slices) {
          sync_lds();
          load_slice(r, sl + 1, 0);
        }
      } else {
        buf ^= 1;
      }
    }
    // the tiles' weights, and the sums over their rows
    const lds_u8* const rows = sm + Lds::kRows + (r & 1) * 2048;
    const float gy = lds4f(rows + Rec::kGhi + 4 * y), ly = lds4f(rows + Rec::kGlo + 4 * y);
    const float by = lds4f(rows + Rec::kBeta + 4 * y);
    float dG = 0.0f, dbe = 0.0f;
    // y and n less the lane's first x, hidden from the optimiser: the comparisons below, taken out of the loop over the
    // heads as lane masks, do not fit the scalar registers
    int yx = y - tile_row4(0, g), nx = n - tile_row4(0, g);
    asm volatile("" : "+v"(yx), "+v"(nx));
    const int on = y < n ? yx : -1;  // no x is up to a step past the last
    // the last slice's buffer, when all have read it
    lds_u8* const hand = sm + Lds::kSlice + (NBUF == 2 ? buf ^ 1 : 0) * Lds::kBuffer + w * 6 * Lds::kTerms;
    sync_lds();
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      f32x4 d;  // e^{G_later - G_earlier}
      {
        const f32x4 gx = lds16f(rows + Rec::kGhi + tile_row4(a, g) * 4), lx = lds16f(rows + Rec::kGlo + tile_row4(a, g) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float diff = (gx[i] - gy) + (lx[i] - ly);
          d[i] = __builtin_amdgcn_exp2f(tile_row4(a, 0) + i > yx ? diff : -diff);
        }
      }
      f32x4 k4 = {0, 0, 0, 0}, q4 = {0, 0, 0, 0};
      if (part == 0) {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          if ((a >> 1) <= (w >> 1)) k4 = P::mma(P::load_frag(sm + Lds::kK + (a * KK + kk) * P::kFrag, lane), frag_y(Lds::kQ, kk), k4);
          if ((a >> 1) >= (w >> 1)) q4 = P::mma(P::load_frag(sm + Lds::kQ + (a * KK + kk) * P::kFrag, lane), frag_y(Lds::kK, kk), q4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = tile_row4(a, 0) + i;
          const float w1 = x <= on ? p.scale * d[i] * m1[a][i] : 0.0f;
          const float w2 = x >= yx && x < nx ? p.scale * d[i] * m2[a][i] : 0.0f;
          // step y itself is in the rows' sum and the columns': neither, else the two products' roundings,
          // which no decay makes small, stay in dG
          dG += x == yx ? 0.0f : w1 * k4[i] - w2 * q4[i];
          m1[a][i] = w1;
          m2[a][i] = w2;
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
          k4 = P::mma(P::load_frag(sm + Lds::kK + (a * KK + kk) * P::kFrag, lane), frag_y(Lds::kK, kk), k4);
        const f32x4 bx = lds16f(rows + Rec::kBeta + tile_row4(a, g) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = tile_row4(a, 0) + i;
          const float n1 = x < on ? -d[i] * m1[a][i] : 0.0f;
          const float n2 = x > yx && x < nx ? -d[i] * bx[i] * m2[a][i] : 0.0f;
          dbe = fmaf(n1, k4[i], dbe);
          dG += (by * n1 - n2) * k4[i];
          m1[a][i] = by * n1 + n2;
        }
      }
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      TermsT x;
      P::split(m1[2 * kk], m1[2 * kk + 1], x);
      P::store_terms(hand + ((part ? 4 : 0) + kk) * Lds::kTerms, lane, x);
      if (part == 0) {
        P::split(m2[2 * kk], m2[2 * kk + 1], x);
        P::store_terms(hand + (2 + kk) * Lds::kTerms, lane, x);
      }
    }
    // what the states give
    float qs = 0.0f, kr = 0.0f, ku = 0.0f;
    if (has) {
      const float egy = lds4f(rows + Rec::kGrow + 4 * y), decy = lds4f(rows + Rec::kDecay + 4 * y);
#pragma unroll
      for (int k = 0; k < kTiles / 2; ++k) {
        float kf[8], qf[8];
        P::floats(frag_y(Lds::kK, a0 / 2 + k), kf);
        P::floats(frag_y(Lds::kQ, a0 / 2 + k), qf);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int a = 2 * k + (e >> 2), i = e & 3;
          const float vy = p.scale * egy * sy[a][i], vr = -egy * sr[a][i], vu = decy * su[a][i];
          qs = fmaf(qf[e], vy, qs);
          kr = fmaf(kf[e], vr, kr);
          ku = fmaf(kf[e], vu, ku);
          dq[a][i] += vy;
          dkk[a][i] += fmaf(by, vr, vu);
        }
      }
    }
    dbe = sum_groups(dbe + kr + rv);
    ku = y < n - 1 ? ku : 0.0f;  // the last step's, without decay, is taken away and added again
    dG = sum_groups(dG + qs + by * kr - ku);
    ku = sum_groups(ku);
    ss = sum_groups(ss);
#pragma unroll
    for (int s = 1; s < 16; s <<= 1) ss += __shfl_xor(ss, s);
    if (g == 0) {
      *sums(part * kC + y) = dG;
      *sums((2 + part) * kC + y) = dbe;
      *sums((4 + part) * kC + y) = ku;
    }
    if (lane == 0) *sums(6 * kC + wave) = ss;
    sync_lds();
    if (has) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        TermsT x1, x2, x3;
        P::load_terms(hand + kk * Lds::kTerms, lane, x1);
        P::load_terms(hand + (2 + kk) * Lds::kTerms, lane, x2);
        P::load_terms(hand + (4 + kk) * Lds::kTerms, lane, x3);
#pragma unroll
        for (int j = 0; j < kTiles; j += 2) {
          Exact kt[2], qt[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int a = a0 + j + i;
            const int f0 = (2 * kk * KK + (a >> 1)) * P::kFrag, f1 = ((2 * kk + 1) * KK + (a >> 1)) * P::kFrag;
            kt[i] = P::load_frag_t(sm + Lds::kK + f0, sm + Lds::kK + f1, a, lane);
            qt[i] = P::load_frag_t(sm + Lds::kQ + f0, sm + Lds::kQ + f1, a, lane);
          }
          P::template mma_rows<NT>(kt, x1, dq + j);
          P::template mma_rows<NT>(kt, x3, dkk + j);
          P::template mma_rows<NT>(qt, x2, dkk + j);
        }
      }
    }
    if (wave == 7) {  // dg: sums over the steps from each on
      const int64_t out = (b * L + t0) * p.nheads + h;
      float x = *sums(lane) + *sums(kC + lane), k = *sums(4 * kC + lane) + *sums(5 * kC + lane);
      x = lane < n ? x : 0.0f;
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) k += __shfl_xor(k, s);
      float whole = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) whole += *sums(6 * kC + i);
      // G_63 is the sum up to the last step there is
      if (lane == n - 1) x += fmaf(lds4f(rows + Rec::kGrow + 4 * (kC - 1)), whole, k);
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) {
        const float o = __shfl_down(x, s);
        if (lane + s < 64) x += o;
      }
      if (lane < n) {
        store_elem(static_cast<IO*>(q.dg) + out + lane * p.nheads, x);
        store_elem(static_cast<IO*>(q.dbeta) + out + lane * p.nheads, *sums(2 * kC + lane) + *sums(3 * kC + lane));
      }
    }
    if constexpr (NBUF == 1 && !P::kStaged) {
      if (r + 1 < rep) {
        sync_lds();  // the handed tiles have been read
        load_slice(r + 1, 0, 0);
      }
    }
  }
  if (y < n && has) {
    const int64_t at = ((b * L + ty) * p.ngroups + grp) * p.dk;
    IO* const oq = static_cast<IO*>(q.dq) + at;
    IO* const ok = static_cast<IO*>(q.dk) + at;
#pragma unroll
    for (int k = 0; k < kTiles / 2; ++k) {
      const int d = 32 * (a0 / 2 + k) + 8 * g;
      if (q.vec_out) {
        if (d < dk) {
          P::store8(oq + d, dq[2 * k], dq[2 * k + 1]);
          P::store8(ok + d, dkk[2 * k], dkk[2 * k + 1]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (d + e < dk) {
            store_elem(oq + d + e, dq[2 * k + (e >> 2)][e & 3]);
            store_elem(ok + d + e, dkk[2 * k + (e >> 2)][e & 3]);
          }
      }
    }
  }
}

template <class P, int KK, int NW, bool LOCAL>
hipError_t back_go(const DeltaBwdParams& q, hipStream_t stream) {
  const int64_t slices = (q.f.dv + 16 * NW - 1) / (16 * NW), items = q.f.batch * q.f.nheads * (q.f.nseg - LOCAL) * slices;
  delta_back_kernel<P, KK, NW, LOCAL><<<dim3((unsigned)items), dim3(64 * NW), 0, stream>>>(q);
  return hipGetLastError();
}

template <class P, int KK, bool LOCAL>
hipError_t back(const DeltaBwdParams& q, hipStream_t stream) {
  // fp32 with long keys: eight wavefronts have not the registers (8192 steps of 32 heads of 128 x
  // 128: 422 us, 401 in workgroups of four)
  if constexpr (LOCAL && !P::kBf16 && KK == 4) return back_go<P, KK, 4, LOCAL>(q, stream);
  else return delta_scan_waves(q.f) == 8 ? back_go<P, KK, 8, LOCAL>(q, stream) : back_go<P, KK, 4, LOCAL>(q, stream);
}

template <class P, int KK>
hipError_t bwd(const DeltaBwdParams& q, hipStream_t stream) {
  hipError_t e;
  if (q.f.nseg > 1) {
    e = back<P, KK, true>(q, stream);
    if (e != hipSuccess) return e;
    e = launch_delta_combine_back(q, stream);
    if (e != hipSuccess) return e;
  }
  e = back<P, KK, false>(q, stream);
  if (e != hipSuccess) return e;
  delta_grad_kernel<P, KK><<<dim3((unsigned)(q.f.batch * q.f.ngroups * q.f.nchunks)), 512, 0, stream>>>(q);
  return hipGetLastError();
}

template <class P>
hipError_t bwd_key(const DeltaBwdParams& q, hipStream_t stream) {
  switch (delta_pad_key(q.f.dk)) {
    case 32: return bwd<P, 1>(q, stream);
    case 64: return bwd<P, 2>(q, stream);
    default: return bwd<P, 4>(q, stream);
  }
}

}  // namespace

hipError_t launch_delta_bwd(const DeltaBwdParams& q, hipStream_t stream) {
  const hipError_t e = launch_delta_states(q.f, stream);
  if (e != hipSuccess) return e;
  if (!q.f.bf16) return bwd_key<F32>(q, stream);
  return q.f.terms == 3 ? bwd_key<Bf16<3>>(q, stream) : bwd_key<Bf16<2>>(q, stream);
}

}  // namespace ssm
