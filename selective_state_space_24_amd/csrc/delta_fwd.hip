// gfx950 kernels of the chunked gated delta rule, forward pass (see delta_common.h for the
// formulas and the tile layouts): the prep kernel makes T and P of every chunk, the scan kernel
// runs over the chunks in order.
#include "delta_common.h"

namespace ssm {

using namespace delta;

namespace {

// --- prep ---------------------------------------------------------------------------------------
// One workgroup of four wavefronts per (batch, head, chunk). Wavefront w makes rows [16w, 16w+16)
// of A and P by MFMA, from the rows of K and Q read straight in fragment order (no LDS; the four
// read the same K rows, out of L1), inverts its diagonal block of I + A by substitution, one
// column a lane, and then makes the blocks T_wj left of it, j = w - 1 .. 0, by fp32 MFMA:
//   T_wj^T = -T_jj^T sum_{j < k <= w} A_kj^T T_wk^T
// transposed, so that each result is the right operand of the next product as it stands.
// Substitution and fp32 blocks: a product form of the inverse in powers of A loses digits where
// keys repeat. G is summed in fp64: e^{G_t - G_s} of two large sums keeps its digits.
//
// Near the memory's rate: 212 us for 16384 chunks with keys of 128 in bf16, which write 0.62 GB of
// records and read 0.27 GB (4.2 TB/s; a large copy 4.8). The SIMDs spend 12 % of the time in matrix and
// 38 % in other vector instructions, wavefronts 58 % of theirs waiting for memory or each other.
constexpr int kAtStride = kC + 4;  // floats per row of A^T in LDS

// inclusive prefix sum over the 64 lanes, in fp64, by DPP moves (see wave_inclusive_sum's steps in
// the scalar-decay chunked form: shifts within rows of 16 lanes, then the rows' last lanes)
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_or_zero(double v) {
  const uint64_t x = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)x, CTRL, ROW_MASK, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(x >> 32), CTRL, ROW_MASK, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double prefix_sum(double v) {
  v += dpp_or_zero<0x111, 0xf>(v);
  v += dpp_or_zero<0x112, 0xf>(v);
  v += dpp_or_zero<0x114, 0xf>(v);
  v += dpp_or_zero<0x118, 0xf>(v);
  v += dpp_or_zero<0x142, 0xa>(v);
  v += dpp_or_zero<0x143, 0xc>(v);
  return v;
}

template <class P, int KK, bool BWD>
__global__ void __launch_bounds__(256) delta_prep_kernel(const DeltaParams p) {
  typedef typename P::IO IO;
  typedef Record<P, BWD> Rec;
  __shared__ __attribute__((aligned(16))) float at_s[kC * kAtStride];
  __shared__ __attribute__((aligned(16))) float tt_s[4 * 16 * 16];
  __shared__ __attribute__((aligned(16))) float row_s[3 * kC];  // G as two floats, beta
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the grid is (chunk, batch x head): with a multiple of eight chunks, those of a group's heads
  // that read the same rows of K and Q are on one accelerator die
  const uint32_t chunk = blockIdx.x, bh = blockIdx.y + 65535u * blockIdx.z;
  if (bh >= (uint32_t)(p.batch * p.nheads)) return;
  const uint32_t b = bh / (uint32_t)p.nheads, h = bh - b * (uint32_t)p.nheads;
  const uint32_t grp = h / (uint32_t)p.rep;
  const int64_t t0 = (int64_t)chunk * kC;
  const int n = (int)(p.L - t0 < kC ? p.L - t0 : kC);  // steps of this chunk
  uint8_t* rec = p.rec + (bh * p.nchunks + chunk) * (int64_t)Rec::kBytes;

  // G: every wavefront sums for itself (lane = step); below 2^-160 a decay is 0 in fp32
  double G = 0.0;
  float be = 0.0f;
  if (lane < n) {
    const float gl = to_f32(static_cast<const IO*>(p.g)[b * p.g_sb + (t0 + lane) * p.g_st + h * p.g_sh]) * kLog2e;
    G = (double)(gl < -160.0f ? -160.0f : gl);
    be = to_f32(static_cast<const IO*>(p.beta)[b * p.be_sb + (t0 + lane) * p.be_st + h * p.be_sh]);
  }

  // rows past the end of the sequence read its last one; what they give is not used
  const IO* Kp = static_cast<const IO*>(p.k) + b * p.k_sb + grp * p.k_sg + t0 * p.k_st;
  const IO* Qp = static_cast<const IO*>(p.q) + b * p.q_sb + grp * p.q_sg + t0 * p.q_st;
  auto load = [&](const IO* base, int64_t st, int blk, typename P::Exact (&f)[KK]) {
    const int t = min(16 * blk + c, n - 1);
    const uint8_t* at = reinterpret_cast<const uint8_t*>(base) + (uint32_t)((t * (int)st + 8 * g) * (int)sizeof(IO));
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) f[kk] = P::load8(reinterpret_cast<const IO*>(at) + 32 * kk);
  };
  typename P::Exact kw[KK], qw[KK];
  load(Kp, p.k_st, w, kw);
  load(Qp, p.q_st, w, qw);

  G = prefix_sum(G);
  const float ghi = (float)G, glo = (float)(G - (double)ghi);
  lds_u8* const row = (lds_u8*)row_s;
  if (w == 0) {
    const double end = __builtin_bit_cast(double, (uint64_t)__builtin_amdgcn_readlane((int)(__builtin_bit_cast(uint64_t, G) >> 32), 63) << 32 |
                                          (uint32_t)__builtin_amdgcn_readlane((int)__builtin_bit_cast(uint64_t, G), 63));
    row_s[lane] = ghi;
    row_s[kC + lane] = glo;
    row_s[2 * kC + lane] = be;
    float* rows = reinterpret_cast<float*>(rec + Rec::kRows);
    rows[lane] = __builtin_amdgcn_exp2f(ghi);
    rows[kC + lane] = __builtin_amdgcn_exp2f((float)(end - G));
    rows[2 * kC + lane] = be;
    rows[3 * kC + lane] = lane < n ? 1.0f : 0.0f;
    if constexpr (BWD) {
      rows[4 * kC + lane] = ghi;
      rows[5 * kC + lane] = glo;
    }
  }
  __syncthreads();

  // A^T and P^T: rows s = 16 blk + 4g + i, column t = 16w + c
  lds_u8* const at = (lds_u8*)at_s;
  const int t = 16 * w + c;
  const float gt = lds4f(row + t * 4), lt = lds4f(row + (kC + t) * 4);
  // 0 past the last step: T is the identity there and P zero
  const float bt = lds4f(row + (2 * kC + t) * 4), st = t < n ? p.scale : 0.0f;
  f32x4 pt[4];
#pragma unroll
  for (int blk = 0; blk < 4; ++blk) {
    pt[blk] = f32x4{0, 0, 0, 0};
    if (blk > w) continue;
    f32x4 a4 = {0, 0, 0, 0};
    typename P::Exact kb[KK];
    if (blk < w) load(Kp, p.k_st, blk, kb);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      const typename P::Exact k1 = blk == w ? kw[kk] : kb[kk];
      a4 = P::mma(k1, kw[kk], a4);
      pt[blk] = P::mma(k1, qw[kk], pt[blk]);
    }
    const f32x4 gs = lds16f(row + (16 * blk + 4 * g) * 4), ls = lds16f(row + (kC + 16 * blk + 4 * g) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = 16 * blk + 4 * g + i;
      const float d = __builtin_amdgcn_exp2f((gt - gs[i]) + (lt - ls[i]));
      const float a = s < t ? a4[i] * (bt * d) : 0.0f;
      *reinterpret_cast<__attribute__((address_space(3))) float*>(at + (s * kAtStride + t) * 4) = a;
      pt[blk][i] = s <= t ? pt[blk][i] * (st * d) : 0.0f;
    }
  }
  // where lane (g, c)'s four entries [t = 16w + c][16 j + 4g .. +4) go in fragment order
  const int a_t = row_tile(t), m_t = row_slot(t);
  auto put = [&](int off, int bytes, int j, const f32x4 v) {
    uint8_t* f = rec + (off + tri_block(a_t, j >> 1) * bytes);
    const int gs = 2 * (j & 1) + (g >> 1);
    P::template put4<P::kTerms>(f, gs, m_t, g & 1, v);
  };
  const int jmax = w | 1;  // a fragment covers two blocks of columns
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j <= jmax) put(Rec::kP, Rec::kPBlock, j, pt[j]);
  sync_lds();

  // T_ww: lane c solves for column c (the four lane groups alike)
  lds_u8* const tt = (lds_u8*)tt_s;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.0f : 0.0f;
#pragma unroll
  for (int k = 0; k < 15; ++k) {
#pragma unroll
    for (int i4 = (k + 1) & ~3; i4 < 16; i4 += 4) {
      const f32x4 a4 = lds16f(at + ((16 * w + k) * kAtStride + 16 * w + i4) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i4 + i > k) x[i4 + i] = fmaf(-a4[i], x[k], x[i4 + i]);
    }
  }
  // T_ww^T by rows: lane (g, c) writes columns 4g .. 4g + 3 of row c
  f32x4 mine;
#pragma unroll
  for (int i = 0; i < 4; ++i) mine[i] = g == 0 ? x[i] : (g == 1 ? x[4 + i] : (g == 2 ? x[8 + i] : x[12 + i]));
  sts16f(tt + ((w * 16 + c) * 16 + 4 * g) * 4, mine);
  sync_lds();

  f32x4 tw[4];  // T_wj^T: rows s = 16j + 4g + i, column t = 16w + c
#pragma unroll
  for (int j = 3; j >= 0; --j) {
    tw[j] = f32x4{0, 0, 0, 0};
    if (j == w) {
#pragma unroll
      for (int i = 0; i < 4; ++i) tw[j][i] = lds4f(tt + ((w * 16 + 4 * g + i) * 16 + c) * 4);
    } else if (j < w) {
      f32x4 z = {0, 0, 0, 0};
#pragma unroll
      for (int k = 3; k > 0; --k) {
        if (k <= j || k > w) continue;
        const f32x4 a4 = lds16f(at + ((16 * j + c) * kAtStride + 16 * k + 4 * g) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) z = __builtin_amdgcn_mfma_f32_16x16x4f32(a4[i], tw[k][i], z, 0, 0, 0);
      }
      const f32x4 tj = lds16f(tt + ((j * 16 + c) * 16 + 4 * g) * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) tw[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(-tj[i], z[i], tw[j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j <= jmax) put(Rec::kT, Rec::kTBlock, j, tw[j]);
}

// --- scan -----------------------------------------------------------------------------------------
// One workgroup = one (batch, head) x 16 NW columns of v; wavefront w owns columns [16w, 16w+16)
// of them and needs nothing from the others but the shared left operands, which the workgroup
// brings into LDS one chunk ahead (NBUF 2; where there is room for one buffer only, it waits for
// its loads). Everything goes there by direct loads, v too, which is then read by columns; y leaves
// four columns at a time one chunk late, so that nothing waits for it. v is read at the start of a
// chunk: where two buffers have room for one tile of v only, the next chunk's is loaded behind a
// barrier in the middle of the chunk.
//
// Bound by the wavefronts' own matrix and vector instructions (54 and 40 % of the SIMDs' time), which
// overlap little at the two wavefronts a SIMD that the registers allow: batch 8, 4096 steps of 32
// heads, 128 x 128 in bf16 takes 440 us; with 16-bit operands 310, and 9 % less if every chunk reads
// the same memory.
//
// kStates, the backward pass's first scan: no y; the state before each chunk and U go to the image.
//
// A sequence with too few columns for the chip is split along L. Over a segment the state is an
// affine function of where it starts, S_end = M S_start + S_local, column by column: kSummary runs
// the segments at once without y, on the columns of v from zeros (S_local) and, with v = 0, on the
// dk columns of the identity (M). The combine kernel passes the state from segment to segment, and
// the scan then runs every segment from its own start. The columns are visited three times
// (dk = dv): see delta_plan for where that pays. The backward pass reads its own records and needs
// M of every segment, the last one too: kSummaryBwd.
enum Mode { kY, kStates, kSummary, kSummaryBwd };
constexpr bool is_summary(Mode m) { return m == kSummary || m == kSummaryBwd; }
constexpr bool is_bwd(Mode m) { return m == kStates || m == kSummaryBwd; }

// M of a segment: columns in tiles of 16, fragments of 32 rows, three terms.
template <class P, int KK>
struct Trans {
  static constexpr int kFrag = P::template kImageFrag<3>;
  static constexpr int kBytes = 2 * KK * KK * kFrag;
};

template <class P, int KK, int NW, Mode MODE>
struct ScanLds {
  typedef Record<P, is_bwd(MODE)> Rec;
  typedef Mover<P, KK, NW, MODE == kY ? 2 : 1> Move;
  static constexpr int kK = 0;
  static constexpr int kQ = 4 * KK * P::kFrag;
  static constexpr int kRec = MODE == kY ? 2 * kQ : kQ;
  // the part of the record that is not copied (P, without y) is left out
  static constexpr int kSkip = MODE == kY ? 0 : Rec::kRows - Rec::kP;
  static constexpr int kRows = kRec + Rec::kRows - kSkip;
  static constexpr int kBytes = kRec + Rec::kBytes - kSkip;
  static constexpr Buffers kBuf = buffers(kBytes, Move::kTileBytes);
  static constexpr int kAll = kBuf.n * kBytes + kBuf.tiles * Move::kTileBytes;
};

template <class P, int KK, int NW, Mode MODE>
__global__ void __launch_bounds__(64 * NW) delta_scan_kernel(const DeltaParams p) {
  typedef typename P::IO IO;
  typedef ScanLds<P, KK, NW, MODE> Lds;
  typedef typename Lds::Rec Rec;
  constexpr int NT = P::kTerms;
  constexpr bool STATES = MODE == kStates;
  constexpr bool SUMMARY = is_summary(MODE);
  constexpr bool Y = MODE == kY;
  constexpr int NBUF = Lds::kBuf.n, VBUF = Lds::kBuf.tiles;
  __shared__ __attribute__((aligned(16))) uint8_t smem[Lds::kAll];
  lds_u8* const sm = (lds_u8*)smem;
  auto tile_at = [&](int buf) { return sm + NBUF * Lds::kBytes + (VBUF == 2 ? buf : 0) * Lds::Move::kTileBytes; };
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // 32-bit arithmetic: there are fewer than 2^31 items
  const uint32_t vslices = (uint32_t)((p.dv + 16 * NW - 1) / (16 * NW));
  const uint32_t slices = SUMMARY ? vslices + (32 * KK + 16 * NW - 1) / (16 * NW) : vslices;
  const uint32_t item = (uint32_t)die_item(blockIdx.x, gridDim.x);
  const uint32_t bhs = item / slices, segs = MODE == kSummary ? (uint32_t)p.nseg - 1 : (uint32_t)p.nseg;
  const int64_t bh = bhs / segs;
  const uint32_t seg = bhs - (uint32_t)bh * segs;
  const uint32_t b = (uint32_t)bh / (uint32_t)p.nheads, h = (uint32_t)bh - b * (uint32_t)p.nheads;
  const uint32_t grp = h / (uint32_t)p.rep;
  const uint32_t slice = item - bhs * slices;
  const bool unit = SUMMARY && slice >= vslices;  // columns of the identity
  const int64_t slice0 = (int64_t)(unit ? slice - vslices : slice) * (16 * NW);
  const int64_t col = slice0 + 16 * w + c;
  const bool live = !unit && col < p.dv;
  const int dk = (int)p.dk;
  const int64_t L = p.L, nch = p.nchunks;
  const int64_t c0 = seg * p.seg_chunks, c1 = c0 + p.seg_chunks < nch ? c0 + p.seg_chunks : nch;
  const IO* Kp = static_cast<const IO*>(p.k) + b * p.k_sb + grp * p.k_sg;
  const IO* Qp = static_cast<const IO*>(p.q) + b * p.q_sb + grp * p.q_sg;
  const IO* Vp = static_cast<const IO*>(p.v) + b * p.v_sb + h * p.v_sh;
  IO* Yp = Y ? static_cast<IO*>(p.y) + b * p.y_sb + h * p.y_sh : nullptr;
  const uint8_t* rec = p.rec + bh * nch * (int64_t)Rec::kBytes;
  // this wavefront's tile of the image (null past its last)
  const int64_t tile = (slice0 >> 4) + w, img_slices = (p.dv + 31) / 32;
  const int64_t img_chunk = img_slices * Image<P, KK>::kBytes;
  uint8_t* const image = STATES && tile < 2 * img_slices
                             ? p.image + bh * nch * img_chunk + (tile >> 1) * Image<P, KK>::kBytes : nullptr;
  const int img_s = (int)(tile & 1) * KK * Image<P, KK>::kFrag, img_u = (int)(tile & 1) * 2 * Image<P, KK>::kFrag;

  typename Lds::Move mv;
  auto place = [&](int rows) {
    const int64_t st[2] = {p.k_st, p.q_st};
    mv.place(w, lane, rows, st, p.v_st, unit ? 16 * NW : p.v_cols - slice0);
  };
  // The loads of a chunk, in kPoints parts: part n's direct loads are issued at point n of the
  // chunk before. All at once they would queue up ahead of the wavefronts' first LDS reads.
  constexpr int kPoints = KK + 4;
  constexpr int kRec1 = Y ? Rec::kBytes / 1024 : Rec::kP / 1024, kRec2 = Y ? 0 : Rec::kRowBytes / 1024;
  constexpr int kFragN = Lds::Move::kFragSteps, kTileN = VBUF == NBUF ? Lds::Move::kTileSteps : 0;
  constexpr int kRec1N = (kRec1 + NW - 1) / NW, kRec2N = (kRec2 + NW - 1) / NW;
  constexpr int kSteps = kFragN + kTileN + kRec1N + kRec2N;
  auto load_tile = [&](int64_t ch, int i, lds_u8* to) {
    if (!unit) mv.row_step(i, w, Vp + ch * kC * p.v_st + slice0, to);
  };
  auto load_part = [&](int64_t ch, int buf, int first, int last) {
    lds_u8* const to = sm + buf * Lds::kBytes;
    const int64_t t0 = ch * kC;
    const uint8_t* rc = rec + ch * (int64_t)Rec::kBytes;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s < first * kSteps / kPoints || s >= last * kSteps / kPoints) continue;
      if (s < kFragN) mv.frag_step(s, w, Kp + t0 * p.k_st, Qp + t0 * p.q_st, to + Lds::kK);
      else if (s < kFragN + kTileN)
        load_tile(ch, s - kFragN, tile_at(buf));
      else if (s < kFragN + kTileN + kRec1N)
        Lds::Move::template run_step<kRec1>(s - kFragN - kTileN, w, lane, rc, to + Lds::kRec);
      else
        Lds::Move::template run_step<kRec2>(s - kFragN - kTileN - kRec1N, w, lane, rc + Rec::kRows, to + Lds::kRows);
    }
  };
  // the tile of v, where it is not among the parts
  auto load_late_tile = [&](int64_t ch) {
    if constexpr (VBUF != NBUF) {
#pragma unroll
      for (int i = 0; i < Lds::Move::kTileSteps; ++i) load_tile(ch, i, tile_at(0));
    }
  };
  // before the parts of a last, shorter chunk
  auto load_first = [&](int64_t ch) {
    if (L - ch * kC < kC) place((int)(L - ch * kC));
  };

  // S in accumulator layout: tile a, register i = S[tile_row4(a, g) + i][col]
  const float* start = SUMMARY ? nullptr : p.s0 ? p.s0 + bh * p.dv * p.dk : nullptr;
  if (!SUMMARY && seg > 0) start = p.starts + bhs * (p.dv * p.dk);
  f32x4 S[2 * KK];
#pragma unroll
  for (int a = 0; a < 2 * KK; ++a) {
    S[a] = f32x4{0, 0, 0, 0};
    if (unit) {
#pragma unroll
      for (int i = 0; i < 4; ++i) S[a][i] = tile_row4(a, g) + i == col ? 1.0f : 0.0f;
    }
  }
  if (start && live) load_state<KK>(start + col * p.dk, dk, p.vec_state, g, S);
  RowStore<P> late;  // y of the chunk before
  auto store_late = [&](int64_t ch) {
    const int64_t left = L - ch * kC;
    late.store(Yp + ch * kC * p.y_st, p.y_st, left < kC ? (int)left : kC, slice0 + 16 * w, p.dv, p.vec_y, lane);
  };
  place(kC);
  load_first(c0);
  load_part(c0, 0, 0, kPoints);
  load_late_tile(c0);
  wait_vmem_all();
  sync_lds();

  for (int64_t ch = c0; ch < c1; ++ch) {
    const int buf = NBUF == 2 ? (int)((ch - c0) & 1) : 0;
    lds_u8* const B = sm + buf * Lds::kBytes;
    f32x4 vf[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      vf[a] = P::template load_col4<Lds::Move::kPitch>(tile_at(buf), tile_row4(a, g), 16 * w, c);
      if constexpr (!Y) {  // zeros in columns of the identity, and past the image's last
#pragma unroll
        for (int i = 0; i < 4; ++i) vf[a][i] = live ? vf[a][i] : 0.0f;
      }
    }
    const bool more = ch + 1 < c1;
    if (more) load_first(ch + 1);
    auto point = [&](int n) {
      if constexpr (NBUF == 2) {
        if (more) load_part(ch + 1, buf ^ 1, n, n + 1);
      }
    };
    const lds_u8* const rows = B + Lds::kRows;
    if constexpr (STATES) {
      if (image) {
        uint8_t* im = image + ch * img_chunk;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
          P::put_kept(im + Image<P, KK>::kS + img_s + kk * Image<P, KK>::kFrag, lane, S[2 * kk], S[2 * kk + 1]);
      }
    } else if constexpr (Y) {
      if (ch > c0) store_late(ch - 1);
    }

    // Left operands come out of LDS one group ahead of the products that take them: with two
    // wavefronts to a SIMD the wait for a group read where it is used would show.
    typedef typename P::Exact Exact;
    typedef typename P::template Terms<NT> TermsT;
    auto get_rows = [&](Exact (&f)[4], int mat, int kk) {
#pragma unroll
      for (int a = 0; a < 4; ++a) f[a] = P::load_frag(B + mat + (a * KK + kk) * P::kFrag, lane);
    };
    auto get_t = [&](TermsT* t, int kk) {
#pragma unroll
      for (int a = 2 * kk; a < 4; ++a)
        P::load_terms(B + Lds::kRec + Rec::kT + tri_block(a, kk) * Rec::kTBlock, lane, t[a - 2 * kk]);
    };
    auto get_p = [&](TermsT* t, int kk) {
#pragma unroll
      for (int a = 2 * kk; a < 4; ++a)
        P::load_terms(B + Lds::kRec + Rec::kP + tri_block(a, kk) * Rec::kPBlock, lane, t[a - 2 * kk]);
    };
    constexpr int kRows = KK > 1 ? 4 : 2, kGroups = 2 * KK / kRows;
    auto get_kt = [&](Exact (&f)[kRows], int kk, int grp) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int a = grp * kRows + r;
        f[r] = P::load_frag_t(B + Lds::kK + (2 * kk * KK + (a >> 1)) * P::kFrag,
                              B + Lds::kK + ((2 * kk + 1) * KK + (a >> 1)) * P::kFrag, a, lane);
      }
    };
    // K S and Q S
    f32x4 ks[4], y[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) ks[a] = y[a] = f32x4{0, 0, 0, 0};
    constexpr bool kAhead = P::kBf16 || KK < 4 || !Y;  // fp32 with long keys has not the registers
    constexpr int kKeep = kAhead ? 2 : 1;
    Exact fk[kKeep][4], fq[kKeep][4];
    TermsT t0[4], t1[2];
    get_rows(fk[0], Lds::kK, 0);
    if constexpr (Y) get_rows(fq[0], Lds::kQ, 0);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      if (kk + 1 == KK) get_t(t0, 0);
      const int from = kAhead ? kk + 1 : kk;
      if (from < KK && from > 0) {
        get_rows(fk[from % kKeep], Lds::kK, from);
        if constexpr (Y) get_rows(fq[from % kKeep], Lds::kQ, from);
      }
      TermsT s;
      P::split(S[2 * kk], S[2 * kk + 1], s);
      point(kk);
      __builtin_amdgcn_sched_barrier(0);
      P::template mma_rows<NT>(fk[kk % kKeep], s, ks);
      if constexpr (Y) P::template mma_rows<NT>(fq[kk % kKeep], s, y);
    }
    if constexpr (VBUF != NBUF) {
      if (more) {
        sync_lds();  // every wavefront has read its columns of v
        load_late_tile(ch + 1);
      }
    }
    // R (beta is 0 for rows past the last step), and e^G (Q S) scale
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = tile_row4(a, g) * 4;
      const f32x4 eg = lds16f(rows + Rec::kGrow + r), be = lds16f(rows + Rec::kBeta + r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ks[a][i] = be[i] * fmaf(-eg[i], ks[a][i], vf[a][i]);
        if constexpr (Y) y[a][i] *= p.scale * eg[i];
      }
    }
    // U = T R
    f32x4 u[4];
    Exact kt[2][kRows];
    TermsT p0[4], p1[2];
#pragma unroll
    for (int a = 0; a < 4; ++a) u[a] = f32x4{0, 0, 0, 0};
    {
      TermsT r;
      get_t(t1, 1);
      P::split(ks[0], ks[1], r);
      point(KK);
      __builtin_amdgcn_sched_barrier(0);
      P::mma_tt_rows(t0, r, u);
      get_kt(kt[0], 0, 0);
      P::split(ks[2], ks[3], r);
      point(KK + 1);
      __builtin_amdgcn_sched_barrier(0);
      P::mma_tt_rows(t1, r, u + 2);
    }
    if constexpr (STATES) {
      if (image) {
        uint8_t* im = image + ch * img_chunk + Image<P, KK>::kU + img_u;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) P::put_kept(im + kk * Image<P, KK>::kFrag, lane, u[2 * kk], u[2 * kk + 1]);
      }
    }
    // S = e^{G_63} S + K^T (e^{G_63 - G} U), and Y += P U
    const float last = lds4f(rows + Rec::kGrow + (kC - 1) * 4);
    if constexpr (Y) get_p(p0, 0);
#pragma unroll
    for (int a = 0; a < 2 * KK; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[a][i] *= last;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const f32x4 d0 = lds16f(rows + Rec::kDecay + tile_row4(2 * kk, g) * 4);
      const f32x4 d1 = lds16f(rows + Rec::kDecay + tile_row4(2 * kk + 1, g) * 4);
      f32x4 e0, e1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e0[i] = d0[i] * u[2 * kk][i];
        e1[i] = d1[i] * u[2 * kk + 1][i];
      }
      TermsT e;
      P::split(e0, e1, e);
#pragma unroll
      for (int grp = 0; grp < kGroups; ++grp) {
        const int n = kk * kGroups + grp;
        if (n + 1 < 2 * kGroups) get_kt(kt[(n + 1) & 1], (n + 1) / kGroups, (n + 1) % kGroups);
        if (n < 2) point(KK + 2 + n);
        __builtin_amdgcn_sched_barrier(0);
        P::template mma_rows<NT>(kt[n & 1], e, S + grp * kRows);
      }
      if constexpr (Y) {
        TermsT uu;
        if (kk == 0) get_p(p1, 1);
        P::split(u[2 * kk], u[2 * kk + 1], uu);
        __builtin_amdgcn_sched_barrier(0);
        if (kk == 0) P::mma_tt_rows(p0, uu, y);
        else P::mma_tt_rows(p1, uu, y + 2);
      }
    }
    if constexpr (Y) late.take(y, c);
    if constexpr (NBUF == 1) {
      if (more) {
        sync_lds();
        load_part(ch + 1, 0, 0, kPoints);
      }
    }
    if (more) {
      wait_vmem_all();
      sync_lds();
    }
  }
  if constexpr (Y) store_late(c1 - 1);
  float* end = nullptr;
  if constexpr (SUMMARY) {
    end = p.local + bhs * (p.dv * p.dk);
    if (unit) {
      uint8_t* f = p.trans + bhs * (int64_t)Trans<P, KK>::kBytes + tile * KK * Trans<P, KK>::kFrag;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
        if (tile < 2 * KK) P::template put_image<3>(f + kk * Trans<P, KK>::kFrag, lane, S[2 * kk], S[2 * kk + 1]);
    }
  } else if (p.s_final && seg + 1 == (uint32_t)p.nseg) {
    end = p.s_final + bh * p.dv * p.dk;
  }
  if (end && live) store_state<KK>(end + col * p.dk, dk, p.vec_state, g, S);
}

// The states the segments start from, one after the other: S <- M S + S_local; or (BACK) the
// gradients of the states after them, last one first: dS <- M^T dS + dS_local. One wavefront = 16
// columns of one head. It is a chain of loads and products: M comes into LDS in halves (of its
// columns), with the segment's S_local beside the first, two halves ahead. `first`: S before the
// first segment, or dS after the last. Summaries stand at segment + bh * sums.
template <class P, int KK, bool BACK>
__global__ void __launch_bounds__(64) delta_combine_kernel(const DeltaParams p, const float* first, int sums) {
  typedef Trans<P, KK> Tr;
  constexpr int kHalves = KK > 1 ? 2 : 1, kPart = Tr::kBytes / kHalves, kUnits = kPart / 1024;
  constexpr int kLocal = 2 * KK;              // units of S_local: a tile each
  // a segment's S_local is read after the loads of the unit two ahead are on their way, which may
  // bring the next segment's or, with a segment to a unit, the one's after it
  constexpr int kSlots = kHalves == 1 ? 3 : 2;
  static_assert(kUnits + kLocal < 64, "the count of loads in flight has six bits");
  __shared__ __attribute__((aligned(128))) uint8_t smem[3 * kPart + kSlots * kLocal * 1024];
  lds_u8* const sm = (lds_u8*)smem;
  const int lane = threadIdx.x, g = lane >> 4, c = lane & 15;
  const uint32_t slices = (uint32_t)((p.dv + 15) / 16);
  const int64_t bh = blockIdx.x / slices;
  const int64_t col = (int64_t)(blockIdx.x % slices) * 16 + c;
  const bool live = col < p.dv;
  const int dk = (int)p.dk, steps = (int)p.nseg - 1;
  const int64_t state = p.dv * p.dk;
  const bool quads = dk % 4 == 0;  // the workspace's rows allow 16-byte access
  const uint8_t* M = p.trans + bh * sums * (int64_t)Tr::kBytes;
  const float* local = p.local + bh * sums * state + (live ? col : p.dv - 1) * p.dk;
  auto segment = [&](int n) { return (int64_t)(BACK ? steps - n : n); };
  // unit u: half u % kHalves of the (u / kHalves)-th segment, into buffer u % 3, its S_local into one of
  // kSlots more. S_local's rows past dk read its first ones, and are left out.
  auto load = [&](int u) {
    if (u >= steps * kHalves) return;
    lds_u8* const to = sm + (u % 3) * kPart;
    Mover<P, KK, 1, 1>::template run<kUnits>(0, lane, M + segment(u / kHalves) * Tr::kBytes + u % kHalves * kPart, to);
    if (u % kHalves == 0) {
      const float* from = local + segment(u / kHalves) * state;
      lds_u8* const beside = sm + 3 * kPart + u / kHalves % kSlots * kLocal * 1024;
#pragma unroll
      for (int a = 0; a < kLocal; ++a) {
        const int r = tile_row4(a, g);
        if (quads) dma16(from + (r < dk ? r : 0), (uint32_t)(uintptr_t)(beside + a * 1024));
      }
    }
  };
  f32x4 S[2 * KK];
#pragma unroll
  for (int a = 0; a < 2 * KK; ++a) S[a] = f32x4{0, 0, 0, 0};
  if (first && live) load_state<KK>(first + bh * state + col * p.dk, dk, p.vec_state, g, S);
  load(0);
  load(1);
  for (int n = 0; n < steps; ++n) {
    f32x4 next[2 * KK];
#pragma unroll
    for (int half = 0; half < kHalves; ++half) {
      const int u = n * kHalves + half;
      // unit u is there when no more is in flight than unit u + 1 takes (loads return in order)
      if (u + 1 >= steps * kHalves) wait_vmem_all();
      else if ((half + 1) % kHalves == 0 && quads) wait_vmem<kUnits + kLocal>();
      else wait_vmem<kUnits>();
      wait_lds_all();  // the reads of unit u - 1, whose buffer is loaded next
      load(u + 2);
      const lds_u8* const part = sm + (u % 3) * kPart;
      if (half == 0) {
#pragma unroll
        for (int a = 0; a < 2 * KK; ++a) {
          next[a] = f32x4{0, 0, 0, 0};
          if (quads && tile_row4(a, g) < dk) next[a] = lds16f(sm + 3 * kPart + (n % kSlots * kLocal + a) * 1024 + lane * 16);
        }
        if (!quads) load_state<KK>(local + segment(n) * state, dk, false, g, next);
      }
      if constexpr (BACK) {  // this half's columns of M are rows of M^T
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
          typename P::template Terms<3> s;
          P::split(S[2 * kk], S[2 * kk + 1], s);
#pragma unroll
          for (int k = 0; k < KK / kHalves; ++k) {
            typename P::template Terms<3> m[2];
            P::load_image_columns(part + 2 * k * KK * Tr::kFrag, KK, kk, 0, lane, m[0]);
            P::load_image_columns(part + 2 * k * KK * Tr::kFrag, KK, kk, 1, lane, m[1]);
            P::mma_tt_rows(m, s, next + 2 * (half * (KK / kHalves) + k));
          }
        }
        continue;
      }
#pragma unroll
      for (int k = 0; k < KK / kHalves; ++k) {
        const int kk = half * (KK / kHalves) + k;
        typename P::template Terms<3> s;
        P::split(S[2 * kk], S[2 * kk + 1], s);
#pragma unroll
        for (int a = 0; a < 2 * KK; a += 2) {
          typename P::template Terms<3> m[2];
          P::load_image_tile(part + 2 * k * KK * Tr::kFrag, KK, a, lane, m[0]);
          P::load_image_tile(part + 2 * k * KK * Tr::kFrag, KK, a + 1, lane, m[1]);
          P::mma_tt_rows(m, s, next + a);
        }
      }
    }
#pragma unroll
    for (int a = 0; a < 2 * KK; ++a) S[a] = next[a];
    const int64_t to = BACK ? segment(n) - 1 : n + 1;
    if (live) store_state<KK>(p.starts + (bh * p.nseg + to) * state + col * p.dk, dk, quads, g, S);
  }
}

template <class P, int KK, Mode MODE, int NW>
hipError_t scan_go(const DeltaParams& p, hipStream_t stream) {
  int64_t items = p.batch * p.nheads * ((p.dv + 16 * NW - 1) / (16 * NW)) * p.nseg;
  if (is_summary(MODE))
    items = p.batch * p.nheads * (p.nseg - (MODE == kSummary)) * ((p.dv + 16 * NW - 1) / (16 * NW) + (32 * KK + 16 * NW - 1) / (16 * NW));
  delta_scan_kernel<P, KK, NW, MODE><<<dim3((unsigned)items), dim3(64 * NW), 0, stream>>>(p);
  return hipGetLastError();
}

template <class P, int KK, Mode MODE>
hipError_t scan_width(const DeltaParams& p, hipStream_t stream) {
  return delta_scan_waves(p) == 8 ? scan_go<P, KK, MODE, 8>(p, stream) : scan_go<P, KK, MODE, 4>(p, stream);
}

template <class P, int KK, bool BACK>
hipError_t combine(const DeltaParams& p, const float* first, int sums, hipStream_t stream) {
  const unsigned items = (unsigned)(p.batch * p.nheads * ((p.dv + 15) / 16));
  delta_combine_kernel<P, KK, BACK><<<dim3(items), 64, 0, stream>>>(p, first, sums);
  return hipGetLastError();
}

// prep and scan
template <class P, int KK, bool STATES>
hipError_t forward(const DeltaParams& p, hipStream_t stream) {
  const int64_t heads = p.batch * p.nheads;
  const dim3 grid((unsigned)p.nchunks, (unsigned)(heads < 65535 ? heads : 65535), (unsigned)((heads + 65534) / 65535));
  delta_prep_kernel<P, KK, STATES><<<grid, 256, 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.nseg > 1) {
    e = scan_width<P, KK, STATES ? kSummaryBwd : kSummary>(p, stream);
    if (e != hipSuccess) return e;
    e = combine<P, KK, false>(p, p.s0, (int)p.nseg - !STATES, stream);
    if (e != hipSuccess) return e;
  }
  return scan_width<P, KK, STATES ? kStates : kY>(p, stream);
}

// Rows of any stride and length as contiguous ones, padded with zeros: 8 entries a thread.
template <typename IO>
__global__ void __launch_bounds__(256) delta_pack_kernel(const DeltaPack p) {
  const DeltaPack::Item t = p.item[blockIdx.y];
  const int64_t per = t.pad / 8, count = p.batch * t.heads * p.L * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int64_t c = i % per * 8, row = i / per;
    const int64_t step = row % p.L, bh = row / p.L, h = bh % t.heads, b = bh / t.heads;
    const IO* from = static_cast<const IO*>(t.src) + b * t.sb + step * t.st + h * t.sh + c;
    IO v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < t.n ? from[e] : (IO)0;
    IO* to = static_cast<IO*>(t.dst) + i * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) to[e] = v[e];
  }
}

template <class P, bool STATES>
hipError_t forward_key(const DeltaParams& p, hipStream_t stream) {
  switch (delta_pad_key(p.dk)) {
    case 32: return forward<P, 1, STATES>(p, stream);
    case 64: return forward<P, 2, STATES>(p, stream);
    default: return forward<P, 4, STATES>(p, stream);
  }
}

template <class P>
hipError_t combine_back(const DeltaParams& p, const float* first, int sums, hipStream_t stream) {
  switch (delta_pad_key(p.dk)) {
    case 32: return combine<P, 1, true>(p, first, sums, stream);
    case 64: return combine<P, 2, true>(p, first, sums, stream);
    default: return combine<P, 4, true>(p, first, sums, stream);
  }
}

}  // namespace

size_t delta_record_bytes(bool bf16, bool bwd) {
  // room for three terms
  if (bwd) return bf16 ? Record<Bf16<3>, true>::kBytes : Record<F32, true>::kBytes;
  return bf16 ? Record<Bf16<3>, false>::kBytes : Record<F32, false>::kBytes;
}

size_t delta_image_bytes(int64_t dk, int64_t dv) {
  switch (delta_pad_key(dk)) {
    case 32: return (size_t)((dv + 31) / 32) * Image<F32, 1>::kBytes;
    case 64: return (size_t)((dv + 31) / 32) * Image<F32, 2>::kBytes;
    default: return (size_t)((dv + 31) / 32) * Image<F32, 4>::kBytes;
  }
}

// Columns per workgroup: as many as leave a workgroup for every CU (a wider one reads K, Q, T and
// P once for more columns). 4096 steps of keys of 128 in bf16, the whole call, at 64 and at 128
// columns: 256 heads of 128 770 and 685 us; 128 heads of 128 376 and 462 us; 64 heads of 256 315 and
// 410 us. In fp32 the wide scan with keys of 128 spills seven registers and is the faster all the same
// (256 heads of 128 1.88 and 1.64 ms).
int delta_scan_waves(const DeltaParams& p) {
  const int64_t tiles = (p.dv + 15) / 16;
  return tiles > 4 && p.batch * p.nheads * ((tiles + 7) / 8) * p.nseg >= kCUs ? 8 : 4;
}

// In steps of one chunk of a workgroup of 128 columns: a whole sequence takes nchunks, a split one
// its summary pass, its scan, up to one for each segment in the combine kernel (less with short
// keys, and as fp32 chunks take longer), and three for the two launches. Split where that is a fifth
// less. The call, whole and split: 2 x 8 heads of 64 x 64 in fp32, 16 chunks 111 and 59 us; 128 x 128
// in bf16, 16 heads of 1024 chunks 4109 and 1250 us, of 64 chunks 266 and 145 us, 32 heads of 64
// chunks 277 and 190 us, of 32 chunks 144 and 125 us (16 heads of 16 chunks are left whole: 78 us). The backward pass takes both scans twice, and its own combine
// run, for two whole ones: the same comparison.
void delta_plan(DeltaParams* p) {
  p->nseg = 1;
  p->seg_chunks = p->nchunks;
  const int64_t heads = p->batch * p->nheads;
  const int64_t wide = heads * ((p->dv + 127) / 128);  // workgroups of 128 columns
  if (wide <= 0 || wide > kCUs / 4) return;
  const int64_t step = delta_pad_key(p->dk) / (p->bf16 ? 1 : 2);
  int64_t best = p->nchunks - p->nchunks / 5;
  for (int64_t n = 2; n <= 64 && 2 * n <= p->nchunks; ++n) {
    const int64_t len = (p->nchunks + n - 1) / n;
    const int64_t rounds = (n * wide + kCUs - 1) / kCUs + (n * (wide + heads) + kCUs - 1) / kCUs;
    const int64_t cost = len * rounds + n * step / 128 + 3;
    if (cost < best) {
      best = cost;
      p->seg_chunks = len;
    }
  }
  if (p->seg_chunks < p->nchunks) p->nseg = (p->nchunks + p->seg_chunks - 1) / p->seg_chunks;
}

DeltaSplitLayout delta_split_layout(const DeltaParams& p) {
  DeltaSplitLayout l = {0, 0, 0, 0};
  if (p.nseg <= 1) return l;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  const size_t segs = (size_t)p.batch * p.nheads * p.nseg, kk = delta_pad_key(p.dk) / 32;
  const size_t state = (size_t)p.dv * p.dk * sizeof(float);
  l.trans = up(segs * state);
  l.starts = l.trans + up(segs * 2 * kk * kk * (p.bf16 ? Bf16<3>::kImageFrag<3> : F32::kImageFrag<3>));
  l.total = l.starts + up(segs * state);
  return l;
}

hipError_t launch_delta_pack(const DeltaPack& p, hipStream_t stream) {
  if (p.count == 0) return hipSuccess;
  int64_t most = 0;
  for (int i = 0; i < p.count; ++i) {
    const int64_t n = p.batch * p.item[i].heads * p.L * (p.item[i].pad / 8);
    if (n > most) most = n;
  }
  const int64_t want = (most + 255) / 256;
  const dim3 grid((unsigned)(want < 16 * kCUs ? want : 16 * kCUs), (unsigned)p.count);
  if (p.bf16) delta_pack_kernel<bf16_bits><<<grid, 256, 0, stream>>>(p);
  else delta_pack_kernel<float><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_delta_fwd(const DeltaParams& p, hipStream_t stream) {
  if (!p.bf16) return forward_key<F32, false>(p, stream);
  return p.terms == 3 ? forward_key<Bf16<3>, false>(p, stream) : forward_key<Bf16<2>, false>(p, stream);
}

hipError_t launch_delta_combine_back(const DeltaBwdParams& q, hipStream_t stream) {
  const int sums = (int)q.f.nseg;
  if (!q.f.bf16) return combine_back<F32>(q.f, q.ds_final, sums, stream);
  return combine_back<Bf16<3>>(q.f, q.ds_final, sums, stream);  // M has three terms in any case
}

hipError_t launch_delta_states(const DeltaParams& p, hipStream_t stream) {
  if (!p.bf16) return forward_key<F32, true>(p, stream);
  return p.terms == 3 ? forward_key<Bf16<3>, true>(p, stream) : forward_key<Bf16<2>, true>(p, stream);
}

}  // namespace ssm
