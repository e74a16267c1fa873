// Building blocks of the chunked gated delta rule on the gfx950 matrix cores.
//
// The rule, per head, with a state S of dk x dv:
//   S_t = a_t S_{t-1} + k_t u_t^T,  u_t = beta_t (v_t - a_t S_{t-1}^T k_t),  a_t = e^{g_t}
//   y_t = scale S_t^T q_t
// Over a chunk of 64 steps that starts from S, with G_t the inclusive sum of g in the chunk and
// D_ts = e^{G_t - G_s} for s <= t:
//   A_ts = beta_t (k_t . k_s) D_ts (s < t),  T = (I + A)^{-1},  P_ts = scale (q_t . k_s) D_ts
//   R = beta (V - e^G (K S)),  U = T R,  Y = scale e^G (Q S) + P U
//   S' = e^{G_63} S + K^T (e^{G_63 - G} U)
// T and P do not depend on S: the prep kernel makes them for every chunk at once; what is left
// runs in order and is a chain of products in which each column of S, V, U and Y is on its own.
//
// Tiles. All products are 16x16x32 (bf16) or 16x16x4 (fp32) MFMA. A wavefront owns 16 columns
// and keeps S, U and every other operand of the chain in accumulator layout (lane (g, c), g =
// lane / 16, c = lane % 16, holds D[4g + i][c]); as the right operand of the next product an
// accumulator pair is used as it is. That needs the contraction index in another order than the
// plain one, so rows are numbered through tile_row: row 4g + i of tile a stands for index
// 32 (a / 2) + 8g + 4 (a % 2) + i. Then lane g's 8 values of a tile pair are 8 consecutive
// indices, which is also what a left operand in plain order holds. The left operands (K, Q, T, P)
// are stored in 16x32 fragments: the fragment (a, kk) holds, at lane (g, c), the 8 entries
// [tile_row(a, c)][32 kk + 8 g .. +8).
//
// Precision. MFMA accumulates in fp32. bf16 inputs are exact operands. Values computed in fp32
// (S, R, U, T, P) enter a product as a sum of bf16 terms, each the bf16 of what the ones before
// left: three terms carry all 24 bits, so that every result is as good as fp32 arithmetic makes it
// before its one rounding to the io type. A caller may choose two, which carry 16
// (SSM_DELTA_OPERANDS_16). fp32 io runs on the fp32 MFMA throughout.
#pragma once
#include "delta_internal.h"
#include "scan_kernels.h"

namespace ssm {
namespace delta {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kC = kDeltaChunk;
constexpr int kTBlocks = 6;  // 16x32 fragments of a lower triangular 64x64 matrix
// fragment (a, kk) of a lower triangular matrix; the two with a < 2, kk = 1 are zero
__host__ __device__ constexpr int tri_block(int a, int kk) { return a < 2 ? a : 2 * a - 2 + kk; }
// steps (or keys) of the accumulator rows 4g .. 4g + 3 of tile a
__device__ __forceinline__ int tile_row4(int a, int g) { return 32 * (a >> 1) + 8 * g + 4 * (a & 1); }
// index of row m of tile a, and its inverse for a row t of a 64-row (128-row) operand
__device__ __forceinline__ int tile_row(int a, int m) { return tile_row4(a, m >> 2) + (m & 3); }
__device__ __forceinline__ int row_tile(int t) { return 2 * (t >> 5) + ((t >> 2) & 1); }
__device__ __forceinline__ int row_slot(int t) { return 4 * ((t >> 3) & 3) + (t & 3); }

__device__ __forceinline__ u32x4 lds16(const lds_u8* p) {
  return *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(p);
}
__device__ __forceinline__ f32x4 lds16f(const lds_u8* p) {
  return *reinterpret_cast<const __attribute__((address_space(3))) f32x4*>(p);
}
__device__ __forceinline__ float lds4f(const lds_u8* p) {
  return *reinterpret_cast<const __attribute__((address_space(3))) float*>(p);
}
__device__ __forceinline__ void sts16(lds_u8* p, u32x4 v) {
  *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(p) = v;
}
__device__ __forceinline__ void sts16f(lds_u8* p, f32x4 v) {
  *reinterpret_cast<__attribute__((address_space(3))) f32x4*>(p) = v;
}
// transposed read of 4 bf16: in each group of 16 lanes, lane i's slot q receives element i % 4
// of the 8 bytes that lane 4q + i / 4 addressed
__device__ __forceinline__ u32x2 ldtr(const lds_u8* p) {
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      reinterpret_cast<lds_s16x4*>(const_cast<lds_u8*>(p)));
  return __builtin_bit_cast(u32x2, v);
}

// Direct load of 16 bytes per lane into LDS at lds + 16 * lane (lds wave-uniform). The compiler
// keeps no account of it: the kernels wait for it (wait_vmem_all and a barrier) before the buffer
// is read, and issue none into a buffer before a barrier has ended every read of it. Nor does it put
// wait states into the assembly: one stands between the write of M0 and the load that takes its base
// from it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src),
               "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory", "m0");
}
#pragma clang diagnostic pop
// The same from the wave-uniform address `src` plus a 32-bit byte offset a lane. With M0's write, five
// wait states after what may be a v_readfirstlane of the address.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void* src, uint32_t off, uint32_t lds) {
  const uint64_t at = (uint64_t)src;
  const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(at >> 32)) << 32 |
                        (uint32_t)__builtin_amdgcn_readfirstlane((int)at);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base),
               "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory", "m0");
}
#pragma clang diagnostic pop
// Barrier for LDS data: this wavefront's LDS accesses complete, then s_barrier. Global loads and
// stores stay in flight (the clobber keeps memory accesses from moving across it).
__device__ __forceinline__ void sync_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
// every LDS access of this wavefront done
__device__ __forceinline__ void wait_lds_all() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// at most N global memory operations of this wavefront in flight
template <int N>
__device__ __forceinline__ void wait_vmem() {
  static_assert(N >= 0 && N < 64, "");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4) << 14);
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void wait_vmem_all() {
  __builtin_amdgcn_s_waitcnt(0x0f70);
  asm volatile("" ::: "memory");
}

// 8 floats of a right operand (one lane's part of a 32-row slice)
struct Eight {
  f32x4 a, b;
};

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// io bf16: exact operands are bf16, computed ones sums of NT bf16 terms
template <int NT>
struct Bf16 {
  typedef bf16_bits IO;
  static constexpr bool kBf16 = true;
  static constexpr int kFrag = 1024;    // bytes of a 16x32 fragment of an exact operand
  static constexpr int kTerms = NT;
  typedef u32x4 Exact;
  template <int N>
  struct Terms {
    u32x4 t[N];
  };
  template <int N>
  static __device__ __forceinline__ void split(const f32x4 a, const f32x4 b, Terms<N>& r) {
    float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = pack_bf16x2(v[2 * e], v[2 * e + 1]);
        r.t[n][e] = w;
        if (n + 1 < N) {
          v[2 * e] -= lo_f(w);
          v[2 * e + 1] -= hi_f(w);
        }
      }
  }
  static __device__ __forceinline__ f32x4 mma1(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  // exact x exact, exact x terms (the first USE of them), terms x terms (their leading products)
  static __device__ __forceinline__ f32x4 mma(const Exact& a, const Exact& b, f32x4 c) {
    return mma1(a, b, c);
  }
  template <int USE, int N>
  static __device__ __forceinline__ f32x4 mma(const Exact& a, const Terms<N>& b, f32x4 c) {
#pragma unroll
    for (int n = USE - 1; n >= 0; --n) c = mma1(a, b.t[n], c);
    return c;
  }
  template <int NA, int N>
  static __device__ __forceinline__ f32x4 mma_tt(const Terms<NA>& a, const Terms<N>& b, f32x4 c) {
#pragma unroll
    for (int s = NA - 1; s >= 0; --s)
#pragma unroll
      for (int i = 0; i <= s; ++i)
        if (s - i < N) c = mma1(a.t[i], b.t[s - i], c);
    return c;
  }
  // The same for R rows of tiles at once, the rows innermost: a product is then not followed by one
  // that waits for it (the matrix core takes a dependent one only when the first has ended).
  template <int USE, int N, int R>
  static __device__ __forceinline__ void mma_rows(const Exact (&a)[R], const Terms<N>& b, f32x4* c) {
#pragma unroll
    for (int n = USE - 1; n >= 0; --n)
#pragma unroll
      for (int r = 0; r < R; ++r) c[r] = mma1(a[r], b.t[n], c[r]);
  }
  template <int NA, int N, int R>
  static __device__ __forceinline__ void mma_tt_rows(const Terms<NA> (&a)[R], const Terms<N>& b, f32x4* c) {
#pragma unroll
    for (int s = NA - 1; s >= 0; --s)
#pragma unroll
      for (int i = 0; i <= s; ++i)
        if (s - i < N)
#pragma unroll
          for (int r = 0; r < R; ++r) c[r] = mma1(a[r].t[i], b.t[s - i], c[r]);
  }
  // 8 consecutive entries
  static __device__ __forceinline__ Exact load8(const IO* p) { return *reinterpret_cast<const u32x4*>(p); }
  static __device__ __forceinline__ void store_frag(lds_u8* f, int lane, const Exact& v) {
    sts16(f + lane * 16, v);
  }
  static __device__ __forceinline__ Exact load_frag(const lds_u8* f, int lane) {
    return lds16(f + lane * 16);
  }
  template <int N>
  static __device__ __forceinline__ void load_terms(const lds_u8* f, int lane, Terms<N>& r) {
#pragma unroll
    for (int n = 0; n < N; ++n) r.t[n] = lds16(f + n * kFrag + lane * 16);
  }
  // The fragment (a, kk) of the transpose of an operand X whose own fragment (a, kk) lies at
  // base(a, kk): entries X[32 kk + 8g + j][tile_row(a, c)], from the fragments (2 kk, a / 2) and
  // (2 kk + 1, a / 2) of X, `step` bytes apart.
  static __device__ __forceinline__ Exact load_frag_t(const lds_u8* f0, const lds_u8* f1, int a,
                                                      int lane) {
    const int g = lane >> 4, c = lane & 15;
    const int off = ((c & 3) * 16 + 4 * g + (c >> 2)) * 16 + 8 * (a & 1);
    const u32x2 x = ldtr(f0 + off), y = ldtr(f1 + off);
    return u32x4{x[0], x[1], y[0], y[1]};
  }
  template <int N>
  static __device__ __forceinline__ void load_terms_t(const lds_u8* f0, const lds_u8* f1, int a,
                                                      int lane, Terms<N>& r) {
#pragma unroll
    for (int n = 0; n < N; ++n) r.t[n] = load_frag_t(f0 + n * kFrag, f1 + n * kFrag, a, lane);
  }
  // bytes of an image fragment of N terms
  template <int N>
  static constexpr int kImageFrag = N * 1024;
  // What the backward pass keeps in memory: two terms, or, for three, fp32, which is less to move; the
  // gradient kernel makes terms of it on the way in.
  static constexpr bool kStaged = NT == 3;
  static __device__ __forceinline__ void put_kept(uint8_t* f, int lane, const f32x4 a, const f32x4 b) {
    if constexpr (kStaged) {
      *reinterpret_cast<f32x4*>(f + lane * 16) = a;
      *reinterpret_cast<f32x4*>(f + 1024 + lane * 16) = b;
    } else {
      put_image<2>(f, lane, a, b);
    }
  }
  // Where lane (g, c)'s 16 bytes of an image fragment lie: slots of odd groups in another order and
  // the 8-byte halves of the last two groups exchanged, so that a transposed read, which takes one
  // half of 8 slots of each group, meets every bank alike.
  static __device__ __forceinline__ int image_slot(int g, int c) { return g * 16 + (c ^ (4 * (g & 1))); }
  static __device__ __forceinline__ u32x4 image_halves(int g, const u32x4 v) {
    return g & 2 ? u32x4{v[2], v[3], v[0], v[1]} : v;
  }
  // An operand that contracts over the 32 columns of an image part (`nk` fragments a tile) and
  // whose row is entry 32 kk + x(c) at lane (g, c): the 8 bytes that lane 4q + r of a group of 16
  // addresses hold the entries x(4r) .. x(4r) + 3 of column 8g + q.
  template <int N>
  static __device__ __forceinline__ void load_image(const lds_u8* part, int nk, int kk, int grp,
                                                    int half, int lane, Terms<N>& r) {
    const int g = lane >> 4, c = lane & 15;
    const int off = ((g >> 1) * nk + kk) * kImageFrag<N> + image_slot(grp, 8 * (g & 1) + (c >> 2)) * 16 +
                    8 * (half ^ (grp >> 1));
    const lds_u8 *const f0 = part + off, *const f1 = part + (off ^ 64);  // columns + 4: slot ^ 4
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const u32x2 x = ldtr(f0 + n * 1024), y = ldtr(f1 + n * 1024);
      r.t[n] = u32x4{x[0], x[1], y[0], y[1]};
    }
  }
  // x(c) = tile_row(a, c) - 32 (a / 2): the rows of tile a, kk = a / 2
  template <int N>
  static __device__ __forceinline__ void load_image_tile(const lds_u8* part, int nk, int a, int lane,
                                                         Terms<N>& r) {
    load_image(part, nk, a >> 1, lane & 3, a & 1, lane, r);
  }
  // x(c) = 16 (w % 2) + c: the entries 16w .. 16w + 15 in order, kk = w / 2
  template <int N>
  static __device__ __forceinline__ void load_image_block(const lds_u8* part, int nk, int w, int lane,
                                                          Terms<N>& r) {
    const int q = lane & 3;
    load_image(part, nk, w >> 1, 2 * (w & 1) + (q >> 1), q & 1, lane, r);
  }
  // A left operand whose rows are the columns of an image part in tile order (row tile a of the 32)
  // and that contracts over the part's entries 32 kk .. +32: the fragments as they lie.
  template <int N>
  static __device__ __forceinline__ void load_image_columns(const lds_u8* part, int nk, int kk, int a,
                                                            int lane, Terms<N>& r) {
    const int g = lane >> 4, col = tile_row(a, lane & 15);
    const lds_u8* const f = part + ((col >> 4) * nk + kk) * kImageFrag<N> + image_slot(g, col & 15) * 16;
#pragma unroll
    for (int n = 0; n < N; ++n) r.t[n] = image_halves(g, lds16(f + n * 1024));
  }
  template <int N>
  static __device__ __forceinline__ void put_image(uint8_t* f, int lane, const f32x4 a, const f32x4 b) {
    Terms<N> t;
    split(a, b, t);
#pragma unroll
    for (int n = 0; n < N; ++n)
      *reinterpret_cast<u32x4*>(f + n * 1024 + image_slot(lane >> 4, lane & 15) * 16) = image_halves(lane >> 4, t.t[n]);
  }
  // the same in LDS
  template <int N>
  static __device__ __forceinline__ void put_image(lds_u8* f, int lane, const f32x4 a, const f32x4 b) {
    Terms<N> t;
    split(a, b, t);
#pragma unroll
    for (int n = 0; n < N; ++n) sts16(f + n * 1024 + image_slot(lane >> 4, lane & 15) * 16, image_halves(lane >> 4, t.t[n]));
  }
  static __device__ __forceinline__ void floats(const u32x4 w, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = lo_f(w[e]);
      f[2 * e + 1] = hi_f(w[e]);
    }
  }
  template <int N>
  static __device__ __forceinline__ void floats(const Terms<N>& t, float (&f)[8]) {
    floats(t.t[0], f);
#pragma unroll
    for (int n = 1; n < N; ++n) {
      float l[8];
      floats(t.t[n], l);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += l[e];
    }
  }
  static __device__ __forceinline__ Exact exact(const f32x4 a, const f32x4 b) {
    return u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]),
                 pack_bf16x2(b[2], b[3])};
  }
  static __device__ __forceinline__ void store8(IO* p, const f32x4 a, const f32x4 b) {
    *reinterpret_cast<u32x4*>(p) = exact(a, b);
  }
  // Rows t .. t + 3 of column `col` of a row-major tile in LDS: lane c of a group of 16 gets
  // column c of the 16 from col0 (col = col0 + c).
  // The 16-byte pieces of row r are stored at piece ^ tile_swizzle(r): the 16 rows that one read
  // takes (four from each lane group's t) then lie on different banks.
  template <int PITCH>
  static __device__ __forceinline__ int tile_swizzle(int r) {
    return (2 * ((r & 3) | (r >> 1 & 4))) & (PITCH / 16 - 1);
  }
  template <int PITCH>
  static __device__ __forceinline__ f32x4 load_col4(const lds_u8* tile, int t, int col0, int c) {
    const int r = t + (c >> 2), piece = (col0 / 8 + ((c & 3) >> 1)) ^ tile_swizzle<PITCH>(r);
    const u32x2 w = ldtr(tile + r * PITCH + piece * 16 + 8 * (c & 1));
    return f32x4{lo_f(w[0]), hi_f(w[0]), lo_f(w[1]), hi_f(w[1])};
  }
  // What a lane stores of a tile that holds rows 4g + i of column c: Quad::kRows rows of
  // Quad::kCols consecutive columns. Lanes c .. c + 3 exchange their 4 x 4 entries, so that lane c
  // has row c % 4 of columns 4 (c / 4) .. + 3.
  struct Quad {
    u32x2 w;
  };
  static constexpr bool kTransposed = true;
  static __device__ __forceinline__ Quad quad(const f32x4 v, int c) {
    const uint32_t p0 = pack_bf16x2(v[0], v[1]), p1 = pack_bf16x2(v[2], v[3]);
    const uint32_t x0 = __builtin_amdgcn_update_dpp(0, p0, 0xb1, 0xf, 0xf, true);  // lane c ^ 1
    const uint32_t x1 = __builtin_amdgcn_update_dpp(0, p1, 0xb1, 0xf, 0xf, true);
    const uint32_t sel = c & 1 ? 0x07060302u : 0x01000504u;
    const uint32_t a0 = __builtin_amdgcn_perm(p0, x0, sel), a1 = __builtin_amdgcn_perm(p1, x1, sel);
    const bool low = (c & 2) == 0;
    const uint32_t got = __builtin_amdgcn_update_dpp(0, low ? a1 : a0, 0x4e, 0xf, 0xf, true);  // c ^ 2
    return Quad{u32x2{low ? a0 : got, low ? got : a1}};
  }
  // terms x exact
  template <int N>
  static __device__ __forceinline__ f32x4 mma_te(const Terms<N>& a, const Exact& b, f32x4 c) {
#pragma unroll
    for (int n = N - 1; n >= 0; --n) c = mma1(a.t[n], b, c);
    return c;
  }
  // eight floats of an image fragment in LDS (some eight; each lane other ones)
  static __device__ __forceinline__ void image_floats(const lds_u8* f, int lane, float (&v)[8]) {
    Terms<NT> t;
    load_terms(f, lane, t);
    floats(t, v);
  }
  // terms of a right operand, handed to another wavefront through LDS
  template <int N>
  static __device__ __forceinline__ void store_terms(lds_u8* f, int lane, const Terms<N>& t) {
#pragma unroll
    for (int n = 0; n < N; ++n) sts16(f + n * 1024 + lane * 16, t.t[n]);
  }
  // four consecutive entries (columns 4 (j4 & 1) .. +4 of the 8 at lane (g, c)) of a fragment of
  // N terms in global memory
  template <int N>
  static __device__ __forceinline__ void put4(uint8_t* f, int g, int c, int half, const f32x4 v) {
    f32x4 r = v;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const u32x2 w = {pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3])};
      *reinterpret_cast<u32x2*>(f + n * kFrag + (g * 16 + c) * 16 + 8 * half) = w;
      r[0] -= lo_f(w[0]); r[1] -= hi_f(w[0]); r[2] -= lo_f(w[1]); r[3] -= hi_f(w[1]);
    }
  }
};

// io fp32: every operand is fp32; a fragment is two halves of 16 bytes a lane
struct F32 {
  typedef float IO;
  static constexpr bool kBf16 = false;
  static constexpr int kFrag = 2048;
  static constexpr int kTerms = 1;
  typedef Eight Exact;
  template <int N>
  struct Terms {
    Eight t;
  };
  template <int N>
  static __device__ __forceinline__ void split(const f32x4 a, const f32x4 b, Terms<N>& r) {
    r.t = Eight{a, b};
  }
  static __device__ __forceinline__ f32x4 mma(const Eight& a, const Eight& b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[i], b.a[i], c, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[i], b.b[i], c, 0, 0, 0);
    return c;
  }
  template <int USE, int N>
  static __device__ __forceinline__ f32x4 mma(const Eight& a, const Terms<N>& b, f32x4 c) {
    return mma(a, b.t, c);
  }
  template <int NA, int N>
  static __device__ __forceinline__ f32x4 mma_tt(const Terms<NA>& a, const Terms<N>& b, f32x4 c) {
    return mma(a.t, b.t, c);
  }
  template <int R>
  static __device__ __forceinline__ void rows8(const Eight (&a)[R], const Eight& b, f32x4* c) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r) c[r] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r].a[i], b.a[i], c[r], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r) c[r] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r].b[i], b.b[i], c[r], 0, 0, 0);
  }
  template <int USE, int N, int R>
  static __device__ __forceinline__ void mma_rows(const Eight (&a)[R], const Terms<N>& b, f32x4* c) {
    rows8(a, b.t, c);
  }
  template <int NA, int N, int R>
  static __device__ __forceinline__ void mma_tt_rows(const Terms<NA> (&a)[R], const Terms<N>& b, f32x4* c) {
    Eight x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = a[r].t;
    rows8(x, b.t, c);
  }
  static __device__ __forceinline__ Exact load8(const IO* p) {
    return Eight{*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)};
  }
  static __device__ __forceinline__ void store_frag(lds_u8* f, int lane, const Exact& v) {
    sts16f(f + lane * 16, v.a);
    sts16f(f + 1024 + lane * 16, v.b);
  }
  static __device__ __forceinline__ Exact load_frag(const lds_u8* f, int lane) {
    return Eight{lds16f(f + lane * 16), lds16f(f + 1024 + lane * 16)};
  }
  template <int N>
  static __device__ __forceinline__ void load_terms(const lds_u8* f, int lane, Terms<N>& r) {
    r.t = load_frag(f, lane);
  }
  static __device__ __forceinline__ Exact load_frag_t(const lds_u8* f0, const lds_u8* f1, int a,
                                                      int lane) {
    const int g = lane >> 4, c = lane & 15;
    // row 8g + j of the 32: tile j / 4 of the pair, slot 4g + j % 4; column 8 (c / 4) + 4 (a % 2)
    // + c % 4 of the 32: lane group c / 4, half a % 2, element c % 4
    const int off = (a & 1) * 1024 + ((c >> 2) * 16 + 4 * g) * 16 + 4 * (c & 3);
    Eight r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.a[j] = lds4f(f0 + off + 16 * j);
      r.b[j] = lds4f(f1 + off + 16 * j);
    }
    return r;
  }
  template <int N>
  static __device__ __forceinline__ void load_terms_t(const lds_u8* f0, const lds_u8* f1, int a,
                                                      int lane, Terms<N>& r) {
    r.t = load_frag_t(f0, f1, a, lane);
  }
  template <int N>
  static constexpr int kImageFrag = 2048;
  static constexpr bool kStaged = false;
  static __device__ __forceinline__ void put_kept(uint8_t* f, int lane, const f32x4 a, const f32x4 b) {
    put_image<1>(f, lane, a, b);
  }
  template <int N>
  static __device__ __forceinline__ void load_image_tile(const lds_u8* part, int nk, int a, int lane,
                                                         Terms<N>& r) {
    const int g = lane >> 4, c = lane & 15;
    image(part + ((g >> 1) * nk + (a >> 1)) * 2048 + (a & 1) * 1024 +
              ((c >> 2) * 16 + 8 * (g & 1)) * 16 + 4 * (c & 3), r);
  }
  template <int N>
  static __device__ __forceinline__ void load_image_block(const lds_u8* part, int nk, int w, int lane,
                                                          Terms<N>& r) {
    const int g = lane >> 4, x = 16 * (w & 1) + (lane & 15);
    image(part + ((g >> 1) * nk + (w >> 1)) * 2048 + ((x >> 2) & 1) * 1024 +
              ((x >> 3) * 16 + 8 * (g & 1)) * 16 + 4 * (x & 3), r);
  }
  template <int N>
  static __device__ __forceinline__ void image(const lds_u8* f, Terms<N>& r) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.t.a[j] = lds4f(f + 16 * j);
      r.t.b[j] = lds4f(f + 64 + 16 * j);
    }
  }
  template <int N>
  static __device__ __forceinline__ void load_image_columns(const lds_u8* part, int nk, int kk, int a,
                                                            int lane, Terms<N>& r) {
    const int g = lane >> 4, col = tile_row(a, lane & 15);
    const lds_u8* const f = part + ((col >> 4) * nk + kk) * 2048 + (g * 16 + (col & 15)) * 16;
    r.t = Eight{lds16f(f), lds16f(f + 1024)};
  }
  template <int N>
  static __device__ __forceinline__ void put_image(uint8_t* f, int lane, const f32x4 a, const f32x4 b) {
    *reinterpret_cast<f32x4*>(f + lane * 16) = a;
    *reinterpret_cast<f32x4*>(f + 1024 + lane * 16) = b;
  }
  static __device__ __forceinline__ void floats(const Eight& w, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = w.a[e];
      f[4 + e] = w.b[e];
    }
  }
  template <int N>
  static __device__ __forceinline__ void floats(const Terms<N>& t, float (&f)[8]) { floats(t.t, f); }
  static __device__ __forceinline__ Exact exact(const f32x4 a, const f32x4 b) { return Eight{a, b}; }
  static __device__ __forceinline__ void store8(IO* p, const f32x4 a, const f32x4 b) {
    *reinterpret_cast<f32x4*>(p) = a;
    *reinterpret_cast<f32x4*>(p + 4) = b;
  }
  template <int PITCH>
  static __device__ __forceinline__ int tile_swizzle(int) { return 0; }
  template <int PITCH>
  static __device__ __forceinline__ f32x4 load_col4(const lds_u8* tile, int t, int col0, int c) {
    f32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = lds4f(tile + (t + i) * PITCH + (col0 + c) * 4);
    return r;
  }
  struct Quad {
    f32x4 w;
  };
  static constexpr bool kTransposed = false;  // as it is: 4 rows of one column
  static __device__ __forceinline__ Quad quad(const f32x4 v, int) { return Quad{v}; }
  template <int N>
  static __device__ __forceinline__ f32x4 mma_te(const Terms<N>& a, const Exact& b, f32x4 c) {
    return mma(a.t, b, c);
  }
  static __device__ __forceinline__ void image_floats(const lds_u8* f, int lane, float (&v)[8]) {
    floats(load_frag(f, lane), v);
  }
  template <int N>
  static __device__ __forceinline__ void store_terms(lds_u8* f, int lane, const Terms<N>& t) {
    store_frag(f, lane, t.t);
  }
  template <int N>
  static __device__ __forceinline__ void put4(uint8_t* f, int g, int c, int half, const f32x4 v) {
    *reinterpret_cast<f32x4*>(f + half * 1024 + (g * 16 + c) * 16) = v;
  }
};

// A record: T's fragments (kTerms copies of each kFrag apart), P's, then per step e^G, e^{G_63 -
// G}, beta and 1 for steps before L (else 0). The backward pass takes G itself too, as a sum of two
// floats.
template <class P, bool BWD>
struct Record {
  static constexpr int kT = 0;
  static constexpr int kTBlock = P::kTerms * P::kFrag;
  static constexpr int kP = kTBlocks * kTBlock;
  static constexpr int kPBlock = kTBlock;
  static constexpr int kRows = kP + kTBlocks * kPBlock;
  static constexpr int kGrow = 0, kDecay = kC * 4, kBeta = 2 * kC * 4, kOn = 3 * kC * 4;
  static constexpr int kGhi = 4 * kC * 4, kGlo = 5 * kC * 4;
  static constexpr int kRowBytes = (BWD ? 8 : 4) * kC * 4;
  static constexpr int kBytes = kRows + kRowBytes;
  static_assert(kP % 1024 == 0 && kRows % 1024 == 0 && kBytes % 1024 == 0,
                "a record is copied in units of 1 KB");
};

// What the backward pass keeps of a chunk and 32 columns of v: the state before the chunk and U
// (dS after it and dR, in the second of two such images), in fragments whose rows are the columns
// of v: the fragment (tile, kk) holds at lane (g, c) the entries [32 kk + 8g .. +8) of column 16
// tile + c, as a scan wavefront has them, in 2 KB: fp32, or two bf16 terms where the caller chose 16
// bits. One term (8 bits) would not do even there: dg is a sum of such products of either sign (one
// step of one state of one entry: 6.9e-3 off).
template <class P, int KK>
struct Image {
  static constexpr int kFrag = 2048;
  static constexpr int kS = 0;
  static constexpr int kU = 2 * KK * kFrag;
  static constexpr int kBytes = kU + 4 * kFrag;
};

// A state in accumulator layout from or to memory, (dv, dk) rows of `dk`: this lane's column.
template <int KK>
__device__ __forceinline__ void load_state(const float* col, int dk, bool vec, int g, f32x4 (&S)[2 * KK]) {
#pragma unroll
  for (int a = 0; a < 2 * KK; ++a) {
    const int r = tile_row4(a, g);
    if (r >= dk) continue;
    if (vec) {
      S[a] = *reinterpret_cast<const f32x4*>(col + r);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i < dk) S[a][i] = col[r + i];
    }
  }
}
template <int KK>
__device__ __forceinline__ void store_state(float* col, int dk, bool vec, int g, const f32x4 (&S)[2 * KK]) {
#pragma unroll
  for (int a = 0; a < 2 * KK; ++a) {
    const int r = tile_row4(a, g);
    if (r >= dk) continue;
    if (vec) {
      *reinterpret_cast<f32x4*>(col + r) = S[a];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i < dk) col[r + i] = S[a][i];
    }
  }
}

// Buffers of a scan's LDS: two of the operands where they have room beside two tiles of columns, or
// beside one; else one of each.
struct Buffers {
  int n, tiles;
};
constexpr Buffers buffers(int bytes, int tile) {
  constexpr int kLds = 160 * 1024;
  return 2 * (bytes + tile) <= kLds ? Buffers{2, 2} : 2 * bytes + tile <= kLds ? Buffers{2, 1} : Buffers{1, 1};
}

// Brings the shared operands of a chunk into LDS by direct loads: NMAT matrices of 4 KK fragments
// (rows of `dk` = 32 KK entries), a row-major tile of 16 NW columns, both from rows of any stride,
// and a run of 1 KB units. Addresses are a wave-uniform base, moved by whole chunks, and 32-bit
// offsets a lane, made once; rows past the end of the sequence (of the last chunk) read its last
// one.
template <class P, int KK, int NW, int NMAT>
struct Mover {
  typedef typename P::IO IO;
  static constexpr int kPer = P::kFrag / 1024;                      // units of a fragment
  static constexpr int kFragUnits = NMAT * 4 * KK * kPer;
  static constexpr int kFragSteps = (kFragUnits + NW - 1) / NW;     // a wavefront's share
  static constexpr int kPitch = 16 * NW * (int)sizeof(IO);          // bytes of a row of the tile
  static constexpr int kTileBytes = kC * kPitch;
  static constexpr int kTileSteps = kTileBytes / 1024 / NW;
  uint32_t frag[kFragSteps], tile[kTileSteps];
  // rows: how many of the 64 there are; st: row strides in elements of each matrix and of the
  // tile's source; cols: columns there are from the tile's first on
  __device__ __forceinline__ void place(int w, int lane, int rows, const int64_t (&st)[2],
                                        int64_t tile_st, int64_t cols) {
    const int g = lane >> 4, c = lane & 15;
#pragma unroll
    for (int i = 0; i < kFragSteps; ++i) {
      const int u = w + i * NW, half = u % kPer, f = u / kPer, fb = f % (4 * KK);
      const int t = min(tile_row(fb / KK, c), rows - 1);
      frag[i] = (uint32_t)((t * st[f / (4 * KK) & (NMAT - 1)] + 32 * (fb % KK) + 8 * g + 4 * half) * sizeof(IO));
    }
    constexpr int kLanes = kPitch / 16, kV = 16 / (int)sizeof(IO);  // lanes to a row of the tile
#pragma unroll
    for (int i = 0; i < kTileSteps; ++i) {
      const int r = (w + i * NW) * (64 / kLanes) + lane / kLanes, t = min(r, rows - 1);
      int64_t col = ((lane % kLanes) ^ P::template tile_swizzle<kPitch>(r)) * kV;
      if (col >= cols) col = cols - kV;
      tile[i] = (uint32_t)((t * tile_st + col) * sizeof(IO));
    }
  }
  __device__ __forceinline__ void frag_step(int i, int w, const IO* a, const IO* b, lds_u8* to) const {
    const int u = w + i * NW;
    if (kFragUnits % NW == 0 || u < kFragUnits)
      dma16(NMAT == 2 && u / kPer >= 4 * KK ? b : a, frag[i], (uint32_t)(uintptr_t)(to + u * 1024));
  }
  __device__ __forceinline__ void row_step(int i, int w, const IO* src, lds_u8* to) const {
    dma16(src, tile[i], (uint32_t)(uintptr_t)(to + (w + i * NW) * 1024));
  }
  // UNITS consecutive ones
  template <int UNITS>
  static __device__ __forceinline__ void run_step(int i, int w, int lane, const uint8_t* src, lds_u8* to) {
    const int u = w + i * NW;
    if (UNITS % NW == 0 || u < UNITS)
      dma16(src, (uint32_t)(u * 1024 + lane * 16), (uint32_t)(uintptr_t)(to + u * 1024));
  }
  template <int UNITS>
  static __device__ __forceinline__ void run(int w, int lane, const uint8_t* src, lds_u8* to) {
#pragma unroll
    for (int i = 0; i < (UNITS + NW - 1) / NW; ++i) run_step<UNITS>(i, w, lane, src, to);
  }
};

// A wavefront's 64 x 16 results, four accumulator tiles, as they are stored by rows of the output:
// `base` is the chunk's first row, `st` its row stride in elements.
template <class P>
struct RowStore {
  typedef typename P::IO IO;
  typename P::Quad v[4];
  __device__ __forceinline__ void take(const f32x4 (&y)[4], int c) {
#pragma unroll
    for (int a = 0; a < 4; ++a) v[a] = P::quad(y[a], c);
  }
  // rows: how many there are; col0: the wavefront's first column, cols: one past the last there is;
  // vec: four columns at once
  __device__ __forceinline__ void store(IO* base, int64_t st, int rows, int64_t col0, int64_t cols,
                                        bool vec, int lane) const {
    const int g = lane >> 4, c = lane & 15;
    if constexpr (P::kTransposed) {
      const int64_t col = col0 + 4 * (c >> 2);
      if (col >= cols) return;
      const int r0 = 8 * g + (c & 3);
      const int64_t off = r0 * st + col;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int r = 32 * (a >> 1) + 4 * (a & 1);
        IO* row = base + r * st + off;
        if (r0 + r >= rows) continue;
        if (vec) {
          *reinterpret_cast<u32x2*>(row) = v[a].w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < cols) row[e] = (IO)(v[a].w[e >> 1] >> (16 * (e & 1)));
        }
      }
    } else {
      const int64_t col = col0 + c;
      if (col >= cols) return;
      const int64_t off = 8 * g * st + col;
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 32 * (a >> 1) + 4 * (a & 1) + i;
          if (8 * g + r < rows) base[r * st + off] = v[a].w[i];
        }
    }
  }
};

// Work items (batch, head, slice) are taken so that an accelerator die, to which workgroups go
// round robin, gets a contiguous range of them: the heads of a group share q and k in its L2.
__device__ __forceinline__ int64_t die_item(int64_t i, int64_t n) {
  return n % 8 == 0 ? (i & 7) * (n >> 3) + (i >> 3) : i;
}

}  // namespace delta
}  // namespace ssm
