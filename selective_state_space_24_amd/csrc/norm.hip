// gfx950 kernels of layer norm, forward and backward.
//
//   y = (x - mean) rstd w + b
//   dx = rstd (w dy - m1 - xh m2),  m1 = mean(w dy), m2 = mean(w dy xh), xh = (x - mean) rstd
//   dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by HBM: the forward pass reads x and writes y, the backward pass reads x and dy and
// writes dx. A row is held in registers by a team of W wavefronts, V N entries a lane, so it is
// read once, and its variance is taken about its mean (no difference of large sums). Above 8192
// entries the backward pass's partial sums do not fit beside the row (sixteen wavefronts, 128 registers
// a lane) and go through scratch memory: 8192 x 16384 takes 365 us in bf16 (2.2 TB/s; 8192 x 8192 89 us,
// 4.5 TB/s) and 653 us in fp32, by single entries 1.03 and 0.96 ms. Rows without 16-byte access are
// otherwise a little slower: 32768 x 4096 in bf16 off by one entry 140 us forward and 167 backward, 99
// and 162 aligned. A team takes
// rows in turn, the next one's loads in flight while it works on this one, and keeps weight and
// bias (and the partial sums of dw and db) in registers across its rows. The backward pass writes
// one row of partial sums per workgroup; a second kernel adds those, in a fixed order.
#include "norm_internal.h"
#include "scan_internal.h"
#include "scan_kernels.h"

namespace ssm {
namespace {

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp0(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROW_MASK, 0xf, false));
}
// sum over the 64 lanes, in every lane
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp0<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8: lane 15 of each row has the row's sum
  v += dpp0<0x112, 0xf>(v);
  v += dpp0<0x114, 0xf>(v);
  v += dpp0<0x118, 0xf>(v);
  v += dpp0<0x142, 0xa>(v);  // row_bcast 15, 31
  v += dpp0<0x143, 0xc>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// V consecutive io elements as they are stored
template <typename IO, int V>
struct Raw {
  u32x4 w;
};
template <typename IO>
struct Raw<IO, 1> {
  IO w;
};

template <typename IO, int V>
__device__ __forceinline__ void get(const Raw<IO, V>& r, float (&f)[V]) {
  if constexpr (V == 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(r.w[k] << 16);
      f[2 * k + 1] = __uint_as_float(r.w[k] & 0xffff0000u);
    }
  } else if constexpr (V == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(r.w[k]);
  } else {
    f[0] = to_f32(r.w);
  }
}
template <typename IO, int V>
__device__ __forceinline__ void put(IO* p, const float (&f)[V]) {
  if constexpr (V == 8) {
    *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                         pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
  } else if constexpr (V == 4) {
    *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
  } else {
    store_elem(p, f[0]);
  }
}

constexpr int threads(int W) { return W <= 4 ? 256 : 64 * W; }
constexpr int teams(int W) { return W <= 4 ? 4 / W : 1; }

// The lane's place: entries (64 W k + at) V .. +V for k < N.
template <int W>
struct Team {
  int at;    // lane number in the team
  int team;  // in the workgroup
  int wave;  // in the team
};
template <int W>
__device__ __forceinline__ Team<W> my_team() {
  const int t = threadIdx.x;
  return Team<W>{t % (64 * W), t / (64 * W), (t >> 6) % W};
}

// Sums of a and b over a team. `slot` alternates between calls, so that one barrier a call is
// enough (every team of the workgroup makes the same calls).
template <int W>
__device__ __forceinline__ void team_sum2(float& a, float& b, float* lds, int slot, const Team<W>& t) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (W > 1) {
    float* s = lds + (slot * teams(W) + t.team) * 2 * W;
    if ((threadIdx.x & 63) == 0) {
      s[t.wave] = a;
      s[W + t.wave] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      a += s[i];
      b += s[W + i];
    }
  }
}

template <typename IO, int V, int N, int W>
__device__ __forceinline__ void load_row(const IO* row, const Team<W>& t, int64_t cols, Raw<IO, V> (&r)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int64_t c = (int64_t)(64 * W * k + t.at) * V;
    r[k] = {};
    if (c < cols) {
      if constexpr (V == 1) r[k].w = row[c];
      else r[k].w = *reinterpret_cast<const u32x4*>(row + c);
    }
  }
}

template <typename IO, int V, int N, int W>
__global__ void __launch_bounds__(threads(W)) norm_fwd_kernel(const NormParams p) {
  __shared__ float lds[2 * teams(W) * 2 * W];
  const Team<W> t = my_team<W>();
  const int64_t step = (int64_t)gridDim.x * teams(W);
  const int64_t cols = p.cols;
  const IO* X = static_cast<const IO*>(p.x);
  int64_t row = (int64_t)blockIdx.x * teams(W) + t.team;
  Raw<IO, V> nx[N];
  load_row<IO, V, N, W>(X + (row < p.rows ? row : p.rows - 1) * p.x_st, t, cols, nx);
  float w[N][V], bi[N][V];
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int64_t c = (int64_t)(64 * W * k + t.at) * V + e;
      w[k][e] = c < cols && p.weight ? p.weight[c] : 1.0f;
      bi[k][e] = c < cols && p.bias ? p.bias[c] : 0.0f;
    }
  const float inv = 1.0f / (float)cols;
  // every team of the workgroup goes round as often as the first
  for (int64_t r0 = (int64_t)blockIdx.x * teams(W); r0 < p.rows; r0 += step, row += step) {
    float x[N][V];
#pragma unroll
    for (int k = 0; k < N; ++k) get<IO, V>(nx[k], x[k]);
    const int64_t next = row + step;
    if (r0 + step < p.rows)
      load_row<IO, V, N, W>(X + (next < p.rows ? next : p.rows - 1) * p.x_st, t, cols, nx);
    float s = 0.0f, z = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) s += x[k][e];  // entries past the row are zeros
    team_sum2<W>(s, z, lds, 0, t);
    const float mean = s * inv;
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int64_t c = (int64_t)(64 * W * k + t.at) * V;
        x[k][e] -= mean;
        q += c < cols ? x[k][e] * x[k][e] : 0.0f;
      }
    z = 0.0f;
    team_sum2<W>(q, z, lds, 1, t);
    const float rstd = 1.0f / sqrtf(q * inv + p.eps);
    if (row < p.rows) {
      IO* y = static_cast<IO*>(p.y) + row * p.y_st;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t c = (int64_t)(64 * W * k + t.at) * V;
        if (c < cols) {
          float o[V];
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = fmaf(x[k][e] * rstd, w[k][e], bi[k][e]);
          put<IO, V>(y + c, o);
        }
      }
      if (t.at == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
      }
    }
  }
}

template <typename IO, int V, int N, int W>
__global__ void __launch_bounds__(threads(W)) norm_bwd_kernel(const NormParams p) {
  constexpr int kTeams = teams(W);
  __shared__ float lds[2 * kTeams * 2 * W];
  __shared__ float sums[kTeams > 1 ? (kTeams - 1) * 64 * W * V * N : 1];
  const Team<W> t = my_team<W>();
  const int64_t step = (int64_t)gridDim.x * kTeams;
  const int64_t cols = p.cols;
  const IO* X = static_cast<const IO*>(p.x);
  const IO* DY = static_cast<const IO*>(p.dy);
  int64_t row = (int64_t)blockIdx.x * kTeams + t.team;
  Raw<IO, V> nx[N], nd[N];
  float nm, nr;
  auto load = [&](int64_t r) {
    if (r >= p.rows) r = p.rows - 1;
    load_row<IO, V, N, W>(X + r * p.x_st, t, cols, nx);
    load_row<IO, V, N, W>(DY + r * p.y_st, t, cols, nd);
    nm = p.mean_in[r];
    nr = p.rstd_in[r];
  };
  load(row);
  float w[N][V], dw[N][V], db[N][V];
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int64_t c = (int64_t)(64 * W * k + t.at) * V + e;
      w[k][e] = c < cols && p.weight ? p.weight[c] : 1.0f;
      dw[k][e] = db[k][e] = 0.0f;
    }
  const float inv = 1.0f / (float)cols;
  int slot = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * kTeams; r0 < p.rows; r0 += step, row += step, slot ^= 1) {
    const bool on = row < p.rows;
    const float mean = nm, rstd = nr;
    float xh[N][V], d[N][V];
    float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      get<IO, V>(nx[k], xh[k]);
      get<IO, V>(nd[k], d[k]);
    }
    if (r0 + step < p.rows) load(row + step);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        xh[k][e] = (xh[k][e] - mean) * rstd;
        // dy of entries past the row is zero
        dw[k][e] = on ? fmaf(d[k][e], xh[k][e], dw[k][e]) : dw[k][e];
        db[k][e] += on ? d[k][e] : 0.0f;
        d[k][e] *= w[k][e];
        m1 += d[k][e];
        m2 = fmaf(d[k][e], xh[k][e], m2);
      }
    team_sum2<W>(m1, m2, lds, slot, t);
    m1 *= inv;
    m2 *= inv;
    if (on) {
      IO* dx = static_cast<IO*>(p.dx) + row * p.dx_st;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int64_t c = (int64_t)(64 * W * k + t.at) * V;
        if (c < cols) {
          float o[V];
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = rstd * (d[k][e] - m1 - xh[k][e] * m2);
          put<IO, V>(dx + c, o);
        }
      }
    }
  }
  // the workgroup's sums: the first team adds what the others leave in LDS
  auto finish = [&](float (&v)[N][V], float* out) {
    if constexpr (kTeams > 1) {
      __syncthreads();
      if (t.team > 0) {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e)
            sums[((t.team - 1) * N * V + k * V + e) * 64 * W + t.at] = v[k][e];
      }
      __syncthreads();
      if (t.team > 0) return;
#pragma unroll
      for (int i = 0; i < kTeams - 1; ++i)
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) v[k][e] += sums[(i * N * V + k * V + e) * 64 * W + t.at];
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int64_t c = (int64_t)(64 * W * k + t.at) * V + e;
        if (c < cols) out[(int64_t)blockIdx.x * cols + c] = v[k][e];
      }
  };
  if (p.dweight) finish(dw, p.part);
  if (p.dbias) finish(db, p.part + p.groups * cols);
}

// dw and db from the partial sums: 64 columns a workgroup, 16 wavefronts that each add every
// sixteenth row of them
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const NormParams p) {
  __shared__ float s[16][64];
  float* out = blockIdx.y ? p.dbias : p.dweight;
  if (!out) return;
  const float* part = p.part + (int64_t)blockIdx.y * p.groups * p.cols;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float a = 0.0f;
  if (c < p.cols) {
    int64_t r = w;
    for (; r + 7 * 16 < p.groups; r += 8 * 16) {  // eight loads in flight
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = part[(r + 16 * i) * p.cols + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) a += v[i];
    }
    for (; r < p.groups; r += 16) a += part[r * p.cols + c];
  }
  s[w][lane] = a;
  __syncthreads();
  if (w == 0 && c < p.cols) {
    a = s[0][lane];
#pragma unroll
    for (int i = 1; i < 16; ++i) a += s[i][lane];
    out[c] = a;
  }
}

constexpr int kMostWaves = 16;
// Wavefronts to a row: the fewest that hold it at `per` entries a lane: two vectors, so that a row
// is in flight on more lanes (forward, 512 x 2048 bf16: 7.0 us at two, 10.4 at four; 32768 x 4096 99
// and 109), four where sixteen wavefronts do not hold it at two.
int team_width(int64_t cols, int per) {
  int w = 1;
  while ((int64_t)64 * w * per < cols) w *= 2;
  return w;
}

// Workgroups that go round over the rows: one to a CU, two of 256 threads where a team then still
// has `many` rows (32768 x 4096 bf16 forward: 143 us at one, 99 at two; 32768 x 4096 fp32 backward,
// 512 threads: 288 at one, 313 at two).
int64_t team_groups(int64_t rows, int W, int64_t least_rows, int64_t many) {
  const int64_t want = (rows + teams(W) * least_rows - 1) / (teams(W) * least_rows);
  if (want <= kCUs) return want;
  const int64_t two = threads(W) > 256 ? 0 : rows / (teams(W) * many);
  return two < kCUs ? kCUs : (two < 2 * kCUs ? two : 2 * kCUs);
}
// Rows a team takes at least in the backward pass, each of whose workgroups leaves a row of partial
// sums (both kernels, 512 x 2048 bf16: 11.5 us at two rows, 13.6 at four; 4096 x 2048: 20.9 us at one
// workgroup to a CU, 23.2 at two).
constexpr int64_t kLeastRows = 2, kManyRows = 16;

template <typename IO, int V, int N, int W, bool BWD>
hipError_t go(const NormParams& p, hipStream_t stream) {
  if constexpr (BWD) {
    norm_bwd_kernel<IO, V, N, W><<<dim3((unsigned)p.groups), threads(W), 0, stream>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!p.dweight && !p.dbias)) return e;
    norm_bwd_sum_kernel<<<dim3((unsigned)((p.cols + 63) / 64), 2), 1024, 0, stream>>>(p);
  } else {
    norm_fwd_kernel<IO, V, N, W><<<dim3((unsigned)team_groups(p.rows, W, 1, 1)), threads(W), 0, stream>>>(p);
  }
  return hipGetLastError();
}

template <typename IO, int V, int N, bool BWD>
hipError_t wide(const NormParams& p, hipStream_t stream) {
  switch (team_width(p.cols, V * N)) {
    case 1: return go<IO, V, N, 1, BWD>(p, stream);
    case 2: return go<IO, V, N, 2, BWD>(p, stream);
    case 4: return go<IO, V, N, 4, BWD>(p, stream);
    case 8: return go<IO, V, N, 8, BWD>(p, stream);
    default: return go<IO, V, N, kMostWaves, BWD>(p, stream);
  }
}

constexpr int kScalarPer = 16;  // entries a lane without vector access
static_assert(64 * kMostWaves * kScalarPer >= kNormMaxCols, "");
// Entries that two vectors a lane, or four, cover.
constexpr int64_t vec_cols(int V, int N) { return (int64_t)64 * kMostWaves * V * N; }
static_assert(vec_cols(IoTraits<float>::kVec, 4) >= kNormMaxCols, "");
int vec_width(int64_t cols, int V) { return cols <= vec_cols(V, 2) ? team_width(cols, 2 * V) : kMostWaves; }

template <typename IO, bool BWD>
hipError_t dispatch(const NormParams& p, hipStream_t stream) {
  constexpr int V = IoTraits<IO>::kVec;
  if (!p.vec) return wide<IO, 1, kScalarPer, BWD>(p, stream);
  if (p.cols <= 64 * V) return go<IO, V, 1, 1, BWD>(p, stream);
  if constexpr (vec_cols(V, 2) < kNormMaxCols) {
    if (p.cols > vec_cols(V, 2)) return go<IO, V, 4, kMostWaves, BWD>(p, stream);
  }
  return wide<IO, V, 2, BWD>(p, stream);
}

}  // namespace

int64_t norm_bwd_groups(int64_t rows, int64_t cols, bool bf16, bool vec) {
  const int V = bf16 ? IoTraits<bf16_bits>::kVec : IoTraits<float>::kVec;
  return team_groups(rows, vec ? vec_width(cols, V) : team_width(cols, kScalarPer), kLeastRows, kManyRows);
}

hipError_t launch_norm_fwd(const NormParams& p, hipStream_t stream) {
  return p.bf16 ? dispatch<bf16_bits, false>(p, stream) : dispatch<float, false>(p, stream);
}
hipError_t launch_norm_bwd(const NormParams& p, hipStream_t stream) {
  return p.bf16 ? dispatch<bf16_bits, true>(p, stream) : dispatch<float, true>(p, stream);
}

}  // namespace ssm
