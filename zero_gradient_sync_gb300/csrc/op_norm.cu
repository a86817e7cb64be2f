// The norms around a block, fused with its gate and residual scale, and their gradient.
//
//   r = a x + b g N_post(y),   z = N_pre(r),   N(v) = (v - mean) rstd w + c
//
// Apart, these are two norms, a product and a scaled sum: x, y, r and the post norm's output go through memory several
// times.  Here a row stays in registers from y to z: x and y are read once, r and z written once (four row passes
// forward; six backward: dr, dz, r, y in, dx, dy out).  What bounds both is memory.
//
// A row is held by a group of threads, eight consecutive elements each (or one element every group-width where rows are
// not 16-byte aligned), NV such pieces a thread.  A group is one warp for short rows, else the whole CTA; CTAs are
// persistent, so parameters are read once per CTA and held in registers, and the next row's loads are issued before the
// current row's sums.  Mean and variance are taken in two passes over the registers: no cancellation.
//
// Gradient, with yh, rh the rows before weights and biases, D = dr + N_pre'(dz) and q = g D for a gate per token, else D:
//   v  = w_pre dz:      D  = dr + rstd_pre (v - rh mean(v rh) - mean(v))          (RMS: without mean(v))
//   v' = b g w_post D:  dy = rstd_post (v' - yh mean(v' yh) - mean(v')),   dx = a D
//   P1 = sum dz rh, P0 = sum dz, S1 = sum q yh, S0 = sum q   over the rows, for each column
//   dw_pre = P1, db_pre = P0, dw_post = b g S1, db_post = b g S0, dgate = b (w_post S1 + c_post S0) for a gate per
//   channel; for one per token, dgate = b (sum over the row of D (w_post yh + c_post)).
// So all five parameter gradients come from four column sums (two for RMS norms without biases), kept in registers over
// the rows of a CTA, left in the workspace as one partial row a CTA, and added in CTA order by a second kernel.
#include <math.h>

#include <initializer_list>

#include "op_common.cuh"

namespace dp {
namespace {

constexpr int NORM_THREADS = 512;   // most threads of a group
constexpr int MAX_PARTS = 1024;     // most CTAs (partial rows) of the gradient
constexpr int FIN_COLS = 32, FIN_ROWS = 16;

struct NormParams {
  void *r, *z, *dx, *dy, *dgate_token;
  const void *x, *y, *dr, *dz;
  const void *w_post, *b_post, *gate, *w_pre, *b_pre;
  float2 *post_stats, *pre_stats;
  float* part;
  int64_t rows;
  int dim, group, per_cta;  // threads of a row, rows of a CTA at a time
  int layer, post, pre, gate_mode, pdt, accumulate;
  float eps, a, b;
};

// The element numbers of a thread: piece j, k-th of eight.
template <int VEC>
__device__ __forceinline__ int col_of(int tid, int group, int j, int k) {
  return VEC ? (tid + j * group) * 8 + k : tid + (j * 8 + k) * group;
}

template <typename T, int VEC, int NV>
struct RowRegs {
  Raw8<T> w[NV];
  __device__ __forceinline__ void load(const T* row, int tid, int group, int dim) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (VEC) {
        const int c = col_of<1>(tid, group, j, 0);
        if (c < dim) w[j] = load_raw8(row + c);
        else {
          const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          w[j].pack(zero);
        }
      } else {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int c = col_of<0>(tid, group, j, k);
          v[k] = c < dim ? Elem<T>::get(row[c]) : 0.0f;
        }
        w[j].pack(v);
      }
    }
  }
};

template <typename T, int VEC, int NV>
__device__ __forceinline__ void store_row(T* row, int tid, int group, int dim, const float (&v)[NV][8]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (VEC) {
      const int c = col_of<1>(tid, group, j, 0);
      if (c < dim) {
        Raw8<T> o;
        o.pack(v[j]);
        store_raw8(row + c, o);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = col_of<0>(tid, group, j, k);
        if (c < dim) row[c] = Elem<T>::put(v[j][k]);
      }
    }
  }
}

template <int VEC, int NV>
__device__ __forceinline__ void load_param(const void* p, int dtype, float none, int tid, int group, int dim,
                                           float (&v)[NV][8]) {
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = col_of<VEC>(tid, group, j, k);
      v[j][k] = c < dim ? param_at(p, c, dtype, none) : 0.0f;
    }
}

// Sums of N values over a group of threads; every thread gets them.  A CTA-wide group alternates between two halves of
// `buf`, so one barrier a call is enough: a half is written again only after the barrier of the call in between.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int warps, float (*buf)[32][4], int& half) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[half][warp][i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = lane < warps ? buf[half][lane][i] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  }
  half ^= 1;
}

// Mean (0 for RMS) and 1 / sqrt(var + eps) of a row held in registers.  Pieces beyond dim hold zeros.
template <int VEC, int NV>
__device__ __forceinline__ float2 row_stats(const float (&v)[NV][8], int layer, float eps, int tid, int group, int dim,
                                            float (*buf)[32][4], int& half) {
  float mean = 0.0f, s[1];
  if (layer) {
    s[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[0] += v[j][k];
    group_sum<1>(s, group >> 5, buf, half);
    mean = s[0] / (float)dim;
  }
  s[0] = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = col_of<VEC>(tid, group, j, k) < dim ? v[j][k] - mean : 0.0f;
      s[0] = fmaf(d, d, s[0]);
    }
  group_sum<1>(s, group >> 5, buf, half);
  return make_float2(mean, 1.0f / sqrtf(s[0] / (float)dim + eps));
}

// Which row a group of threads starts with, and the step between its rows.
__device__ __forceinline__ int64_t first_row(const NormParams& P, int& tid) {
  if (P.per_cta == 1) {
    tid = threadIdx.x;
    return blockIdx.x;
  }
  tid = threadIdx.x & 31;
  return (int64_t)blockIdx.x * P.per_cta + (threadIdx.x >> 5);
}

template <typename TS, typename TB, int VEC, int NV>
__global__ void __launch_bounds__(NORM_THREADS) norm_kernel(const __grid_constant__ NormParams P) {
  __shared__ float buf[2][32][4];
  int half = 0, tid;
  const int64_t row0 = first_row(P, tid), step = (int64_t)gridDim.x * P.per_cta;
  const int group = P.group, dim = P.dim;
  float A[NV][8], B[NV][8], wp[NV][8], bp[NV][8];  // b g w_post, b g b_post, w_pre, b_pre
  if (P.y) {
    load_param<VEC, NV>(P.w_post, P.pdt, 1.0f, tid, group, dim, A);
    load_param<VEC, NV>(P.b_post, P.pdt, 0.0f, tid, group, dim, B);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = col_of<VEC>(tid, group, j, k);
        const float g = P.gate_mode == DP_GATE_CHANNEL && c < dim ? P.b * param_at(P.gate, c, P.pdt, 1.0f) : P.b;
        A[j][k] *= g;
        B[j][k] *= g;
      }
  }
  if (P.pre) {
    load_param<VEC, NV>(P.w_pre, P.pdt, 1.0f, tid, group, dim, wp);
    load_param<VEC, NV>(P.b_pre, P.pdt, 0.0f, tid, group, dim, bp);
  }
  for (int64_t row = row0; row < P.rows; row += step) {
    RowRegs<TS, VEC, NV> xr;
    xr.load(static_cast<const TS*>(P.x) + row * dim, tid, group, dim);
    float r[NV][8];
    if (P.y) {
      RowRegs<TB, VEC, NV> yr;
      yr.load(static_cast<const TB*>(P.y) + row * dim, tid, group, dim);
      float v[NV][8];
#pragma unroll
      for (int j = 0; j < NV; ++j) yr.w[j].unpack(v[j]);
      float2 st = make_float2(0.0f, 1.0f);
      if (P.post) {
        st = row_stats<VEC, NV>(v, P.layer, P.eps, tid, group, dim, buf, half);
        if (P.post_stats && tid == 0) P.post_stats[row] = st;
      }
      const float gt = P.gate_mode == DP_GATE_TOKEN ? param_at(P.gate, row, P.pdt, 1.0f) : 1.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        xr.w[j].unpack(r[j]);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          r[j][k] = fmaf(P.a, r[j][k], gt * fmaf((v[j][k] - st.x) * st.y, A[j][k], B[j][k]));
      }
      store_row<TS, VEC, NV>(static_cast<TS*>(P.r) + row * dim, tid, group, dim, r);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) xr.w[j].unpack(r[j]);
    }
    if (P.pre) {
      const float2 st = row_stats<VEC, NV>(r, P.layer, P.eps, tid, group, dim, buf, half);
      if (P.pre_stats && tid == 0) P.pre_stats[row] = st;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) r[j][k] = fmaf((r[j][k] - st.x) * st.y, wp[j][k], bp[j][k]);
      store_row<TB, VEC, NV>(static_cast<TB*>(P.z) + row * dim, tid, group, dim, r);
    }
  }
}

// LAYER: rows are centred.  SUM0: some gradient needs S0 or P0 (a bias is there).  The workspace holds, for each group of
// threads, S1 and P1 and (SUM0) S0 and P0, dim floats each.
template <typename TS, typename TB, int VEC, int NV, bool LAYER, bool SUM0>
__global__ void __launch_bounds__(NORM_THREADS) norm_grad_kernel(const __grid_constant__ NormParams P) {
  __shared__ float buf[2][32][4];
  int half = 0, tid;
  const int64_t row0 = first_row(P, tid), step = (int64_t)gridDim.x * P.per_cta;
  const int group = P.group, dim = P.dim;
  const bool has_y = P.y != nullptr, token = P.gate_mode == DP_GATE_TOKEN;
  float A[NV][8], wp[NV][8];  // b g w_post, w_pre
  float S1[NV][8], P1[NV][8], S0[NV][8], P0[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) S1[j][k] = P1[j][k] = S0[j][k] = P0[j][k] = 0.0f;
  if (has_y) {
    load_param<VEC, NV>(P.w_post, P.pdt, 1.0f, tid, group, dim, A);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = col_of<VEC>(tid, group, j, k);
        A[j][k] *= P.gate_mode == DP_GATE_CHANNEL && c < dim ? P.b * param_at(P.gate, c, P.pdt, 1.0f) : P.b;
      }
  }
  if (P.pre) load_param<VEC, NV>(P.w_pre, P.pdt, 1.0f, tid, group, dim, wp);
  const float inv = 1.0f / (float)dim;

  for (int64_t row = row0; row < P.rows; row += step) {
    float D[NV][8];
    RowRegs<TB, VEC, NV> yr;
    if (has_y) yr.load(static_cast<const TB*>(P.y) + row * dim, tid, group, dim);
    if (P.dr) {
      RowRegs<TS, VEC, NV> w;
      w.load(static_cast<const TS*>(P.dr) + row * dim, tid, group, dim);
#pragma unroll
      for (int j = 0; j < NV; ++j) w.w[j].unpack(D[j]);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) D[j][k] = 0.0f;
    }
    if (P.pre) {
      RowRegs<TB, VEC, NV> zr;
      RowRegs<TS, VEC, NV> rr;
      zr.load(static_cast<const TB*>(P.dz) + row * dim, tid, group, dim);
      rr.load(static_cast<const TS*>(P.x) + row * dim, tid, group, dim);
      const float2 st = P.pre_stats[row];
      float v[NV][8], h[NV][8], s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        zr.w[j].unpack(v[j]);
        rr.w[j].unpack(h[j]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          h[j][k] = (h[j][k] - st.x) * st.y;
          P1[j][k] = fmaf(v[j][k], h[j][k], P1[j][k]);
          if (SUM0) P0[j][k] += v[j][k];
          v[j][k] *= wp[j][k];  // zero beyond dim
          s[0] = fmaf(v[j][k], h[j][k], s[0]);
          if (LAYER) s[1] += v[j][k];
        }
      }
      if (LAYER) group_sum<2>(s, group >> 5, buf, half);
      else {
        float one[1] = {s[0]};
        group_sum<1>(one, group >> 5, buf, half);
        s[0] = one[0];
      }
      const float c1 = s[0] * inv, c0 = LAYER ? s[1] * inv : 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) D[j][k] = fmaf(st.y, fmaf(-h[j][k], c1, v[j][k]) - c0, D[j][k]);
    }
    if (has_y) {
      const float2 st = P.post ? P.post_stats[row] : make_float2(0.0f, 1.0f);
      const float gt = token ? param_at(P.gate, row, P.pdt, 1.0f) : 1.0f;
      float h[NV][8], s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        yr.w[j].unpack(h[j]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int c = col_of<VEC>(tid, group, j, k);
          h[j][k] = (h[j][k] - st.x) * st.y;
          const float q = gt * D[j][k], v = A[j][k] * D[j][k];
          S1[j][k] = fmaf(q, h[j][k], S1[j][k]);
          if (SUM0) S0[j][k] += q;
          s[0] = fmaf(v, h[j][k], s[0]);
          if (LAYER) s[1] += v;
          if (token && P.b_post && c < dim) s[2] = fmaf(D[j][k], param_at(P.b_post, c, P.pdt, 0.0f), s[2]);
        }
      }
      if (P.post || token) {
        if (LAYER || token) group_sum<3>(s, group >> 5, buf, half);
        else {
          float one[1] = {s[0]};
          group_sum<1>(one, group >> 5, buf, half);
          s[0] = one[0];
        }
      }
      if (token && P.dgate_token && tid == 0)
        grad_put(P.dgate_token, row, P.pdt, P.accumulate, fmaf(P.b, s[2], s[0]));
      const float c1 = P.post ? s[0] * inv : 0.0f, c0 = P.post && LAYER ? s[1] * inv : 0.0f, f = gt * st.y;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) h[j][k] = f * (fmaf(-h[j][k], c1, A[j][k] * D[j][k]) - c0);
      store_row<TB, VEC, NV>(static_cast<TB*>(P.dy) + row * dim, tid, group, dim, h);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) D[j][k] *= P.a;
    store_row<TS, VEC, NV>(static_cast<TS*>(P.dx) + row * dim, tid, group, dim, D);
  }
  // One partial row a group of threads.
  const int64_t part = (int64_t)blockIdx.x * P.per_cta + (P.per_cta == 1 ? 0 : threadIdx.x >> 5);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = col_of<VEC>(tid, group, j, k);
      if (c < dim) {
        float* p = P.part + part * (SUM0 ? 4 : 2) * dim + c;
        p[0] = S1[j][k];
        p[dim] = P1[j][k];
        if (SUM0) {
          p[2 * (int64_t)dim] = S0[j][k];
          p[3 * (int64_t)dim] = P0[j][k];
        }
      }
    }
}

struct FinishParams {
  const float* part;
  int64_t parts;
  int dim, sum0, gate_mode, pdt, accumulate;
  const void *w_post, *b_post, *gate;
  void *dw_post, *db_post, *dgate, *dw_pre, *db_pre;
  float b;
};

// Adds the partial rows of 32 columns in 16 interleaved parts, then the parts in order.
__global__ void __launch_bounds__(FIN_COLS* FIN_ROWS) norm_finish_kernel(const __grid_constant__ FinishParams P) {
  __shared__ float sums[FIN_ROWS][4][FIN_COLS];
  const int c = blockIdx.x * FIN_COLS + threadIdx.x;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < P.dim) {
#pragma unroll 4
    for (int64_t i = threadIdx.y; i < P.parts; i += FIN_ROWS) {
      const float* p = P.part + i * (P.sum0 ? 4 : 2) * P.dim + c;
      s[0] += p[0];
      s[1] += p[P.dim];
      if (P.sum0) {
        s[2] += p[2 * (int64_t)P.dim];
        s[3] += p[3 * (int64_t)P.dim];
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) sums[threadIdx.y][q][threadIdx.x] = s[q];
  __syncthreads();
  if (threadIdx.y != 0 || c >= P.dim) return;
  for (int y = 1; y < FIN_ROWS; ++y)
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] += sums[y][q][threadIdx.x];
  const float g = P.b * (P.gate_mode == DP_GATE_CHANNEL ? param_at(P.gate, c, P.pdt, 1.0f) : 1.0f);
  if (P.dw_post) grad_put(P.dw_post, c, P.pdt, P.accumulate, g * s[0]);
  if (P.db_post) grad_put(P.db_post, c, P.pdt, P.accumulate, g * s[2]);
  if (P.dgate)
    grad_put(P.dgate, c, P.pdt, P.accumulate,
             P.b * fmaf(param_at(P.w_post, c, P.pdt, 1.0f), s[0], param_at(P.b_post, c, P.pdt, 0.0f) * s[2]));
  if (P.dw_pre) grad_put(P.dw_pre, c, P.pdt, P.accumulate, s[1]);
  if (P.db_pre) grad_put(P.db_pre, c, P.pdt, P.accumulate, s[3]);
}

// ---------------------------------------------------------------------------------------------------- host side

// Pieces of eight a thread holds: one up to 4096 columns, so that a row has as many threads as it can use.
int pieces_of(int dim) { return dim <= NORM_THREADS * 8 ? 1 : dim <= NORM_THREADS * 16 ? 2 : 4; }

struct Shape {
  int nv, group, per_cta, threads;
};
Shape shape_of(int dim) {
  Shape s;
  s.nv = pieces_of(dim);
  s.group = (dim + s.nv * 8 * 32 - 1) / (s.nv * 8 * 32) * 32;
  s.per_cta = s.group == 32 ? 4 : 1;
  s.threads = s.group * s.per_cta;
  return s;
}

template <typename K>
int norm_grid(K kernel, const Shape& s, int64_t rows, int most) {
  const int64_t want = (rows + s.per_cta - 1) / s.per_cta;
  const int g = occupancy_grid(kernel, s.threads, 0, want < most ? (int)want : most);
  return g;
}

template <typename TS, typename TB, int VEC, int NV>
void run_forward(const NormParams& P, const Shape& s, cudaStream_t stream) {
  auto k = norm_kernel<TS, TB, VEC, NV>;
  k<<<norm_grid(k, s, P.rows, INT32_MAX), s.threads, 0, stream>>>(P);
}
template <typename TS, typename TB, int VEC, int NV>
int run_grad(const NormParams& P, const Shape& s, bool sum0, cudaStream_t stream) {
  auto k = P.layer ? norm_grad_kernel<TS, TB, VEC, NV, true, true>
           : sum0  ? norm_grad_kernel<TS, TB, VEC, NV, false, true>
                   : norm_grad_kernel<TS, TB, VEC, NV, false, false>;
  const int grid = norm_grid(k, s, P.rows, MAX_PARTS / s.per_cta);
  k<<<grid, s.threads, 0, stream>>>(P);
  return grid * s.per_cta;
}

// f(stream type, block type, VEC, NV) for the sizes and types of one call.
template <typename F>
auto dispatch(const dp_block_norm_t& p, bool vec, int nv, F&& f) {
#define DP_NV(TS, TB, V) \
  (nv == 1 ? f.template operator()<TS, TB, V, 1>() : nv == 2 ? f.template operator()<TS, TB, V, 2>() \
                                                             : f.template operator()<TS, TB, V, 4>())
#define DP_VEC(TS, TB) (vec ? DP_NV(TS, TB, 1) : DP_NV(TS, TB, 0))
  if (p.stream_dtype == DP_BF16) return DP_VEC(bf16_t, bf16_t);
  if (p.block_dtype == DP_BF16) return DP_VEC(float, bf16_t);
  return DP_VEC(float, float);
#undef DP_VEC
#undef DP_NV
}

struct Forward {
  const NormParams& P;
  const Shape& s;
  cudaStream_t stream;
  template <typename TS, typename TB, int VEC, int NV>
  int operator()() const {
    run_forward<TS, TB, VEC, NV>(P, s, stream);
    return 0;
  }
};
struct Gradient {
  const NormParams& P;
  const Shape& s;
  bool sum0;
  cudaStream_t stream;
  template <typename TS, typename TB, int VEC, int NV>
  int operator()() const {
    return run_grad<TS, TB, VEC, NV>(P, s, sum0, stream);
  }
};

dp_status_t check_norm(const dp_block_norm_t* p, bool has_y, bool gate) {
  if (!p) return op_fail(DP_ERR_INVALID_ARG, "p is NULL");
  if (p->rows < 0 || p->rows > INT32_MAX) return op_fail(DP_ERR_INVALID_ARG, "rows = %lld not in 0..2^31-1", (long long)p->rows);
  if (p->dim < 1 || p->dim > DP_MAX_NORM_DIM) return op_fail(DP_ERR_INVALID_ARG, "dim = %d not in 1..%d", p->dim, DP_MAX_NORM_DIM);
  if (p->kind != DP_NORM_RMS && p->kind != DP_NORM_LAYER) return op_fail(DP_ERR_INVALID_ARG, "kind = %d unknown", p->kind);
  if (p->norms & ~(DP_NORM_POST | DP_NORM_PRE)) return op_fail(DP_ERR_INVALID_ARG, "norms = %d unknown", p->norms);
  if (p->gate_mode < DP_GATE_NONE || p->gate_mode > DP_GATE_TOKEN) return op_fail(DP_ERR_INVALID_ARG, "gate_mode = %d unknown", p->gate_mode);
  DP_TRY(check_dtype(p->stream_dtype, "stream_dtype"));
  DP_TRY(check_dtype(p->block_dtype, "block_dtype"));
  DP_TRY(check_dtype(p->param_dtype, "param_dtype"));
  if (p->stream_dtype == DP_BF16 && p->block_dtype == DP_F32)
    return op_fail(DP_ERR_INVALID_ARG, "fp32 block tensors need an fp32 stream");
  if (p->accumulate != 0 && p->accumulate != 1) return op_fail(DP_ERR_INVALID_ARG, "accumulate = %d is neither 0 nor 1", p->accumulate);
  if (!(p->eps > 0.0f) || !(p->eps < 1e30f)) return op_fail(DP_ERR_INVALID_ARG, "eps must be finite and > 0");
  if (!(fabsf(p->res_scale) < 1e30f) || !(fabsf(p->branch_scale) < 1e30f))
    return op_fail(DP_ERR_INVALID_ARG, "res_scale and branch_scale must be finite");
  if (p->rows == 0) return DP_OK;  // empty tensors have no address: nothing says which of them are there
  if ((p->gate_mode != DP_GATE_NONE) != gate)
    return op_fail(DP_ERR_INVALID_ARG, "gate and gate_mode disagree");
  if (!has_y && (p->norms & DP_NORM_POST || gate || p->res_scale != 1.0f))
    return op_fail(DP_ERR_INVALID_ARG, "without y there is no post norm, no gate and res_scale is 1");
  if (!has_y && !(p->norms & DP_NORM_PRE)) return op_fail(DP_ERR_INVALID_ARG, "neither a block output nor a norm before the next block");
  return DP_OK;
}

NormParams base_params(const dp_block_norm_t& p, const Shape& s) {
  NormParams P = {};
  P.rows = p.rows;
  P.dim = p.dim;
  P.group = s.group;
  P.per_cta = s.per_cta;
  P.layer = p.kind == DP_NORM_LAYER;
  P.post = (p.norms & DP_NORM_POST) != 0;
  P.pre = (p.norms & DP_NORM_PRE) != 0;
  P.gate_mode = p.gate_mode;
  P.pdt = p.param_dtype;
  P.accumulate = p.accumulate;
  P.eps = p.eps;
  P.a = p.res_scale;
  P.b = p.branch_scale;
  return P;
}

bool all16(std::initializer_list<const void*> ps) {
  for (const void* q : ps)
    if (!is_aligned(q, 16)) return false;
  return true;
}

}  // namespace
}  // namespace dp

using namespace dp;

extern "C" {

dp_status_t dp_block_norm(const dp_block_norm_t* p, void* r, void* z, const void* x, const void* y,
                          const void* w_post, const void* b_post, const void* gate, const void* w_pre,
                          const void* b_pre, float* post_stats, float* pre_stats, dp_stream_t stream) {
  DP_TRY(check_norm(p, y != nullptr, gate != nullptr));
  const bool some = p->rows > 0, pre = (p->norms & DP_NORM_PRE) != 0;
  const int es = elem_size(p->stream_dtype), eb = elem_size(p->block_dtype), ep = elem_size(p->param_dtype);
  DP_TRY(check_dev(x, es, some, "x"));
  DP_TRY(check_dev(y, eb, false, "y"));
  DP_TRY(check_dev(r, es, some && y, "r"));
  DP_TRY(check_dev(z, eb, some && pre, "z"));
  if (some && !y && r) return op_fail(DP_ERR_INVALID_ARG, "r must be NULL without y");
  if (some && !pre && z) return op_fail(DP_ERR_INVALID_ARG, "z must be NULL without DP_NORM_PRE");
  DP_TRY(check_dev(w_post, ep, false, "w_post"));
  DP_TRY(check_dev(b_post, ep, false, "b_post"));
  DP_TRY(check_dev(gate, ep, false, "gate"));
  DP_TRY(check_dev(w_pre, ep, false, "w_pre"));
  DP_TRY(check_dev(b_pre, ep, false, "b_pre"));
  DP_TRY(check_dev(post_stats, 8, false, "post_stats"));
  DP_TRY(check_dev(pre_stats, 8, false, "pre_stats"));
  if (!some) return DP_OK;
  const Shape s = shape_of(p->dim);
  NormParams P = base_params(*p, s);
  P.r = r;
  P.z = z;
  P.x = x;
  P.y = y;
  // Without the post norm its weight and bias are not used: N_post(y) = y.
  P.w_post = P.post ? w_post : nullptr;
  P.b_post = P.post ? b_post : nullptr;
  P.gate = gate;
  P.w_pre = w_pre;
  P.b_pre = b_pre;
  P.post_stats = reinterpret_cast<float2*>(post_stats);
  P.pre_stats = reinterpret_cast<float2*>(pre_stats);
  NvtxRange range("block norm");
  dispatch(*p, p->dim % 8 == 0 && all16({x, y, r, z}), s.nv, Forward{P, s, (cudaStream_t)stream});
  return op_launched("block norm launch", 1);
}

size_t dp_block_norm_workspace_size(int64_t rows, int64_t dim) {
  if (rows < 0 || rows > INT32_MAX || dim < 1 || dim > DP_MAX_NORM_DIM) {
    op_fail(DP_ERR_INVALID_ARG, "rows = %lld or dim = %lld out of range", (long long)rows, (long long)dim);
    return 0;
  }
  const int64_t parts = rows + 3 < MAX_PARTS ? rows + 3 : MAX_PARTS;
  return (size_t)(parts * 4 * dim * 4 + 255) / 256 * 256;
}

dp_status_t dp_block_norm_grad(const dp_block_norm_t* p, void* dx, void* dy, const void* dr, const void* dz,
                               const void* r, const void* y, const void* w_post, const void* b_post, const void* gate,
                               const void* w_pre, const float* post_stats, const float* pre_stats, void* dw_post,
                               void* db_post, void* dgate, void* dw_pre, void* db_pre, void* ws, dp_stream_t stream_) {
  DP_TRY(check_norm(p, y != nullptr, gate != nullptr));
  const bool some = p->rows > 0, pre = (p->norms & DP_NORM_PRE) != 0, post = (p->norms & DP_NORM_POST) != 0;
  const int es = elem_size(p->stream_dtype), eb = elem_size(p->block_dtype), ep = elem_size(p->param_dtype);
  DP_TRY(check_dev(dx, es, some, "dx"));
  DP_TRY(check_dev(dy, eb, some && y, "dy"));
  DP_TRY(check_dev(dr, es, false, "dr"));
  DP_TRY(check_dev(dz, eb, some && pre, "dz"));
  DP_TRY(check_dev(r, es, some && pre, "r"));
  DP_TRY(check_dev(y, eb, false, "y"));
  if (some && !y && dy) return op_fail(DP_ERR_INVALID_ARG, "dy must be NULL without y");
  DP_TRY(check_dev(w_post, ep, false, "w_post"));
  DP_TRY(check_dev(b_post, ep, false, "b_post"));
  DP_TRY(check_dev(gate, ep, false, "gate"));
  DP_TRY(check_dev(w_pre, ep, false, "w_pre"));
  DP_TRY(check_dev(post_stats, 8, some && post, "post_stats"));
  DP_TRY(check_dev(pre_stats, 8, some && pre, "pre_stats"));
  DP_TRY(check_dev(dw_post, ep, false, "dw_post"));
  DP_TRY(check_dev(db_post, ep, false, "db_post"));
  DP_TRY(check_dev(dgate, ep, false, "dgate"));
  DP_TRY(check_dev(dw_pre, ep, false, "dw_pre"));
  DP_TRY(check_dev(db_pre, ep, false, "db_pre"));
  if (!post && (dw_post || db_post)) return op_fail(DP_ERR_INVALID_ARG, "dw_post and db_post need DP_NORM_POST");
  if (!pre && (dw_pre || db_pre)) return op_fail(DP_ERR_INVALID_ARG, "dw_pre and db_pre need DP_NORM_PRE");
  if (p->gate_mode == DP_GATE_NONE && dgate) return op_fail(DP_ERR_INVALID_ARG, "dgate needs a gate");
  DP_TRY(check_dev(ws, 256, some, "ws"));
  const cudaStream_t stream = (cudaStream_t)stream_;
  NvtxRange range("block norm gradient");
  int64_t parts = 0;
  int launches = 0;
  // S0 and P0 are summed for the biases' gradients, and for a channel gate's where the post norm has a bias.
  const bool sum0 = p->kind == DP_NORM_LAYER || db_post || db_pre || (dgate && post && b_post);
  if (some) {
    const Shape s = shape_of(p->dim);
    NormParams P = base_params(*p, s);
    P.dx = dx;
    P.dy = dy;
    P.dr = dr;
    P.dz = dz;
    P.x = r;
    P.y = y;
    P.w_post = post ? w_post : nullptr;
    P.b_post = post ? b_post : nullptr;
    P.gate = gate;
    P.w_pre = w_pre;
    P.post_stats = reinterpret_cast<float2*>(const_cast<float*>(post_stats));
    P.pre_stats = reinterpret_cast<float2*>(const_cast<float*>(pre_stats));
    P.dgate_token = p->gate_mode == DP_GATE_TOKEN ? dgate : nullptr;
    P.part = static_cast<float*>(ws);
    parts = dispatch(*p, p->dim % 8 == 0 && all16({dx, dy, dr, dz, r, y}), s.nv, Gradient{P, s, sum0, stream});
    ++launches;
  }
  FinishParams F = {};
  F.part = static_cast<const float*>(ws);
  F.parts = parts;
  F.dim = p->dim;
  F.sum0 = sum0;
  F.gate_mode = p->gate_mode;
  F.pdt = p->param_dtype;
  F.accumulate = p->accumulate;
  F.w_post = post ? w_post : nullptr;
  F.b_post = post ? b_post : nullptr;
  F.gate = gate;
  F.dw_post = dw_post;
  F.db_post = db_post;
  F.dgate = p->gate_mode == DP_GATE_CHANNEL ? dgate : nullptr;
  F.dw_pre = dw_pre;
  F.db_pre = db_pre;
  F.b = p->branch_scale;
  if (F.dw_post || F.db_post || F.dgate || F.dw_pre || F.db_pre) {
    norm_finish_kernel<<<(p->dim + FIN_COLS - 1) / FIN_COLS, dim3(FIN_COLS, FIN_ROWS), 0, stream>>>(F);
    ++launches;
  }
  return launches ? op_launched("block norm gradient launch", launches) : DP_OK;
}

}  // extern "C"
