// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = s E[id_t]            dE[v] (+)= s sum_{t : id_t = v} dout[t]
//
// Both move bytes and compute almost nothing.  The lookup reads and writes each row once.  The gradient has to read
// dout once (T d) and write the table's gradient once (V d, or the touched rows twice when it is added): adding each
// token's row into the table with atomics would read and write rows once per token, in an order that changes from run
// to run.  Instead the token numbers (4 bytes against a row of 2 d) are sorted first, and each row's sum is then taken
// in registers, in the order of the sorted tokens, and written once.
//
//   1. emb_sort_kernel: one cluster of 8 CTAs sorts (id, token) by id, stable, with an LSD radix sort whose digits'
//      counts the CTAs exchange through distributed shared memory.  When the gradient is written (not added), the
//      launch's other clusters fill the table with zeros meanwhile: the fill is longer than the sort.
//   2. emb_sum_kernel: the sorted tokens are cut into chunks of equal length, whatever the ids; a warp takes one chunk
//      and 256 columns and adds the chunk's runs of equal ids.  A run inside a chunk is finished there; a run that
//      crosses chunks leaves fp32 partial sums.
//   3. emb_join_kernel: a run's partial sums are added in chunk order.  So a token that fills half the batch costs as
//      much as any other, and nothing depends on the order in which CTAs run.
#include "op_common.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace dp {
namespace {

constexpr int SORT_CTAS = 8;       // one portable cluster
constexpr int SORT_THREADS = 1024;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int MAX_RADIX = 256;
constexpr int COLS = 256;          // columns of a warp: 8 per lane
constexpr int JOIN_WARPS = 8;

struct EmbWs {  // 4-byte words
  int64_t key[2], tok[2], part;
  int64_t words;
};
__host__ __device__ inline int64_t up64(int64_t x) { return (x + 63) & ~int64_t(63); }

// Tokens of a chunk: long enough that few partial sums are written (two rows of fp32 a chunk against chunk rows of
// bf16), short enough to give every SM several warps.
inline int chunk_of(int64_t tokens, int64_t dim) {
  const int64_t slabs = (dim + COLS - 1) / COLS;
  for (int c = 32; c > 8; c >>= 1)
    if ((tokens + c - 1) / c * slabs >= 148 * 16) return c;
  return 8;
}
inline EmbWs emb_ws(int64_t tokens, int64_t dim) {
  EmbWs w;
  const int64_t t = up64(tokens);
  const int c = chunk_of(tokens, dim);
  w.key[0] = 0;
  w.key[1] = t;
  w.tok[0] = 2 * t;
  w.tok[1] = 3 * t;
  w.part = 4 * t;
  w.words = w.part + (tokens + c - 1) / c * 2 * up64(dim);
  return w;
}

// ------------------------------------------------------------------------------------------------------- lookup

template <typename T>
__global__ void __launch_bounds__(256) emb_lookup_kernel(T* __restrict__ out, const T* __restrict__ table,
                                                         const void* __restrict__ ids, int id64, int64_t tokens,
                                                         int64_t vocab, int64_t dim, float scale, int vec) {
  // A warp a token: ids of one warp's token are one broadcast load, a row is read in consecutive 16-byte words.
  const int lane = threadIdx.x & 31;
  const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t t = warp; t < tokens; t += warps) {
    const int64_t id = id64 ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
    const bool live = id >= 0 && id < vocab;
    const T* src = table + (live ? id : 0) * dim;
    T* dst = out + t * dim;
    if (vec) {
#pragma unroll 4
      for (int64_t c = lane * 8; c < dim; c += 256) {
        float v[8];
        if (live) {
          const Raw8<T> w = load_raw8(src + c);
          w.unpack(v);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] *= scale;
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = 0.0f;
        }
        Raw8<T> o;
        o.pack(v);
        store_raw8(dst + c, o);
      }
    } else {
#pragma unroll 4
      for (int64_t c = lane; c < dim; c += 32) dst[c] = Elem<T>::put(live ? Elem<T>::get(src[c]) * scale : 0.0f);
    }
  }
}

// --------------------------------------------------------------------------------------------------------- sort

struct SortParams {
  const void* ids;
  int id64;
  int64_t tokens, vocab, pad_id;
  uint32_t* key[2];
  uint32_t* tok[2];
  int passes, bits;
  char* fill;  // bytes to set to zero, or NULL
  int64_t fill_bytes;
};

__device__ __forceinline__ uint32_t key_of(const SortParams& P, int64_t t) {
  const int64_t id = P.id64 ? static_cast<const int64_t*>(P.ids)[t] : static_cast<const int32_t*>(P.ids)[t];
  return (id < 0 || id >= P.vocab || id == P.pad_id) ? (uint32_t)P.vocab : (uint32_t)id;
}

// One LSD pass, most of it a warp's own: warp w of CTA c owns the w-th run of the c-th eighth of the array.  It counts
// its digits; the counts are scanned over digits, then CTAs, then warps, which gives every warp its first place for
// every digit; then it places its elements in order, 32 at a time, equal digits of the 32 by their lanes' order.  That
// order is the array's own, so the sort is stable and the same in every run.
__global__ void __cluster_dims__(SORT_CTAS, 1, 1) __launch_bounds__(SORT_THREADS)
    emb_sort_kernel(const __grid_constant__ SortParams P) {
  if (blockIdx.x >= SORT_CTAS) {  // whole clusters: these never meet the sort's barriers
    const int64_t me = (int64_t)(blockIdx.x - SORT_CTAS) * SORT_THREADS + threadIdx.x;
    const int64_t step = (int64_t)(gridDim.x - SORT_CTAS) * SORT_THREADS;
    const int64_t head0 = (16 - (int64_t)((uintptr_t)P.fill & 15)) & 15;
    const int64_t head = head0 < P.fill_bytes ? head0 : P.fill_bytes;
    const int64_t words = (P.fill_bytes - head) / 16;
    uint4* w = reinterpret_cast<uint4*>(P.fill + head);
    for (int64_t i = me; i < words; i += step) w[i] = make_uint4(0, 0, 0, 0);
    if (me < head) P.fill[me] = 0;
    const int64_t tail = head + words * 16;
    if (me < P.fill_bytes - tail) P.fill[tail + me] = 0;
    return;
  }
  __shared__ uint32_t wcount[SORT_WARPS][MAX_RADIX];
  __shared__ uint32_t total[MAX_RADIX];  // this CTA's counts, read by the others
  __shared__ uint32_t base[MAX_RADIX];
  __shared__ uint32_t scan[8];
  cg::cluster_group cluster = cg::this_cluster();
  const int cta = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t per = (P.tokens + SORT_CTAS * SORT_WARPS - 1) / (SORT_CTAS * SORT_WARPS);
  const int64_t lo0 = per * (cta * SORT_WARPS + warp);
  const int64_t lo = lo0 < P.tokens ? lo0 : P.tokens;
  const int64_t hi = lo + per < P.tokens ? lo + per : P.tokens;
  const uint32_t radix = 1u << P.bits, mask = radix - 1;

  for (int pass = 0; pass < P.passes; ++pass) {
    const int shift = pass * P.bits;
    const uint32_t* ksrc = P.key[(pass + 1) & 1];
    const uint32_t* tsrc = P.tok[(pass + 1) & 1];
    uint32_t* kdst = P.key[pass & 1];
    uint32_t* tdst = P.tok[pass & 1];
    for (uint32_t d = lane; d < radix; d += 32) wcount[warp][d] = 0;
    __syncwarp();
#pragma unroll 4
    for (int64_t i = lo + lane; i < hi; i += 32) {
      const uint32_t k = pass == 0 ? key_of(P, i) : ksrc[i];
      atomicAdd(&wcount[warp][(k >> shift) & mask], 1u);
    }
    __syncthreads();
    uint32_t mine = 0;
    if (threadIdx.x < radix) {  // this CTA's total of one digit; the warps' counts become their offsets in it
      for (int w = 0; w < SORT_WARPS; ++w) {
        const uint32_t c = wcount[w][threadIdx.x];
        wcount[w][threadIdx.x] = mine;
        mine += c;
      }
      total[threadIdx.x] = mine;
    }
    cluster.sync();
    uint32_t all = 0, before = 0;
    if (threadIdx.x < radix) {
#pragma unroll
      for (int c = 0; c < SORT_CTAS; ++c) {
        const uint32_t v = *cluster.map_shared_rank(&total[threadIdx.x], c);
        before += c < cta ? v : 0;
        all += v;
      }
    }
    uint32_t incl = all;  // scan over the digits: the first 8 warps hold them
    if (threadIdx.x < MAX_RADIX) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) scan[warp] = incl;
    }
    __syncthreads();
    if (threadIdx.x < radix) {
      uint32_t first = incl - all + before;
      for (int w = 0; w < warp; ++w) first += scan[w];
      base[threadIdx.x] = first;
    }
    __syncthreads();
    for (uint32_t d = lane; d < radix; d += 32) wcount[warp][d] += base[d];
    __syncwarp();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      const bool on = i < hi;
      const uint32_t k = on ? (pass == 0 ? key_of(P, i) : ksrc[i]) : 0;
      const uint32_t t = on ? (pass == 0 ? (uint32_t)i : tsrc[i]) : 0;
      const uint32_t digit = on ? (k >> shift) & mask : 0xffffffffu;
      const uint32_t peers = __match_any_sync(0xffffffffu, digit);
      const uint32_t below = __popc(peers & ((1u << lane) - 1));
      uint32_t at = 0;
      if (on) at = wcount[warp][digit] + below;
      __syncwarp();
      if (on && below == 0) wcount[warp][digit] += __popc(peers);
      __syncwarp();
      if (on) {
        kdst[at] = k;
        tdst[at] = t;
      }
    }
    cluster.sync();  // the pass's elements are placed; nobody reads this pass's totals any more
  }
}

// ------------------------------------------------------------------------------------------------- segmented sum

struct SumParams {
  void* dtable;
  const void* dout;
  const uint32_t* key;
  const uint32_t* tok;
  float* part;
  int64_t tokens, dim, pitch;  // pitch: floats of one partial row
  uint32_t vocab;
  float scale;
  int accumulate, chunk, slabs;
};

template <typename T, int VEC>
__device__ __forceinline__ void load_cols(const T* row, int64_t col0, int lane, int64_t dim, float (&v)[8]) {
  if (VEC) {
    const int64_t c = col0 + lane * 8;
    if (c < dim) {
      const Raw8<T> w = load_raw8(row + c);
      w.unpack(v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t c = col0 + lane + 32 * k;
      v[k] = c < dim ? Elem<T>::get(row[c]) : 0.0f;
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void finish_row(const SumParams& P, uint32_t key, int64_t col0, int lane, float (&acc)[8]) {
  T* row = static_cast<T*>(P.dtable) + (int64_t)key * P.dim;
  float v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = acc[k] * P.scale;
  if (P.accumulate) {
    float old[8];
    load_cols<T, VEC>(row, col0, lane, P.dim, old);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __fadd_rn(old[k], v[k]);
  }
  if (VEC) {
    const int64_t c = col0 + lane * 8;
    if (c < P.dim) {
      Raw8<T> o;
      o.pack(v);
      store_raw8(row + c, o);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t c = col0 + lane + 32 * k;
      if (c < P.dim) row[c] = Elem<T>::put(v[k]);
    }
  }
}

// Partial rows are kept in the lanes' order (each lane's eight sums together): only the same lane reads them.
__device__ __forceinline__ float4* part_at(const SumParams& P, int64_t chunk, int which, int slab, int lane) {
  return reinterpret_cast<float4*>(P.part + (chunk * 2 + which) * P.pitch + (int64_t)slab * COLS + lane * 8);
}

template <typename T, int VEC>
__global__ void __launch_bounds__(128) emb_sum_kernel(const __grid_constant__ SumParams P) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t chunk = unit / P.slabs;
  const int slab = (int)(unit - chunk * P.slabs);
  const int64_t first = chunk * P.chunk;
  if (first >= P.tokens) return;
  const int64_t col0 = (int64_t)slab * COLS;
  const int n = (int)(P.tokens - first < P.chunk ? P.tokens - first : P.chunk);
  // Lane j holds the chunk's j-th key and token (a chunk has at most 32).
  const uint32_t none = 0xffffffffu;
  const uint32_t mykey = lane < n ? P.key[first + lane] : none;
  const uint32_t mytok = lane < n ? P.tok[first + lane] : 0;
  const uint32_t prev = first > 0 ? P.key[first - 1] : none;
  const uint32_t next = first + n < P.tokens ? P.key[first + n] : none;
  const uint32_t dead = __ballot_sync(0xffffffffu, mykey >= P.vocab);  // dropped tokens sort behind all rows
  const int live = min(n, dead ? __ffs(dead) - 1 : 32);
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
  bool open = false;  // the current run began in an earlier chunk
  uint32_t cur = none;
  constexpr int U = 8;  // rows in flight
  for (int j0 = 0; j0 < live; j0 += U) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t t = __shfl_sync(0xffffffffu, mytok, min(j0 + u, live - 1));
      if (j0 + u < live) load_cols<T, VEC>(static_cast<const T*>(P.dout) + (int64_t)t * P.dim, col0, lane, P.dim, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t key = __shfl_sync(0xffffffffu, mykey, min(j0 + u, live - 1));
      if (j0 + u < live) {
        if (key != cur) {
          if (cur != none) {  // the run ended inside this chunk
            if (open) {
              float4* p = part_at(P, chunk, 0, slab, lane);
              p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
              p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
            } else {
              finish_row<T, VEC>(P, cur, col0, lane, acc);
            }
          }
          open = j0 + u == 0 && key == prev;
          cur = key;
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = v[u][k];
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = __fadd_rn(acc[k], v[u][k]);
        }
      }
    }
  }
  if (cur != none) {
    const bool goes_on = live == n && next == cur;
    if (open || goes_on) {
      float4* p = part_at(P, chunk, open ? 0 : 1, slab, lane);
      p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    } else {
      finish_row<T, VEC>(P, cur, col0, lane, acc);
    }
  }
}

// One CTA for each chunk boundary and slab: works where a run begins in the chunk and goes on into the next.  The run's
// further chunks are shared out among the warps in eight consecutive parts, each added in order, then joined in order.
template <typename T, int VEC>
__global__ void __launch_bounds__(JOIN_WARPS * 32) emb_join_kernel(const __grid_constant__ SumParams P) {
  const int64_t chunk = blockIdx.x / P.slabs;
  const int slab = (int)(blockIdx.x - chunk * P.slabs);
  const int64_t first = chunk * P.chunk, last = first + P.chunk - 1;
  if (last + 1 >= P.tokens) return;
  const uint32_t key = P.key[last];
  if (key >= P.vocab || P.key[last + 1] != key) return;                       // no run crosses this boundary
  if (first > 0 && P.key[first] == key && P.key[first - 1] == key) return;    // it began in an earlier chunk
  // The run's end, by bisection of the sorted keys: the first index above `last` that holds another key.
  int64_t a = last + 1, b = P.tokens;  // key[a] == key, key[b] != key or b == tokens
  while (b - a > 1) {
    const int64_t m = a + (b - a) / 2;
    if (P.key[m] == key) a = m; else b = m;
  }
  const int64_t chunks = a / P.chunk - chunk;  // chunks after this one that hold part of the run
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t per = (chunks + JOIN_WARPS - 1) / JOIN_WARPS;
  const int64_t c0 = chunk + 1 + per * warp;
  const int64_t c1 = c0 + per < chunk + 1 + chunks ? c0 + per : chunk + 1 + chunks;
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
  if (warp == 0) {
    const float4* p = part_at(P, chunk, 1, slab, lane);
    const float4 x = p[0], y = p[1];
    acc[0] = x.x; acc[1] = x.y; acc[2] = x.z; acc[3] = x.w; acc[4] = y.x; acc[5] = y.y; acc[6] = y.z; acc[7] = y.w;
  }
#pragma unroll 4
  for (int64_t c = c0; c < c1; ++c) {
    const float4* p = part_at(P, c, 0, slab, lane);
    const float4 x = p[0], y = p[1];
    acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
    acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
  }
  __shared__ float4 sums[JOIN_WARPS][64];
  sums[warp][lane * 2] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  sums[warp][lane * 2 + 1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  __syncthreads();
  if (warp != 0) return;
  for (int w = 1; w < JOIN_WARPS; ++w) {
    const float4 x = sums[w][lane * 2], y = sums[w][lane * 2 + 1];
    acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
    acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
  }
  finish_row<T, VEC>(P, key, (int64_t)slab * COLS, lane, acc);
}

// ---------------------------------------------------------------------------------------------------- host side

dp_status_t check_sizes(int64_t tokens, int64_t vocab, int64_t dim) {
  if (tokens < 0 || tokens > INT32_MAX) return op_fail(DP_ERR_INVALID_ARG, "tokens = %lld not in 0..2^31-1", (long long)tokens);
  if (vocab < 1 || vocab >= INT32_MAX) return op_fail(DP_ERR_INVALID_ARG, "vocab = %lld not in 1..2^31-2", (long long)vocab);
  if (dim < 1 || dim > (int64_t(1) << 24)) return op_fail(DP_ERR_INVALID_ARG, "dim = %lld not in 1..2^24", (long long)dim);
  if ((tokens / 8 + 1) * ((dim + COLS - 1) / COLS) > INT32_MAX)   // the grid of the sums
    return op_fail(DP_ERR_INVALID_ARG, "tokens x dim = %lld x %lld is too large", (long long)tokens, (long long)dim);
  return DP_OK;
}
dp_status_t check_ids(const void* ids, int64_t tokens, int id_bits) {
  if (id_bits != 32 && id_bits != 64) return op_fail(DP_ERR_INVALID_ARG, "id_bits = %d is neither 32 nor 64", id_bits);
  return check_dev(ids, id_bits / 8, tokens > 0, "ids");
}

template <typename T, int VEC>
void launch_sum(const SumParams& P, cudaStream_t stream) {
  const int64_t chunks = (P.tokens + P.chunk - 1) / P.chunk;
  emb_sum_kernel<T, VEC><<<(unsigned)((chunks * P.slabs + 3) / 4), 128, 0, stream>>>(P);
  emb_join_kernel<T, VEC><<<(unsigned)(chunks * P.slabs), JOIN_WARPS * 32, 0, stream>>>(P);
}

}  // namespace
}  // namespace dp

using namespace dp;

extern "C" {

dp_status_t dp_embedding(void* out, const void* table, const void* ids, int64_t tokens, int64_t vocab, int64_t dim,
                         float scale, int32_t dtype, int32_t id_bits, dp_stream_t stream) {
  DP_TRY(check_sizes(tokens, vocab, dim));
  DP_TRY(check_dtype(dtype, "dtype"));
  DP_TRY(check_ids(ids, tokens, id_bits));
  const int e = elem_size(dtype);
  DP_TRY(check_dev(out, e, tokens > 0, "out"));
  DP_TRY(check_dev(table, e, tokens > 0, "table"));
  if (tokens == 0) return DP_OK;
  const int vec = dim % 8 == 0 && is_aligned(out, 16) && is_aligned(table, 16);
  const int64_t ctas = (tokens + 7) / 8, most = (int64_t)sm_count() * 64;
  const unsigned grid = (unsigned)(ctas < most ? ctas : most);
  NvtxRange range("embedding lookup");
  if (dtype == DP_BF16)
    emb_lookup_kernel<bf16_t><<<grid, 256, 0, (cudaStream_t)stream>>>((bf16_t*)out, (const bf16_t*)table, ids, id_bits == 64,
                                                                     tokens, vocab, dim, scale, vec);
  else
    emb_lookup_kernel<float><<<grid, 256, 0, (cudaStream_t)stream>>>((float*)out, (const float*)table, ids, id_bits == 64,
                                                                    tokens, vocab, dim, scale, vec);
  return op_launched("embedding lookup launch", 1);
}

size_t dp_embedding_workspace_size(int64_t tokens, int64_t vocab, int64_t dim) {
  if (check_sizes(tokens, vocab, dim) != DP_OK) return 0;
  return (size_t)emb_ws(tokens, (dim + COLS - 1) / COLS * COLS).words * 4;
}

dp_status_t dp_embedding_grad(void* dtable, const void* dout, const void* ids, int64_t tokens, int64_t vocab,
                              int64_t dim, float scale, int64_t pad_id, int32_t accumulate, int32_t dtype,
                              int32_t id_bits, void* ws, dp_stream_t stream_) {
  DP_TRY(check_sizes(tokens, vocab, dim));
  DP_TRY(check_dtype(dtype, "dtype"));
  DP_TRY(check_ids(ids, tokens, id_bits));
  if (accumulate != 0 && accumulate != 1) return op_fail(DP_ERR_INVALID_ARG, "accumulate = %d is neither 0 nor 1", accumulate);
  const int e = elem_size(dtype);
  DP_TRY(check_dev(dtable, e, true, "dtable"));
  DP_TRY(check_dev(dout, e, tokens > 0, "dout"));
  DP_TRY(check_dev(ws, 256, tokens > 0, "ws"));
  const cudaStream_t stream = (cudaStream_t)stream_;
  if (tokens == 0 && accumulate) return DP_OK;

  const int64_t cols = (dim + COLS - 1) / COLS * COLS;
  const EmbWs w = emb_ws(tokens, cols);
  uint32_t* words = static_cast<uint32_t*>(ws);
  SortParams S;
  S.ids = ids;
  S.id64 = id_bits == 64;
  S.tokens = tokens;
  S.vocab = vocab;
  S.pad_id = pad_id;
  for (int i = 0; i < 2; ++i) {
    S.key[i] = words + w.key[i];
    S.tok[i] = words + w.tok[i];
  }
  int bits = 1;  // keys are 0..vocab
  while (vocab >> bits) ++bits;
  S.passes = (bits + 7) / 8;
  S.bits = (bits + S.passes - 1) / S.passes;
  if (tokens == 0) S.passes = 0;
  S.fill = accumulate ? nullptr : static_cast<char*>(dtable);
  S.fill_bytes = accumulate ? 0 : vocab * dim * e;
  const int64_t want = (S.fill_bytes + SORT_THREADS * 16 * 4 - 1) / (SORT_THREADS * 16 * 4);
  const int64_t most = (int64_t)sm_count() * 2;
  const int64_t fill_ctas = ((want < most ? want : most) + SORT_CTAS - 1) / SORT_CTAS * SORT_CTAS;
  NvtxRange range("embedding gradient");
  emb_sort_kernel<<<(unsigned)(SORT_CTAS + fill_ctas), SORT_THREADS, 0, stream>>>(S);
  if (tokens == 0) return op_launched("embedding gradient launch", 1);

  SumParams P;
  P.dtable = dtable;
  P.dout = dout;
  P.key = S.key[(S.passes - 1) & 1];
  P.tok = S.tok[(S.passes - 1) & 1];
  P.part = reinterpret_cast<float*>(words + w.part);
  P.tokens = tokens;
  P.dim = dim;
  P.pitch = up64(cols);
  P.vocab = (uint32_t)vocab;
  P.scale = scale;
  P.accumulate = accumulate;
  P.chunk = chunk_of(tokens, cols);
  P.slabs = (int)(cols / COLS);
  const int vec = dim % 8 == 0 && is_aligned(dtable, 16) && is_aligned(dout, 16);
  if (dtype == DP_BF16)
    vec ? launch_sum<bf16_t, 1>(P, stream) : launch_sum<bf16_t, 0>(P, stream);
  else
    vec ? launch_sum<float, 1>(P, stream) : launch_sum<float, 0>(P, stream);
  return op_launched("embedding gradient launch", 3);
}

}  // extern "C"
