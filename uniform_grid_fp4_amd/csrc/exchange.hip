// Token exchange with expert order (gfx950): dispatch, combine and their
// backward passes.  A token's k choices hold the rows given by its slots
// (negative: ~row is a row without a choice).  All four move whole rows and
// compute next to nothing: they are bound by memory.  Each row is read or
// written once, by threads that hold one 16-byte vector of a token's row and go
// over its choices, so the token's own row is read once whatever k is, and the
// sums (FP32, in the order of the choices) need no atomics.  16384 tokens, 6144
// columns, k = 8, bf16, no padding, from HBM: dispatch 362 us (1.81 GB, 5.0 TB/s;
// 310 us with x in the cache), combine with residual 384 us (2.01 GB, 5.2 TB/s),
// dispatch's backward 320 us (1.81 GB, 5.7 TB/s), combine's 684 us (3.42 GB, 5.0
// TB/s).  2048 columns, k = 6, FP32: 189, 201, 158 and 350 us (5.0, 5.3, 5.9 and
// 5.0 TB/s).
#include "block_device.h"
#include "block_kernels.h"

namespace ufp4 {

// The row of a slot, or -1 for one outside the array (INT32_MIN always is).
__device__ __forceinline__ int64_t slot_row(int32_t slot, int64_t rows) {
  const int32_t r = slot < 0 ? ~slot : slot;
  return r < rows ? r : -1;
}

// The slots of up to KB choices from the j-th on; those past k are "no row".
template <int KB>
struct Choices {
  int32_t slot[KB];
  __device__ __forceinline__ Choices(const ExchangeArgs &a, int64_t t, int j0) {
#pragma unroll
    for (int j = 0; j < KB; ++j) slot[j] = j0 + j < a.k ? a.slots[t * a.k + j0 + j] : INT32_MIN;
  }
};

// Units of work: LPT lanes take LPT vectors of one token's row.  A wave (64) per
// unit keeps the token, its slots and every branch on them scalar; rows of up to
// 16 vectors take a DPP row of lanes each, four tokens to a wave (31549 tokens
// of 64 columns, k = 8, all four directions: 53 us, a workgroup per token 327 us).
template <int LPT>
__device__ __forceinline__ int64_t first_unit() {
  int in = threadIdx.x / LPT;
  if (LPT >= 64) in = __builtin_amdgcn_readfirstlane(in);
  return (int64_t)blockIdx.x * (256 / LPT) + in;
}
template <int LPT>
__device__ __forceinline__ int64_t unit_step() {
  return (int64_t)gridDim.x * (256 / LPT);
}

// Where a lane's vector starts: the one that passes the end of the row is taken
// back to end with it, so that no lane goes element by element (24002 tokens of
// 575 columns, k = 4, no padding, all four directions: 197 us, masked accesses
// 285 us).  Elements that two lanes then hold get the same value from both.  Rows
// shorter than a vector keep the masked accesses.
template <int V>
__device__ __forceinline__ int64_t vec_start(int64_t c, int64_t cols) {
  return cols >= V ? min(c, cols - V) : c;
}

// Thread = one vector of one token's row, written to its k rows.
template <typename T, int KB, int LPT>
__global__ __launch_bounds__(256) void dispatch_kernel(const ExchangeArgs a, int64_t chunks) {
  constexpr int V = Elem<T>::V;
  const int64_t rows = a.tokens * a.k;
  for (int64_t u = first_unit<LPT>(); u < a.tokens * chunks; u += unit_step<LPT>()) {
    const int64_t t = u / chunks;
    int64_t c = ((u - t * chunks) * LPT + threadIdx.x % LPT) * V;
    if (c >= a.cols) continue;
    c = vec_start<V>(c, a.cols);
    const u32x4 v = load_vec(static_cast<const T *>(a.in) + t * a.ld_in + c, a.cols - c);
    for (int j0 = 0; j0 < a.k; j0 += KB) {
      const Choices<KB> ch(a, t, j0);
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        const int64_t r = slot_row(ch.slot[j], rows);
        if (r >= 0)
          store_as(static_cast<T *>(a.out) + r * a.cols + c, a.cols - c,
                   ch.slot[j] < 0 ? u32x4(0) : v, a.stream);
      }
    }
  }
}

// Thread = one vector of one token's row: the (weighted) sum of its k rows,
// KB of them in flight at once.
template <typename T, bool GATED, int KB, int LPT>
__global__ __launch_bounds__(256) void combine_kernel(const ExchangeArgs a, int64_t chunks) {
  constexpr int V = Elem<T>::V;
  const int64_t rows = a.tokens * a.k;
  for (int64_t u = first_unit<LPT>(); u < a.tokens * chunks; u += unit_step<LPT>()) {
    const int64_t t = u / chunks;
    int64_t c = ((u - t * chunks) * LPT + threadIdx.x % LPT) * V;
    if (c >= a.cols) continue;
    c = vec_start<V>(c, a.cols);
    const T *in = static_cast<const T *>(a.in) + c;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    u32x4 res = u32x4(0);
    if (GATED && a.res != nullptr)
      res = load_vec(static_cast<const T *>(a.res) + t * a.ld_res + c, a.cols - c);
    for (int j0 = 0; j0 < a.k; j0 += KB) {
      const Choices<KB> ch(a, t, j0);
      u32x4 v[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        v[j] = u32x4(0);
        if (ch.slot[j] >= 0 && ch.slot[j] < rows)
          v[j] = load_as(in + (int64_t)ch.slot[j] * a.cols, a.cols - c, a.stream);
      }
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        if (ch.slot[j] < 0 || ch.slot[j] >= rows) continue;
        const float g = GATED ? a.gates[t * a.k + j0 + j] : 1.0f;
        float f[V];
        Elem<T>::unpack(v[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i)
          sum[i] = GATED ? __builtin_fmaf(g, f[i], sum[i]) : sum[i] + f[i];
      }
    }
    if (GATED && a.res != nullptr) {
      float f[V];
      Elem<T>::unpack(res, f);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += f[i];
    }
    store_as(static_cast<T *>(a.out) + t * a.cols + c, a.cols - c, Elem<T>::pack(sum),
             a.stream);
  }
}

// LPT lanes per token at a time, LPT vectors of its row after the other: dys =
// g dy in each choice's row, and the dot products of its row of ys with dy,
// which is read once per KB choices.  Up to 192 vectors a wave does it without a
// barrier (16384 tokens of 1408 columns, k = 6: 118 us, a workgroup 137 us);
// longer rows take a workgroup (2048 columns: 175 us, a wave 188 us).
template <typename T, int KB, int LPT>
__global__ __launch_bounds__(256) void combine_bwd_kernel(const ExchangeArgs a) {
  constexpr int V = Elem<T>::V;
  __shared__ float s_dot[2][KB][4];
  const int64_t rows = a.tokens * a.k;
  const int lane = threadIdx.x % LPT;
  int turn = 0;
  for (int64_t t = first_unit<LPT>(); t < a.tokens; t += unit_step<LPT>()) {
    const T *dy = static_cast<const T *>(a.dy) + t * a.ld_dy;
    for (int j0 = 0; j0 < a.k; j0 += KB, turn ^= 1) {
      const Choices<KB> ch(a, t, j0);
      float g[KB], dot[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        dot[j] = 0.0f;
        g[j] = ch.slot[j] >= 0 ? a.gates[t * a.k + j0 + j] : 0.0f;
      }
      for (int64_t c0 = lane * V; c0 < a.cols; c0 += LPT * V) {
        const int64_t c = vec_start<V>(c0, a.cols);
        float d[V];
        u32x4 v[KB];
        const u32x4 vd = load_vec(dy + c, a.cols - c);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          v[j] = u32x4(0);
          if (ch.slot[j] >= 0 && ch.slot[j] < rows)
            v[j] = load_as(static_cast<const T *>(a.in) + (int64_t)ch.slot[j] * a.cols + c,
                           a.cols - c, a.stream);
        }
        Elem<T>::unpack(vd, d);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const int64_t r = slot_row(ch.slot[j], rows);
          if (r < 0) continue;
          float f[V];
          if (ch.slot[j] >= 0) {
            Elem<T>::unpack(v[j], f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              dot[j] = c + i >= c0 ? __builtin_fmaf(f[i], d[i], dot[j]) : dot[j];
              f[i] = d[i] * g[j];
            }
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = 0.0f;
          }
          store_as(static_cast<T *>(a.out) + r * a.cols + c, a.cols - c, Elem<T>::pack(f),
                   a.stream);
        }
      }
      if constexpr (LPT == 256) {
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          dot[j] = lanes_sum(dot[j]);
          if ((threadIdx.x & 63) == 0) s_dot[turn][j][threadIdx.x >> 6] = dot[j];
        }
        __syncthreads();
        if (lane < KB && j0 + lane < a.k) {
          const float *s = s_dot[turn][lane];
          a.d_gates[t * a.k + j0 + lane] = ((s[0] + s[1]) + s[2]) + s[3];
        }
      } else {
        float mine = 0.0f;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const float sum = LPT == 64 ? lanes_sum(dot[j]) : row_sum(dot[j]);
          mine = lane == j ? sum : mine;
        }
        if (lane < KB && j0 + lane < a.k) a.d_gates[t * a.k + j0 + lane] = mine;
      }
    }
  }
}

// A launch holds fewer than 2^32 threads; work beyond the grid is looped over.
static unsigned grid_of(int64_t blocks) {
  return (unsigned)(blocks < (1 << 23) ? blocks : (1 << 23));
}

template <typename T, int KB, int LPT>
static hipError_t exchange_units(const ExchangeArgs &a, int what, hipStream_t st) {
  constexpr int64_t kUnits = 256 / LPT;
  const int64_t per = LPT * Elem<T>::V, chunks = (a.cols + per - 1) / per;
  const dim3 grid(grid_of((a.tokens * chunks + kUnits - 1) / kUnits)), block(256);
  if (what == 0)
    hipLaunchKernelGGL((dispatch_kernel<T, KB, LPT>), grid, block, 0, st, a, chunks);
  else if (what == 1)
    hipLaunchKernelGGL((combine_kernel<T, false, KB, LPT>), grid, block, 0, st, a, chunks);
  else if (what == 2)
    hipLaunchKernelGGL((combine_kernel<T, true, KB, LPT>), grid, block, 0, st, a, chunks);
  else
    hipLaunchKernelGGL((combine_bwd_kernel<T, KB, LPT>),
                       dim3(grid_of((a.tokens + kUnits - 1) / kUnits)), block, 0, st, a);
  return hipGetLastError();
}

template <typename T, int KB>
static hipError_t exchange_of(const ExchangeArgs &a, int what, hipStream_t st) {
  const int64_t vecs = (a.cols + Elem<T>::V - 1) / Elem<T>::V;
  if (vecs <= 16) return exchange_units<T, KB, 16>(a, what, st);
  if (what == 3 && vecs > 192) {
    hipLaunchKernelGGL((combine_bwd_kernel<T, KB, 256>), dim3(grid_of(a.tokens)), dim3(256), 0, st,
                       a);
    return hipGetLastError();
  }
  return exchange_units<T, KB, 64>(a, what, st);
}

// Rows in flight per thread: the smallest of 1, 2, 4, 8 that holds k.
template <typename T>
static hipError_t exchange(ExchangeArgs a, int what, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  // the sums too: with their reader, 16384 x 6144 x 8 takes 423 us, and 431 us
  // when only the rows in expert order stream
  a.stream = a.tokens * a.k * a.cols * (int64_t)sizeof(T) >= kStreamBytes;
  if (a.k <= 1) return exchange_of<T, 1>(a, what, st);
  if (a.k <= 2) return exchange_of<T, 2>(a, what, st);
  if (a.k <= 4) return exchange_of<T, 4>(a, what, st);
  return exchange_of<T, 8>(a, what, st);
}

hipError_t launch_dispatch(const ExchangeArgs &a, hipStream_t st) {
  return a.bf16 ? exchange<uint16_t>(a, 0, st) : exchange<float>(a, 0, st);
}
hipError_t launch_combine(const ExchangeArgs &a, hipStream_t st) {
  const int what = a.gates != nullptr ? 2 : 1;
  return a.bf16 ? exchange<uint16_t>(a, what, st) : exchange<float>(a, what, st);
}
hipError_t launch_combine_bwd(const ExchangeArgs &a, hipStream_t st) {
  return a.bf16 ? exchange<uint16_t>(a, 3, st) : exchange<float>(a, 3, st);
}

}  // namespace ufp4
