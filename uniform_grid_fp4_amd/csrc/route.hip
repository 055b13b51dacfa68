// MoE router (gfx950): softmax, top-k choices, gates, counts, group offsets,
// each choice's row in expert order, the balance and z losses, and the
// backward pass.
//   lse = log sum exp(l),  p = exp(l - lse)
//   balance = E sum_e (counts_e / (k N)) (sum_t p_te / N),  z = sum lse^2 / N
//
// Sixteen lanes (one DPP row) hold one token's logits, so that the row
// reductions are four DPP steps and a wave works on four tokens at once.  A
// workgroup takes kRouteTokens = 64 tokens: the choices of an expert are then
// one 64-bit mask in LDS, its count a population count, and a choice's place
// among the workgroup's tokens the population count below its token's bit, all
// independent of the order in which the lanes ran.  A second kernel scans the
// counts over the workgroups and sums their probabilities, a third turns
// places into rows.  Few tokens (one workgroup) take a single launch.
//
// 65536 x 256 bf16 logits, top 8, an eighth of the tokens padding: choices 28 us
// for 29 MB, bound by instruction issue (870 vector instructions for a wave's
// four tokens, 14.3M in all: 23 us on 1024 SIMDs), scan 6.4 us, places 5.8 us;
// backward 16 us for 63 MB (3.9 TB/s).  The same in FP32, whose rounds take two
// row reductions each: 50 us (1320 instructions), 6.4, 6.1, and 22 us for 126 MB
// (5.7 TB/s).  16384 x 64 FP32, top 6: 7.0, 3.2, 4.2 and 5.1 us, in bf16 6.5, 3.4,
// 4.4 and 5.3 us, one token 4.5 us: latency and launches.
//
// Sums over a row are FP32; sums of p over tokens are FP32 within a workgroup
// and FP64 across, z and the losses FP64.
#include "block_device.h"
#include "block_kernels.h"

namespace ufp4 {

constexpr int kBwdGroups = 16;                   // tokens in flight, backward
// Threads of the forward kernel: with 1024 each group of 16 lanes has one token
// and the latencies of the choices run side by side (16384 x 64: 7.5 us, with
// 256 threads 11.4 us); the registers of long rows allow 256 and four tokens in
// turn.  A single workgroup with few tokens has no use for more than 256.
constexpr int route_threads(int r, bool alone) { return alone || r > 16 ? 256 : 1024; }
// Workgroups per launch: a launch holds fewer than 2^32 threads, and 2^28 tokens
// or more take several, each from its first block of kRouteTokens tokens on.
constexpr int64_t kRouteGrid = int64_t(1) << 21;

// Workspace of a call with nblk workgroups, E experts:
//   uint32 base [E + 1][nblk]  choices per expert (last: choices that do not
//                              exist) and workgroup, then their exclusive sums
//   float  psum [E][nblk]      sums of p
//   double z    [nblk], uint32 live [nblk]
//   uint32 total[E + 2]        choices per expert, missing choices, tokens
//   double ptotal[E + 1]       sums of p, and of lse^2
struct RouteWs {
  uint32_t *base;
  float *psum;
  double *z;
  uint32_t *live;
  uint32_t *total;
  double *ptotal;
  int64_t nblk;
};
__host__ __device__ inline size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }
__host__ __device__ inline size_t route_layout(int64_t nblk, int e, void *p, RouteWs *w) {
  char *at = static_cast<char *>(p);
  size_t used = 0;
  const size_t sizes[6] = {4u * (size_t)nblk * (e + 1), 4u * (size_t)nblk * e, 8u * (size_t)nblk,
                           4u * (size_t)nblk, 4u * (size_t)(e + 2), 8u * (size_t)(e + 1)};
  void *parts[6];
  for (int i = 0; i < 6; ++i) {
    parts[i] = at + used;
    used += up16(sizes[i]);
  }
  if (w != nullptr) {
    w->base = static_cast<uint32_t *>(parts[0]);
    w->psum = static_cast<float *>(parts[1]);
    w->z = static_cast<double *>(parts[2]);
    w->live = static_cast<uint32_t *>(parts[3]);
    w->total = static_cast<uint32_t *>(parts[4]);
    w->ptotal = static_cast<double *>(parts[5]);
    w->nblk = nblk;
  }
  return used;
}
static int64_t route_blocks(int64_t tokens) {
  const int64_t n = (tokens + kRouteTokens - 1) / kRouteTokens;
  return n < 1 ? 1 : n;
}
size_t route_workspace_bytes(int64_t tokens, int n_experts) {
  const int64_t nblk = route_blocks(tokens);
  return nblk == 1 ? 0 : route_layout(nblk, n_experts, nullptr, nullptr);
}

// A logit as an unsigned number of the same order, equal for -0 and +0.
__device__ __forceinline__ uint32_t order_key(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}
constexpr uint32_t kKeyMinusInf = 0x007FFFFFu;   // order_key(-inf): nothing at or below is chosen

// exp(l - from) for the softmax sums, l <= from.  The argument's rounding makes
// a term off by |l - from| 2^-23 of itself; terms far from the maximum, where
// that grows, are small.
__device__ __forceinline__ float exp_term(float l, float from) {
  return __builtin_amdgcn_exp2f((l - from) * 1.44269504f);
}

__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  v = min(v, row_rotate<8>(v));
  v = min(v, row_rotate<4>(v));
  v = min(v, row_rotate<2>(v));
  return min(v, row_rotate<1>(v));
}

// Expert held by lane l in register i: sixteen lanes take runs of W
// consecutive experts (one 16-byte load where the runs are that long).
// FULL: there are exactly 16 R experts, and no lane has to ask whether its own
// exist.
template <typename T, int R, bool FULL>
struct Hold {
  static constexpr int W = R < Elem<T>::V ? R : Elem<T>::V;
  __device__ static __forceinline__ int expert(int lane, int i) {
    return (i / W) * (16 * W) + lane * W + i % W;
  }
  __device__ static __forceinline__ bool exists(int lane, int i, int e) {
    return FULL || expert(lane, i) < e;
  }
  // The token's logits; -inf past the last expert.
  __device__ static __forceinline__ void load(const T *p, int e, int lane, float (&f)[R]) {
#pragma unroll
    for (int i = 0; i < R; i += W) {
      const int at = expert(lane, i);
      if (W == Elem<T>::V && (FULL || at + W <= e)) {
        float v[Elem<T>::V];
        Elem<T>::unpack(*reinterpret_cast<const u32x4_any *>(p + at), v);
#pragma unroll
        for (int j = 0; j < W; ++j) f[i + j] = v[j];
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) f[i + j] = FULL || at + j < e ? Elem<T>::get(p[at + j]) : -INFINITY;
      }
    }
  }
};

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t below = (uint32_t)__shfl_up((int)v, o, 64);
    if (lane >= o) v += below;
  }
  return v;
}

// Exclusive sums of v[0..n), n <= 1024, in LDS by a workgroup of 256 threads,
// four entries per thread; returns the total.  s_tmp: 4 words.
__device__ uint32_t scan_shared(uint32_t *v, int n, uint32_t *s_tmp) {
  const int at = threadIdx.x * 4, wave = threadIdx.x >> 6;
  uint32_t x[4], mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = at + i < n ? v[at + i] : 0u;
    mine += x[i];
  }
  const uint32_t upto = wave_scan(mine);
  if ((threadIdx.x & 63) == 63) s_tmp[wave] = upto;
  __syncthreads();
  uint32_t run = upto - mine, total = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < wave) run += s_tmp[i];
    total += s_tmp[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (at + i < n) v[at + i] = run;
    run += x[i];
  }
  __syncthreads();
  return total;
}

__device__ __forceinline__ void write_totals(const RouteArgs &a, double balance, double z,
                                             uint32_t tokens) {
  const double n = (double)tokens;
  *a.n_tokens = (int64_t)tokens;
  a.offsets[a.n_experts] = a.tokens * a.k;
  a.losses[0] = tokens ? (float)((double)a.n_experts * balance / ((double)a.k * n * n)) : 0.0f;
  a.losses[1] = tokens ? (float)(z / n) : 0.0f;
}

// Choices, gates and, for the workgroup's 64 tokens, places and counts; with
// ALONE (one workgroup) everything else too.  Dynamic LDS: 12 bytes per expert and 4 for each wave.
template <typename T, int R, bool FULL, bool ALONE>
__global__ __launch_bounds__(route_threads(R, ALONE)) void route_kernel(const RouteArgs a,
                                                                       const RouteWs ws,
                                                                       int64_t block0) {
  constexpr int kThreads = route_threads(R, ALONE), kWaves = kThreads / 64;
  constexpr int kGroups = kThreads / 16, kPer = kRouteTokens / kGroups;   // tokens per group
  extern __shared__ __align__(16) char s_dyn[];
  __shared__ uint32_t s_scan[4];
  __shared__ uint32_t s_lost[kRouteTokens], s_live[kRouteTokens];
  __shared__ float s_lse[kRouteTokens];
  __shared__ double s_part[4];
  const int E = FULL ? 16 * R : a.n_experts, k = a.k;
  const int64_t block = ALONE ? 0 : block0 + blockIdx.x;
  using H = Hold<T, R, FULL>;
  unsigned long long *s_mask = reinterpret_cast<unsigned long long *>(s_dyn);
  uint32_t *s_off = reinterpret_cast<uint32_t *>(s_dyn + 8 * E);
  float *s_p = reinterpret_cast<float *>(s_dyn + 12 * E);         // [kWaves][E]
  const int lane = threadIdx.x & 15, group = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < E; e += kThreads) s_mask[e] = 0;
  float psum[R];
#pragma unroll
  for (int i = 0; i < R; ++i) psum[i] = 0.0f;
  __syncthreads();
  // a token's logits, all -inf (and false) for one that takes no part
  const auto fetch = [&](int64_t t, float (&f)[R]) {
    const bool live = t < a.tokens && (a.valid == nullptr || a.valid[t] != 0);
    if (live) {
      H::load(static_cast<const T *>(a.logits) + t * a.ld, E, lane, f);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) f[i] = -INFINITY;
    }
    return live;
  };
  int32_t choice[kPer], found[kPer];             // lane j: the token's j-th choice
#pragma unroll
  for (int n = 0; n < kPer; ++n) {
    choice[n] = -1;
    found[n] = 0;
    const int local = n * kGroups + group;
    const int64_t t = block * kRouteTokens + local;
    if (block * kRouteTokens + n * kGroups >= a.tokens) {   // the whole workgroup
      if (lane == 0) {
        s_lost[local] = 0;
        s_live[local] = 0;
        s_lse[local] = 0.0f;
      }
      continue;
    }
    const bool here = t < a.tokens;
    float f[R];
    bool live = fetch(t, f);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < R; ++i) top = fmaxf(top, f[i]);
    top = row_max(top);
    // terms of the sum; a row without a finite logit sums to 0, a NaN shows in
    // the sum
    const float from = top > -INFINITY ? top : 0.0f;
    float e[R], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      e[i] = exp_term(f[i], from);
      sum += e[i];
    }
    sum = row_sum(sum);
    const bool odd = sum != sum;                 // a NaN, or infinities
    live = live && (top > -INFINITY || odd);
    // the choices: k rounds of the largest logit left, the lowest expert among
    // equals; lane j keeps round j's
    int32_t mine = -1, count = 0;
    float picked = -INFINITY;
    if constexpr (sizeof(T) == 2) {
      // a bf16's order in 16 bits and 1023 - expert below it make keys that
      // differ, so the next choice is the largest key below the last one:
      // key - last wraps to the top of the range for exactly those
      // (a lane's own keys leave out the lane's bits, which its `last` takes off)
      const uint32_t mine_bits = (uint32_t)(15 - lane) * H::W;
      uint32_t key[R], last = 1u << 26;
#pragma unroll
      for (int i = 0; i < R; ++i)
        key[i] = (order_key(f[i]) >> 16 << 10) | (1023u - (uint32_t)H::expert(15, i));
      if (__any(odd)) {
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (f[i] != f[i]) key[i] = 0u;
      }
      for (int j = 0; j < k; ++j) {
        uint32_t below = last - mine_bits;
        asm("" : "+v"(below));                   // one subtraction per key, not two
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) best = max(best, key[i] - below);
        best = row_max(best);
        last = (best & 0x80000000u) ? best + last : 0u;
        if (last <= (kKeyMinusInf >> 16 << 10 | 1023u)) last = 0u;
        if (lane == j && last != 0u) {
          mine = (int32_t)(1023u - (last & 1023u));
          const uint32_t o = (last << 6) & 0xFFFF0000u;
          picked = key_logit((o & 0x80000000u) ? o : o | 0xFFFFu);
        }
        count += last != 0u ? 1 : 0;
      }
    } else {
      uint32_t key[R];
#pragma unroll
      for (int i = 0; i < R; ++i) key[i] = f[i] != f[i] ? 0u : order_key(f[i]);
      for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) best = max(best, key[i]);
        best = row_max(best);
        if (best <= kKeyMinusInf) best = 0u;
        uint32_t who = 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (key[i] == best) who = min(who, (uint32_t)H::expert(lane, i));
        who = row_min(who);
#pragma unroll
        for (int i = 0; i < R; ++i)
          if ((uint32_t)H::expert(lane, i) == who) key[i] = 0u;
        if (lane == j && best != 0u) {
          mine = (int32_t)who;
          picked = key_logit(best);
        }
        count += best != 0u ? 1 : 0;
      }
    }
    const float lse = live ? top + logf(sum) : -INFINITY;
    const float inv = live ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) psum[i] = __builtin_fmaf(e[i], inv, psum[i]);
    float gate = mine >= 0 ? expf(picked - top) : 0.0f;
    const float total = row_sum(gate);
    gate = mine < 0 ? 0.0f : odd ? sum : (a.renorm ? gate / total : gate * inv);
    choice[n] = mine;
    found[n] = count;
    if (here && lane < k) {
      a.experts[t * k + lane] = mine;
      a.gates[t * k + lane] = gate;
    }
    if (mine >= 0) atomicOr(&s_mask[mine], 1ull << local);
    if (lane == 0) {
      if (here) a.lse[t] = lse;
      s_lost[local] = here ? (uint32_t)(k - count) : 0u;
      s_live[local] = live ? 1u : 0u;
      s_lse[local] = live ? lse : 0.0f;
    }
  }
  // p sums: the wave's four groups, then the waves through LDS
#pragma unroll
  for (int i = 0; i < R; ++i) {
    psum[i] = rows_sum(psum[i]);
    const int e = H::expert(lane, i);
    if ((threadIdx.x & 48) == 0 && H::exists(lane, i, E)) s_p[wave * E + e] = psum[i];
  }
  __syncthreads();
  // wave 0, lane = token: missing choices before each token, tokens, z
  uint32_t lost_all = 0, tokens = 0;
  double z = 0.0;
  if (threadIdx.x < kRouteTokens) {
    const uint32_t own = s_lost[threadIdx.x];
    const uint32_t run = wave_scan(own);
    lost_all = (uint32_t)__shfl((int)run, 63, 64);
    s_lost[threadIdx.x] = run - own;
    tokens = (uint32_t)__popcll(__ballot(s_live[threadIdx.x] != 0));
    z = lanes_sum((double)s_lse[threadIdx.x] * (double)s_lse[threadIdx.x]);
  }
  double balance = 0.0;
  for (int e = threadIdx.x; e < E; e += kThreads) {
    const uint32_t c = (uint32_t)__popcll(s_mask[e]);
    float p = s_p[e];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) p += s_p[w * E + e];
    if (ALONE) {
      s_off[e] = c;
      a.counts[e] = (int64_t)c;
      balance += (double)c * (double)p;
    } else {
      ws.base[e * ws.nblk + block] = c;
      ws.psum[e * ws.nblk + block] = p;
    }
  }
  uint32_t routed = 0;
  if (ALONE) {
    balance = lanes_sum(balance);
    if ((threadIdx.x & 63) == 0) s_part[wave] = balance;
    __syncthreads();
    routed = scan_shared(s_off, E, s_scan);
    for (int e = threadIdx.x; e < E; e += 256) a.offsets[e] = (int64_t)s_off[e];
    if (threadIdx.x == 0)
      write_totals(a, ((s_part[0] + s_part[1]) + s_part[2]) + s_part[3], z, tokens);
  } else {
    if (threadIdx.x == 0) {
      ws.base[E * ws.nblk + block] = lost_all;
      ws.z[block] = z;
      ws.live[block] = tokens;
    }
    __syncthreads();                             // s_lost
  }
#pragma unroll
  for (int n = 0; n < kPer; ++n) {
    const int local = n * kGroups + group;
    const int64_t t = block * kRouteTokens + local;
    if (t >= a.tokens || lane >= k) continue;
    const int e = choice[n];
    uint32_t place;
    if (e >= 0) {
      place = (uint32_t)__popcll(s_mask[e] & ((1ull << local) - 1ull));
      if (ALONE) place += s_off[e];
    } else {
      // a token's choices that exist come first
      place = s_lost[local] + (uint32_t)(lane - found[n]);
      place = ~(ALONE ? place + routed : place);
    }
    a.slots[t * k + lane] = (int32_t)place;
  }
}

// One wave per expert (and one for the missing choices, one for z and the
// tokens): exclusive sums of its counts over the workgroups, in place, and the
// sum of its p in FP64.
__global__ __launch_bounds__(64) void route_scan_kernel(const RouteArgs a, const RouteWs ws,
                                                        int nblk) {
  const int E = a.n_experts, c = blockIdx.x, lane = threadIdx.x;
  double d = 0.0;
  uint32_t run = 0;
  if (c <= E) {
    uint32_t *base = ws.base + (int64_t)c * nblk;
    const float *p = ws.psum + (int64_t)c * nblk;
    for (int b = lane * 4; b - lane * 4 < nblk; b += 256) {
      uint32_t v[4];
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = b + i < nblk ? base[b + i] : 0u;
        if (c < E) d += b + i < nblk ? (double)p[b + i] : 0.0;
        mine += v[i];
      }
      const uint32_t upto = wave_scan(mine);
      uint32_t at = run + upto - mine;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (b + i < nblk) base[b + i] = at;
        at += v[i];
      }
      run += (uint32_t)__shfl((int)upto, 63, 64);
    }
  } else {
    for (int b = lane; b < nblk; b += 64) {
      run += ws.live[b];
      d += ws.z[b];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) run += (uint32_t)__shfl_xor((int)run, o, 64);
  }
  d = lanes_sum(d);
  if (lane == 0) {
    ws.total[c] = run;
    if (c != E) ws.ptotal[c > E ? E : c] = d;
  }
}

// Places to rows, for the 64 tokens of a workgroup; the first block's workgroup
// writes the counts, offsets and losses.
__global__ __launch_bounds__(256) void route_place_kernel(const RouteArgs a, const RouteWs ws,
                                                          int64_t block0) {
  __shared__ uint32_t s_off[kRouteMaxExperts];
  __shared__ uint32_t s_scan[4];
  __shared__ double s_part[4];
  const int E = a.n_experts, k = a.k;
  const int64_t block = block0 + blockIdx.x;
  const bool first = block == 0;
  double balance = 0.0;
  for (int e = threadIdx.x; e < E; e += 256) {
    const uint32_t c = ws.total[e];
    s_off[e] = c;
    if (first) {
      a.counts[e] = (int64_t)c;
      balance += (double)c * ws.ptotal[e];
    }
  }
  __syncthreads();
  const uint32_t routed = scan_shared(s_off, E, s_scan);
  if (first) {
    balance = lanes_sum(balance);
    if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = balance;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 256) a.offsets[e] = (int64_t)s_off[e];
    if (threadIdx.x == 0)
      write_totals(a, ((s_part[0] + s_part[1]) + s_part[2]) + s_part[3], ws.ptotal[E],
                   ws.total[E + 1]);
  }
  const uint32_t *base = ws.base + block;
  const int64_t nblk = ws.nblk;
  const int64_t i0 = block * kRouteTokens * k;
  const int64_t i1 = min(i0 + (int64_t)kRouteTokens * k, a.tokens * k);
  for (int64_t i = i0 + threadIdx.x; i < i1; i += 256) {
    const int32_t e = a.experts[i], place = a.slots[i];
    a.slots[i] = e >= 0 ? (int32_t)(s_off[e] + base[e * nblk] + (uint32_t)place)
                        : (int32_t)~(routed + base[E * nblk] + (uint32_t)~place);
  }
}

// d l_e = p_e (c_e - sum p c - s) + 2 dz lse p_e / N, plus g_j (dg_j - s') at
// the chosen, where c_e = dbal E counts_e / (k N^2); with renorm s = 0 and
// s' = sum g dg, without s = sum g dg and s' = 0.  Dynamic LDS: per group a
// row of E floats that takes the chosen experts' terms to the lanes that hold
// them, zero in between.
template <typename T, int R, bool FULL>
__global__ __launch_bounds__(256) void route_bwd_kernel(const RouteArgs a, int64_t nblk) {
  extern __shared__ __align__(16) char s_dyn[];
  const int E = FULL ? 16 * R : a.n_experts, k = a.k;
  using H = Hold<T, R, FULL>;
  const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
  float *s_add = reinterpret_cast<float *>(s_dyn) + group * E;
  for (int e = lane; e < E; e += 16) s_add[e] = 0.0f;
  const double n = (double)*a.n_tokens;
  const double dbal = a.d_losses != nullptr ? (double)a.d_losses[0] : 0.0;
  const double dz = a.d_losses != nullptr ? (double)a.d_losses[1] : 0.0;
  const float z_of = n > 0.0 ? (float)(2.0 * dz / n) : 0.0f;
  const float c_of = n > 0.0 ? (float)(dbal * E / ((double)k * n * n)) : 0.0f;
  float c[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = H::expert(lane, i);
    c[i] = H::exists(lane, i, E) ? c_of * (float)a.counts[e] : 0.0f;
  }
  __syncthreads();
  for (int64_t t = (int64_t)blockIdx.x * kBwdGroups + group; t < nblk * kBwdGroups;
       t += (int64_t)gridDim.x * kBwdGroups) {
    const bool here = t < a.tokens;
    const float lse = here ? a.lse[t] : -INFINITY;
    const bool live = lse != -INFINITY;
    float f[R];
    if (live) {
      H::load(static_cast<const T *>(a.logits) + t * a.ld, E, lane, f);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) f[i] = -INFINITY;
    }
    int32_t mine = -1;
    float g = 0.0f, dg = 0.0f;
    if (live && lane < k) {
      mine = a.experts[t * k + lane];
      if (mine >= E) mine = -1;
      g = a.gates[t * k + lane];
      dg = mine >= 0 && a.d_gates != nullptr ? a.d_gates[t * k + lane] : 0.0f;
    }
    const float s = row_sum(g * dg);
    if (mine >= 0) s_add[mine] = a.renorm ? g * (dg - s) : g * dg;
    // p as exp(l - lse) over its own sum: lse's rounding, which for large logits
    // is larger than the logits' distances, cancels.  No l exceeds lse, and the
    // largest is within 2 log(experts) of it, so the sum is never lost.
    const float from = live ? lse : 0.0f;
    float sum = 0.0f, pc = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      f[i] = exp_term(f[i], from);
      sum += f[i];
      pc = __builtin_fmaf(f[i], c[i], pc);
    }
    const float inv = live ? 1.0f / row_sum(sum) : 0.0f;
    pc = row_sum(pc) * inv;
    const float shift = (live ? z_of * lse : 0.0f) - pc - (a.renorm ? 0.0f : s);
    // the group's row in LDS is one wave's: its accesses stay in order
    __builtin_amdgcn_wave_barrier();
    if (here) {
      T *out = static_cast<T *>(a.d_logits) + t * E;
#pragma unroll
      for (int i = 0; i < R; i += H::W) {
        constexpr int W = H::W;
        const int e = H::expert(lane, i);
        float d[Elem<T>::V];
        if (W == Elem<T>::V && (FULL || e + W <= E)) {
#pragma unroll
          for (int j = 0; j < W; ++j)
            d[j] = __builtin_fmaf(f[i + j] * inv, c[i + j] + shift, s_add[e + j]);
          *reinterpret_cast<u32x4_any *>(out + e) = Elem<T>::pack(d);
        } else {
#pragma unroll
          for (int j = 0; j < W; ++j)
            if (FULL || e + j < E)
              out[e + j] =
                  Elem<T>::put(__builtin_fmaf(f[i + j] * inv, c[i + j] + shift, s_add[e + j]));
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (mine >= 0) s_add[mine] = 0.0f;
    __builtin_amdgcn_wave_barrier();
  }
}

static size_t route_lds(int r, bool alone, int n_experts) {
  return (size_t)(12 + route_threads(r, alone) / 64 * 4) * (size_t)n_experts;
}

static dim3 route_grid(int64_t nblk, int64_t from) {
  const int64_t left = nblk - from;
  return dim3((unsigned)(left < kRouteGrid ? left : kRouteGrid));
}

template <typename T, int R, bool FULL>
static hipError_t route_fwd(const RouteArgs &a, hipStream_t st) {
  const int64_t nblk = route_blocks(a.tokens);
  RouteWs ws{};
  if (nblk > 1) route_layout(nblk, a.n_experts, a.workspace, &ws);
  if (nblk == 1) {
    hipLaunchKernelGGL((route_kernel<T, R, FULL, true>), dim3(1),
                       dim3(route_threads(R, true)), route_lds(R, true, a.n_experts), st, a, ws,
                       int64_t(0));
    return hipGetLastError();
  }
  // What the choices did not write must not be read: the first launch that fails
  // ends the call.
  for (int64_t b = 0; b < nblk; b += kRouteGrid) {
    hipLaunchKernelGGL((route_kernel<T, R, FULL, false>), route_grid(nblk, b),
                       dim3(route_threads(R, false)), route_lds(R, false, a.n_experts), st, a, ws,
                       b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(route_scan_kernel, dim3((unsigned)(a.n_experts + 2)), dim3(64), 0, st, a, ws,
                     (int)nblk);
  hipError_t e = hipGetLastError();
  for (int64_t b = 0; e == hipSuccess && b < nblk; b += kRouteGrid) {
    hipLaunchKernelGGL(route_place_kernel, route_grid(nblk, b), dim3(256), 0, st, a, ws, b);
    e = hipGetLastError();
  }
  return e;
}

template <typename T, int R, bool FULL>
static hipError_t route_back(const RouteArgs &a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  const int64_t nblk = (a.tokens + kBwdGroups - 1) / kBwdGroups;
  const unsigned grid = (unsigned)(nblk < 2048 ? nblk : 2048);
  hipLaunchKernelGGL((route_bwd_kernel<T, R, FULL>), dim3(grid), dim3(256),
                     (size_t)kBwdGroups * 4u * (size_t)a.n_experts, st, a, nblk);
  return hipGetLastError();
}

// Logits per lane: the smallest power of two that holds the experts.
template <typename T>
static hipError_t route_any(const RouteArgs &a, bool back, hipStream_t st) {
#define UFP4_ROUTE(R)                                                                          \
  if (a.n_experts == 16 * R)                                                                   \
    return back ? route_back<T, R, true>(a, st) : route_fwd<T, R, true>(a, st);                \
  if (a.n_experts < 16 * R) return back ? route_back<T, R, false>(a, st) : route_fwd<T, R, false>(a, st)
  UFP4_ROUTE(1);
  UFP4_ROUTE(2);
  UFP4_ROUTE(4);
  UFP4_ROUTE(8);
  UFP4_ROUTE(16);
  UFP4_ROUTE(32);
  UFP4_ROUTE(64);
#undef UFP4_ROUTE
  return hipErrorInvalidValue;
}

hipError_t launch_route(const RouteArgs &a, hipStream_t st) {
  return a.bf16 ? route_any<uint16_t>(a, false, st) : route_any<float>(a, false, st);
}
hipError_t launch_route_bwd(const RouteArgs &a, hipStream_t st) {
  return a.bf16 ? route_any<uint16_t>(a, true, st) : route_any<float>(a, true, st);
}

}  // namespace ufp4
