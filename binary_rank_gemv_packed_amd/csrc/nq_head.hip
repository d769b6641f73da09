// Norms of queries and keys for each head with the rotation of their positions,
// forward, forward into the cache of keys and values, and backward.  For one head
// of one token, D channels x, weights w, R rotated channels:
//
//   n = x r (w + o),  r = (mean x^2 + eps)^-1/2       (n = x without the norm)
//   (y_a, y_b) = (n_a cos p - n_b sin p, n_a sin p + n_b cos p)  for pair i < R / 2,
//   p = position of the pair's axis times inv_freq[i];  y = n for the other channels.
//
// Pair i is channels (i, i + R / 2), interleaved (2i, 2i + 1).  Backward, from dy:
//   g = dy turned by -p,  dw = sum of g x r over tokens and heads,
//   t = g (w + o),  dx = r (t - x r mean(t x r)).
//
// The angle is formed in 64 bits, in turns, for positions are far (the product's
// rounding is 2^-52 of it); its fraction of a turn, its sine and cosine and all
// other arithmetic are fp32, and each output is rounded once, to its type.
#include "nq_common.h"
#include "nq_internal.h"

#include <type_traits>

namespace nq {

namespace {

typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));

// ------------------------------------------------------------------ lanes
// LG lanes hold one head's D channels as pairs: lane m the pairs VEC m .. VEC m +
// VEC - 1, and with C chunks also those LG VEC further on.  VEC = 4 where 8 divides D
// and R, so that a lane's pairs are all turned or none, and are two runs of four
// channels; VEC = 1 elsewhere.
template <int VEC, int LG, int C>
struct HeadLanes {
  static constexpr int N = VEC * C;  // pairs of a lane
  int m, D, half;                    // half = R / 2
  bool near;                         // interleaved
  __device__ __forceinline__ int pair(int i) const { return (i / VEC * LG + m) * VEC + i % VEC; }
  __device__ __forceinline__ bool in(int i) const { return 2 * pair(i) < D; }
  __device__ __forceinline__ bool turned(int i) const { return pair(i) < half; }
  // the channels of pair i
  __device__ __forceinline__ int first(int i) const { return near || !turned(i) ? 2 * pair(i) : pair(i); }
  __device__ __forceinline__ int second(int i) const { return near || !turned(i) ? 2 * pair(i) + 1 : pair(i) + half; }
};

template <typename T>
__device__ __forceinline__ float head_get(const T* p, int k) {
  return to_f32<T>(p[k]);
}

// Four elements from channel k on.
__device__ __forceinline__ void four(const float* p, int k, float* v) {
  const u32x4_at2 u = *reinterpret_cast<const u32x4_at2*>(p + k);
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void four(const uint16_t* p, int k, float* v) {
  const u32x2_at2 u = *reinterpret_cast<const u32x2_at2*>(p + k);
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
}
__device__ __forceinline__ void four(const _Float16* p, int k, float* v) {
  const u32x2_at2 u = *reinterpret_cast<const u32x2_at2*>(p + k);
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[i / 2] >> (16 * (i & 1))));
}
__device__ __forceinline__ void put_four(float* p, int k, const float* v) {
  u32x4_at2 u;
#pragma unroll
  for (int i = 0; i < 4; i++) u[i] = __float_as_uint(v[i]);
  *reinterpret_cast<u32x4_at2*>(p + k) = u;
}
__device__ __forceinline__ void put_four(uint16_t* p, int k, const float* v) {
  u32x2_at2 u;
#pragma unroll
  for (int i = 0; i < 2; i++) u[i] = f32_to_bf16(v[2 * i]) | (uint32_t)f32_to_bf16(v[2 * i + 1]) << 16;
  *reinterpret_cast<u32x2_at2*>(p + k) = u;
}
__device__ __forceinline__ void put_one(float* p, int k, float v) { p[k] = v; }
__device__ __forceinline__ void put_one(uint16_t* p, int k, float v) { p[k] = f32_to_bf16(v); }

// A lane's pairs of one head: v[i] and v[N + i] are the two members of pair i;
// zeros behind D and where there is no head (p null).
template <int VEC, int LG, int C, typename T>
__device__ __forceinline__ void head_load(const HeadLanes<VEC, LG, C>& l, const T* p, float (&v)[2 * VEC * C]) {
  constexpr int N = VEC * C;
  if constexpr (VEC == 4) {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = 0.0f;
    if (p && l.in(0)) {
      const bool near = l.near || !l.turned(0);
      float a[4], b[4];
      four(p, l.first(0), a);
      four(p, near ? l.first(0) + 4 : l.second(0), b);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[i] = near ? (i < 2 ? a[2 * i] : b[2 * i - 4]) : a[i];
        v[4 + i] = near ? (i < 2 ? a[2 * i + 1] : b[2 * i - 3]) : b[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const bool on = p && l.in(i);
      v[i] = on ? head_get(p, l.first(i)) : 0.0f;
      v[N + i] = on ? head_get(p, l.second(i)) : 0.0f;
    }
  }
}

template <int VEC, int LG, int C, typename T>
__device__ __forceinline__ void head_put(const HeadLanes<VEC, LG, C>& l, T* p, const float (&v)[2 * VEC * C]) {
  constexpr int N = VEC * C;
  if constexpr (VEC == 4) {
    if (!l.in(0)) return;
    const bool near = l.near || !l.turned(0);
    float a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      a[i] = near ? v[(i & 1) * 4 + i / 2] : v[i];
      b[i] = near ? v[(i & 1) * 4 + 2 + i / 2] : v[4 + i];
    }
    put_four(p, l.first(0), a);
    put_four(p, near ? l.first(0) + 4 : l.second(0), b);
  } else {
#pragma unroll
    for (int i = 0; i < N; i++)
      if (l.in(i)) {
        put_one(p, l.first(i), v[i]);
        put_one(p, l.second(i), v[N + i]);
      }
  }
}

// The weights plus their offset, or ones.
template <int VEC, int LG, int C>
__device__ __forceinline__ void head_weights(const HeadLanes<VEC, LG, C>& l, const HeadArgs& a, const void* w,
                                             float (&v)[2 * VEC * C]) {
  if (!w || !a.norm) {
#pragma unroll
    for (int i = 0; i < 2 * VEC * C; i++) v[i] = 1.0f;
    return;
  }
  if (a.param_dtype == 0) head_load(l, static_cast<const float*>(w), v);
  else if (a.param_dtype == 1) head_load(l, static_cast<const _Float16*>(w), v);
  else head_load(l, static_cast<const uint16_t*>(w), v);
#pragma unroll
  for (int i = 0; i < 2 * VEC * C; i++) v[i] += a.weight_offset;
}

// Sine and cosine of a lane's pairs at token t.
template <int VEC, int LG, int C>
__device__ __forceinline__ void head_angles(const HeadLanes<VEC, LG, C>& l, const HeadArgs& a, int t,
                                            float (&c)[VEC * C], float (&s)[VEC * C]) {
#pragma unroll
  for (int i = 0; i < VEC * C; i++) {
    c[i] = 1.0f;
    s[i] = 0.0f;
    if (l.turned(i)) {
      const int p = l.pair(i);
      const int axis = (p >= a.end[0]) + (p >= a.end[1]) + (p >= a.end[2]);
      double u = (double)a.positions[(size_t)axis * a.tokens + t] * a.inv_freq[p] * 0.15915494309189533577;
      u -= rint(u);
      sincospif((float)(2.0 * u), &s[i], &c[i]);
    }
  }
}

// Sum over the LG lanes of a head, to each of them, in a fixed order.
template <int LG>
__device__ __forceinline__ float head_sum(float v) {
#define NQ_DPP_ADD(ctrl) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, false))
  NQ_DPP_ADD(0xB1);                           // lane ^ 1
  NQ_DPP_ADD(0x4E);                           // lane ^ 2
  if constexpr (LG >= 8) NQ_DPP_ADD(0x141);   // the other four of eight
  if constexpr (LG >= 16) NQ_DPP_ADD(0x140);  // the other eight of sixteen
#undef NQ_DPP_ADD
  if constexpr (LG >= 32) v += __shfl_xor(v, 16);
  if constexpr (LG >= 64) v += __shfl_xor(v, 32);
  return v;
}

__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const uint16_t*) { return to_f32<uint16_t>(f32_to_bf16(v)); }

// ------------------------------------------------------------------ forward
// A wave takes one token, or one of `parts` shares of a token's heads, so that the
// angles are formed once for all of them; 64 / LG heads at a time, the next ones
// asked for before the present ones are worked on.  Heads are numbered q, k, and with a
// cache (KIND >= 0) v; keys and values then pass through shared memory to lanes of eight
// channels each, as the cache's stores take them, after the rounding to T that k_out
// would have had: the cache holds what a write of k_out would have put there.
template <typename T, int VEC, int LG, int C, int KIND>
__global__ void __launch_bounds__(256) head_fwd_kernel(HeadArgs a, int parts) {
  constexpr int N = VEC * C, SLOTS = 64 / LG;
  constexpr bool WRITE = KIND >= 0;
  __shared__ float turn_over[WRITE ? 4 * 512 : 1];
  const int lane = threadIdx.x & 63, slot = lane / LG;
  const long long job = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
  const bool on = job < (long long)a.tokens * parts;
  const int t = on ? (int)(job / parts) : 0, part = (int)(job % parts);
  const HeadLanes<VEC, LG, C> l{lane % LG, a.D, a.rot / 2, a.interleaved};
  const int heads = a.q_heads + a.k_heads * (WRITE ? 2 : 1), step = parts * SLOTS;
  auto row = [&](int u) -> const T* {
    if (!on || u >= heads) return nullptr;
    if (u < a.q_heads) return static_cast<const T*>(a.q) + t * a.q_stride + (size_t)u * a.D;
    u -= a.q_heads;
    if (u < a.k_heads) return static_cast<const T*>(a.k) + t * a.k_stride + (size_t)u * a.D;
    return static_cast<const T*>(a.v) + t * a.v_stride + (size_t)(u - a.k_heads) * a.D;
  };
  float next[2 * N], wq[2 * N], wk[2 * N], c[N], s[N];
  head_load(l, row(part * SLOTS + slot), next);
  head_weights(l, a, a.w_q, wq);
  head_weights(l, a, a.w_k, wk);
  KvPlace at{nullptr, 0, 0};
  if (WRITE && on) at = kv_place(a.cache, a.data, a.slots[t]);
  head_angles(l, a, t, c, s);
  const int rounds = ceil_div(heads, step);  // the same in every wave, for the barriers
  for (int k = 0; k < rounds; k++) {
    const int u = part * SLOTS + slot + k * step;
    float x[2 * N], y[2 * N];
#pragma unroll
    for (int i = 0; i < 2 * N; i++) x[i] = next[i];
    if (k + 1 < rounds) head_load(l, row(u + step), next);
    const bool is_q = u < a.q_heads, is_v = WRITE && u >= a.q_heads + a.k_heads;
    float r = 1.0f;
    if (a.norm) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * N; i++) ss = fmaf(x[i], x[i], ss);
      r = 1.0f / sqrtf(head_sum<LG>(ss) / (float)a.D + a.eps);
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
      const float na = a.norm ? x[i] * r * (is_q ? wq[i] : wk[i]) : x[i];
      const float nb = a.norm ? x[N + i] * r * (is_q ? wq[N + i] : wk[N + i]) : x[N + i];
      const bool turn = l.turned(i);
      y[i] = turn ? na * c[i] - nb * s[i] : na;
      y[N + i] = turn ? na * s[i] + nb * c[i] : nb;
    }
    if (on && is_q) head_put(l, static_cast<T*>(a.q_out) + ((size_t)t * a.q_heads + u) * a.D, y);
    if constexpr (!WRITE) {
      if (on && !is_q && u < heads) head_put(l, static_cast<T*>(a.k_out) + ((size_t)t * a.k_heads + u - a.q_heads) * a.D, y);
    } else {
      __syncthreads();
      float* mine = turn_over + (threadIdx.x >> 6) * 512 + slot * a.D;
#pragma unroll
      for (int i = 0; i < N; i++)
        if (l.in(i)) {
          mine[l.first(i)] = is_v ? x[i] : round_to(y[i], (const T*)nullptr);
          mine[l.second(i)] = is_v ? x[N + i] : round_to(y[N + i], (const T*)nullptr);
        }
      __syncthreads();
      const bool held = on && !is_q && u < heads && 8 * l.m < a.D;
      float e[8] = {};
      if (held) {
#pragma unroll
        for (int i = 0; i < 8; i++) e[i] = mine[8 * l.m + i];
      }
      const int head = u - a.q_heads - (is_v ? a.k_heads : 0);
      // whole waves go through either store: its exchanges want every lane of a head
      if (__any(held && !is_v)) kv_store<KIND, LG, false>(a.cache, at, held ? head : 0, l.m, held && !is_v, e);
      if (__any(held && is_v)) kv_store<KIND, LG, true>(a.cache, at, held ? head : 0, l.m, held && is_v, e);
    }
  }
}

// ------------------------------------------------------------------ backward
// Shares of tokens as in the forward; the waves of the grid take them in turn.  The
// sums for both weights stay in registers over all of a wave's tokens and are joined
// over a head's slots, the workgroup's waves and (head_join_kernel) the workgroups in
// a fixed order.
template <typename T, int VEC, int LG, int C>
__global__ void __launch_bounds__(1024) head_bwd_kernel(HeadArgs a, int parts) {
  constexpr int N = VEC * C, SLOTS = 64 / LG;
  __shared__ float red[16][HEAD_MAX_DIM];
  const int lane = threadIdx.x & 63, slot = lane / LG, wave = threadIdx.x >> 6;
  const HeadLanes<VEC, LG, C> l{lane % LG, a.D, a.rot / 2, a.interleaved};
  float sums[2][2 * N];
#pragma unroll
  for (int i = 0; i < 2 * N; i++) sums[0][i] = sums[1][i] = 0.0f;
  const long long jobs = (long long)a.tokens * parts;
  for (long long job = (long long)blockIdx.x * 16 + wave; job < jobs; job += (long long)gridDim.x * 16) {
    const int t = (int)(job / parts), part = (int)(job % parts);
    float c[N], s[N];
    head_angles(l, a, t, c, s);
#pragma unroll
    for (int kind = 0; kind < 2; kind++) {
      const int heads = kind ? a.k_heads : a.q_heads, step = parts * SLOTS;
      const T* xs = kind ? static_cast<const T*>(a.k) + t * a.k_stride : static_cast<const T*>(a.q) + t * a.q_stride;
      const T* gs = static_cast<const T*>(kind ? a.dk : a.dq) + (size_t)t * heads * a.D;
      T* out = static_cast<T*>(kind ? a.k_out : a.q_out) + (size_t)t * heads * a.D;
      float w[2 * N], x[2 * N], d[2 * N];
      if (part * SLOTS < heads) {
        const int u = part * SLOTS + slot;
        head_load(l, a.norm && u < heads ? xs + (size_t)u * a.D : nullptr, x);
        head_load(l, u < heads ? gs + (size_t)u * a.D : nullptr, d);
        head_weights(l, a, kind ? a.w_k : a.w_q, w);
      }
      for (int base = part * SLOTS; base < heads; base += step) {
        const int u = base + slot;
        float g[2 * N], n[2 * N];
#pragma unroll
        for (int i = 0; i < N; i++) {
          const bool turn = l.turned(i);
          g[i] = turn ? d[i] * c[i] + d[N + i] * s[i] : d[i];
          g[N + i] = turn ? d[N + i] * c[i] - d[i] * s[i] : d[N + i];
          n[i] = x[i];
          n[N + i] = x[N + i];
        }
        if (base + step < heads) {
          const int v = u + step;
          head_load(l, a.norm && v < heads ? xs + (size_t)v * a.D : nullptr, x);
          head_load(l, v < heads ? gs + (size_t)v * a.D : nullptr, d);
        }
        if (a.norm) {
          float ss = 0.0f, dot = 0.0f;
#pragma unroll
          for (int i = 0; i < 2 * N; i++) ss = fmaf(n[i], n[i], ss);
          const float r = 1.0f / sqrtf(head_sum<LG>(ss) / (float)a.D + a.eps);
#pragma unroll
          for (int i = 0; i < 2 * N; i++) {
            n[i] *= r;
            sums[kind][i] = fmaf(g[i], n[i], sums[kind][i]);
            g[i] *= w[i];
            dot = fmaf(g[i], n[i], dot);
          }
          const float mean = head_sum<LG>(dot) / (float)a.D;
#pragma unroll
          for (int i = 0; i < 2 * N; i++) g[i] = r * (g[i] - n[i] * mean);
        }
        if (u < heads) head_put(l, out + (size_t)u * a.D, g);
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int kind = 0; kind < 2; kind++) {
#pragma unroll
    for (int i = 0; i < 2 * N; i++) {
#pragma unroll
      for (int o = LG; o < 64; o *= 2) sums[kind][i] += __shfl_xor(sums[kind][i], o);
    }
    __syncthreads();
    if (slot == 0) {
#pragma unroll
      for (int i = 0; i < N; i++)
        if (l.in(i)) {
          red[wave][l.first(i)] = sums[kind][i];
          red[wave][l.second(i)] = sums[kind][N + i];
        }
    }
    __syncthreads();
    if ((int)threadIdx.x < a.D) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; i++) v += red[i][threadIdx.x];
      a.part[((size_t)blockIdx.x * 2 + kind) * a.D + threadIdx.x] = v;
    }
  }
}

// Sums of the workgroups' sums: 64 channels of one weight (blockIdx.y) a workgroup,
// wave w the parts w, w + 16, ...
__global__ void __launch_bounds__(1024) head_join_kernel(HeadArgs a, int blocks) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (col < a.D) {
#pragma unroll 8
    for (int k = w; k < blocks; k += 16) s += a.part[((size_t)k * 2 + blockIdx.y) * a.D + col];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w || col >= a.D) return;
#pragma unroll
  for (int i = 1; i < 16; i++) s += red[i][lane];
  float* to = blockIdx.y ? a.dw_k : a.dw_q;
  if (to) to[col] = s;
}

// ------------------------------------------------------------------ host
// Calls f with the type and the lanes of a head.
template <typename F>
void head_dispatch(const HeadArgs& a, F f) {
  auto by_lanes = [&](auto t) {
    using One = std::integral_constant<int, 1>;
    using Four = std::integral_constant<int, 4>;
    if (a.D % 8 == 0 && a.rot % 8 == 0) {
      if (a.D <= 64) f(t, Four{}, std::integral_constant<int, 8>{}, One{});
      else if (a.D <= 128) f(t, Four{}, std::integral_constant<int, 16>{}, One{});
      else if (a.D <= 256) f(t, Four{}, std::integral_constant<int, 32>{}, One{});
      else f(t, Four{}, std::integral_constant<int, 64>{}, One{});
    } else if (a.D <= 128) {
      f(t, One{}, std::integral_constant<int, 64>{}, One{});
    } else {
      f(t, One{}, std::integral_constant<int, 64>{}, Four{});
    }
  };
  if (a.act_dtype == 0) by_lanes(float{});
  else by_lanes(uint16_t{});
}

// Shares of a token's heads: enough that `waves` waves have work, at most one for
// each round of heads.
int head_parts(int tokens, int heads, int slots, int waves) {
  const int most = ceil_div(heads, slots), want = ceil_div(waves, tokens);
  return want < 1 ? 1 : want < most ? want : most;
}

template <typename Kind>
hipError_t head_launch(const HeadArgs& a, Kind) {
  constexpr int KIND = Kind::value;
  head_dispatch(a, [&](auto t, auto vec, auto lg, auto c) {
    constexpr int LG = decltype(lg)::value, VEC = decltype(vec)::value, C = decltype(c)::value;
    if constexpr (KIND < 0 || VEC == 1 || LG < 64) {  // a cache's heads have 256 channels at most
      const int parts = head_parts(a.tokens, a.q_heads + a.k_heads * (KIND < 0 ? 1 : 2), 64 / LG, 2048);
      const long long jobs = (long long)a.tokens * parts;
      hipLaunchKernelGGL((head_fwd_kernel<decltype(t), VEC, LG, C, KIND>), dim3((unsigned)((jobs + 3) / 4)), dim3(256), 0,
                         a.stream, a, parts);
    }
  });
  return hipGetLastError();
}

}  // namespace

int head_bwd_parts(int tokens) { return tokens ? 256 : 0; }

hipError_t head_forward(const HeadArgs& a) { return head_launch(a, std::integral_constant<int, -1>{}); }

hipError_t head_write(const HeadArgs& a) {
  if (a.cache.kind == KV_BF16) return head_launch(a, std::integral_constant<int, KV_BF16>{});
  if (a.cache.kind == KV_INT8) return head_launch(a, std::integral_constant<int, KV_INT8>{});
  return head_launch(a, std::integral_constant<int, KV_INT4>{});
}

hipError_t head_backward(const HeadArgs& a) {
  int blocks = 0;
  if (a.tokens) {
    head_dispatch(a, [&](auto t, auto vec, auto lg, auto c) {
      constexpr int LG = decltype(lg)::value;
      const int heads = a.q_heads > a.k_heads ? a.q_heads : a.k_heads;
      const int parts = head_parts(a.tokens, heads, 64 / LG, 4096);
      const long long jobs = (long long)a.tokens * parts;
      blocks = (int)(jobs < 256 * 16 ? (jobs + 15) / 16 : 256);
      hipLaunchKernelGGL((head_bwd_kernel<decltype(t), decltype(vec)::value, LG, decltype(c)::value>), dim3(blocks),
                         dim3(1024), 0, a.stream, a, parts);
    });
  }
  if (a.part || !a.tokens) hipLaunchKernelGGL(head_join_kernel, dim3(ceil_div(a.D, 64), 2), dim3(1024), 0, a.stream, a, blocks);
  return hipGetLastError();
}

}  // namespace nq
