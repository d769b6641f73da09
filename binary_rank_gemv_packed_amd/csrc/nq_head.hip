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
// rounding is 2^-52 of it), and in the forward so are its sine and cosine, rounded to fp32
// (once a wave and pair: formed in fp32 they would cost an output another 2^-24 here and
// there, which turns some of its bf16 roundings).  All other arithmetic is fp32, and each
// output is rounded once, to its type.
#include "nq_common.h"
#include "nq_internal.h"

#include <type_traits>

namespace nq {

namespace {

typedef uint32_t u32x1_at2 __attribute__((ext_vector_type(1), aligned(2)));
typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));

// ------------------------------------------------------------------ lanes
// LG lanes hold one head's D channels as pairs: lane m the pairs VEC m .. VEC m +
// VEC - 1, and with C chunks also those LG VEC further on.  VEC = 4 or 2 where 2 VEC
// divides D and R (R only where members of a pair are R / 2 apart), so that a lane's pairs are two
// runs of VEC channels; VEC = 1 elsewhere: 2048 tokens of 64 + 8 heads of 100 in bf16 21.6 us
// with 2 and 33.8 with 1 (backward 29.3 and 43.8), of 96 15.9 with 4.
template <int VEC, int LG, int C>
struct HeadLanes {
  static constexpr int N = VEC * C;  // pairs of a lane
  int m, D, half;                    // half = R / 2
  bool near;                         // interleaved
  __device__ __forceinline__ int pair(int i) const { return (i / VEC * LG + m) * VEC + i % VEC; }
  __device__ __forceinline__ bool in(int i) const { return 2 * pair(i) < D; }
  __device__ __forceinline__ bool turned(int i) const { return pair(i) < half; }
  __device__ __forceinline__ bool beside() const { return near || !turned(0); }  // members of pairs lie side by side
  // the channels of pair i
  __device__ __forceinline__ int first(int i) const { return near || !turned(i) ? 2 * pair(i) : pair(i); }
  __device__ __forceinline__ int second(int i) const { return near || !turned(i) ? 2 * pair(i) + 1 : pair(i) + half; }
};

// VEC elements, and a lane's pairs of one head as they are stored, until get(): what
// is asked for early takes no more registers than its bytes.
template <typename T, int VEC>
struct Run {
  static constexpr int WORDS = VEC * (int)sizeof(T) / 4;
  typedef typename std::conditional<WORDS == 4, u32x4_at2, typename std::conditional<WORDS == 2, u32x2_at2, u32x1_at2>::type>::type word;
  word u;
  __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const word*>(p); }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[i]);
    else if constexpr (std::is_same<T, _Float16>::value)
      return (float)__builtin_bit_cast(_Float16, (uint16_t)(u[i / 2] >> (16 * (i & 1))));
    else return __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  }
};

template <int VEC, typename T>
__device__ __forceinline__ void put_run(T* p, const float* v) {
  typename Run<T, VEC>::word u;
#pragma unroll
  for (int i = 0; i < Run<T, VEC>::WORDS; i++) {
    if constexpr (sizeof(T) == 4) u[i] = __float_as_uint(v[i]);
    else u[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  }
  *reinterpret_cast<typename Run<T, VEC>::word*>(p) = u;
}
__device__ __forceinline__ void put_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_one(uint16_t* p, float v) { *p = f32_to_bf16(v); }

// Element `k` of a row as a byte offset of 32 bits from the row's address, which is the
// same for the wave.
template <typename T>
__device__ __forceinline__ T* head_at(T* row, uint32_t k) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type byte;
  return reinterpret_cast<T*>(reinterpret_cast<byte*>(row) + k * (uint32_t)sizeof(T));
}

// A lane's pairs of one head that begins at element k of a row: zeros behind D and
// where `on` is false.  get() gives v[i] and v[N + i], the two members of pair i.
template <typename T, int VEC, int LG, int C>
struct HeadRow {
  static constexpr int N = VEC * C;
  Run<T, VEC == 1 ? 4 : VEC> a, b;  // VEC > 1
  T one[VEC == 1 ? 2 * N : 1];
  __device__ __forceinline__ void load(const HeadLanes<VEC, LG, C>& l, const T* row, uint32_t k, bool on) {
    if constexpr (VEC > 1) {
#pragma unroll
      for (int i = 0; i < Run<T, VEC>::WORDS; i++) a.u[i] = b.u[i] = 0;
      if (on && l.in(0)) {
        a.load(head_at(row, k + l.first(0)));
        b.load(head_at(row, k + (l.beside() ? l.first(0) + VEC : l.second(0))));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; i++) {
        one[i] = one[N + i] = T(0);
        if (on && l.in(i)) {
          one[i] = *head_at(row, k + l.first(i));
          one[N + i] = *head_at(row, k + l.second(i));
        }
      }
    }
  }
  __device__ __forceinline__ void get(const HeadLanes<VEC, LG, C>& l, float (&v)[2 * N]) const {
    if constexpr (VEC > 1) {
      const bool beside = l.beside();
#pragma unroll
      for (int i = 0; i < VEC; i++) {
        v[i] = beside ? (2 * i < VEC ? a.get(2 * i) : b.get(2 * i - VEC)) : a.get(i);
        v[VEC + i] = beside ? (2 * i < VEC ? a.get(2 * i + 1) : b.get(2 * i + 1 - VEC)) : b.get(i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * N; i++) v[i] = to_f32<T>(one[i]);
    }
  }
};

template <int VEC, int LG, int C, typename T>
__device__ __forceinline__ void head_put(const HeadLanes<VEC, LG, C>& l, T* row, uint32_t k, const float (&v)[2 * VEC * C]) {
  constexpr int N = VEC * C;
  if constexpr (VEC > 1) {
    if (!l.in(0)) return;
    const bool beside = l.beside();
    float a[VEC], b[VEC];
#pragma unroll
    for (int i = 0; i < VEC; i++) {
      a[i] = beside ? v[(i & 1) * VEC + i / 2] : v[i];
      b[i] = beside ? v[(i & 1) * VEC + VEC / 2 + i / 2] : v[VEC + i];
    }
    put_run<VEC>(head_at(row, k + l.first(0)), a);
    put_run<VEC>(head_at(row, k + (beside ? l.first(0) + VEC : l.second(0))), b);
  } else {
#pragma unroll
    for (int i = 0; i < N; i++)
      if (l.in(i)) {
        put_one(head_at(row, k + l.first(i)), v[i]);
        put_one(head_at(row, k + l.second(i)), v[N + i]);
      }
  }
}

// The weights plus their offset, or ones: asked for by load(), so that nothing waits for
// them before it has to.
template <int VEC, int LG, int C>
struct HeadWeights {
  HeadRow<float, VEC, LG, C> wide;
  HeadRow<uint16_t, VEC, LG, C> narrow;
  int dtype;  // -1: none
  __device__ __forceinline__ void load(const HeadLanes<VEC, LG, C>& l, const HeadArgs& a, const void* w) {
    dtype = w && a.norm ? a.param_dtype : -1;
    if (dtype == 0) wide.load(l, static_cast<const float*>(w), 0, true);
    else if (dtype > 0) narrow.load(l, static_cast<const uint16_t*>(w), 0, true);
  }
  __device__ __forceinline__ void get(const HeadLanes<VEC, LG, C>& l, float offset, float (&v)[2 * VEC * C]) const {
    if (dtype == 0) {
      wide.get(l, v);
    } else if (dtype == 1) {
      HeadRow<_Float16, VEC, LG, C> half;
      if constexpr (VEC > 1) {
        half.a.u = narrow.a.u;
        half.b.u = narrow.b.u;
      } else {
#pragma unroll
        for (int i = 0; i < 2 * VEC * C; i++) half.one[i] = __builtin_bit_cast(_Float16, narrow.one[i]);
      }
      half.get(l, v);
    } else if (dtype == 2) {
      narrow.get(l, v);
    }
#pragma unroll
    for (int i = 0; i < 2 * VEC * C; i++) v[i] = dtype < 0 ? 1.0f : v[i] + offset;
  }
};

// The same at once.
template <int VEC, int LG, int C>
__device__ __forceinline__ void head_weights(const HeadLanes<VEC, LG, C>& l, const HeadArgs& a, const void* w,
                                             float (&v)[2 * VEC * C]) {
  const int dtype = w && a.norm ? a.param_dtype : -1;
  auto as = [&](auto t) {
    HeadRow<decltype(t), VEC, LG, C> r;
    r.load(l, static_cast<const decltype(t)*>(w), 0, true);
    r.get(l, v);
  };
  if (dtype == 0) as(float{});
  else if (dtype == 1) as(_Float16{});
  else if (dtype == 2) as(uint16_t{});
#pragma unroll
  for (int i = 0; i < 2 * VEC * C; i++) v[i] = dtype < 0 ? 1.0f : v[i] + a.weight_offset;
}

// Orders a wave's accesses to shared memory between its lanes: LDS takes them in turn.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Cosines and sines of one token.  A wave's lanes form one pair's each (those of one
// head's, where its slots would form them again for every head): load() asks for what
// they are made of, get() makes them and passes them on through `shared`, the wave's
// own 2 x (LG VEC C) floats.  WIDE: in 64 bits, for the forward; the backward pass has no
// registers for it.
template <int VEC, int LG, int C, bool WIDE>
struct HeadAngles {
  static constexpr int N = LG * VEC * C, EACH = (N + 63) / 64;
  int64_t position[EACH];
  double freq[EACH];
  __device__ __forceinline__ void load(const HeadLanes<VEC, LG, C>& l, const HeadArgs& a, int t) {
#pragma unroll
    for (int i = 0; i < EACH; i++) {
      const int p = 64 * i + (threadIdx.x & 63);
      position[i] = 0;
      freq[i] = 0.0;
      if (p < l.half) {
        const int axis = (p >= a.end[0]) + (p >= a.end[1]) + (p >= a.end[2]);
        position[i] = a.positions[(size_t)axis * a.tokens + t];
        freq[i] = a.inv_freq[p];
      }
    }
  }
  __device__ __forceinline__ void get(const HeadLanes<VEC, LG, C>& l, float* shared, float (&c)[VEC * C], float (&s)[VEC * C]) const {
#pragma unroll
    for (int i = 0; i < EACH; i++) {
      const int p = 64 * i + (threadIdx.x & 63);
      if (64 * i >= l.half) break;
      double u = (double)position[i] * freq[i] * 0.15915494309189533577;
      u -= rint(u);
      float sine, cosine;
      if constexpr (WIDE) {
        double sine64, cosine64;
        sincospi(2.0 * u, &sine64, &cosine64);
        sine = (float)sine64;
        cosine = (float)cosine64;
      } else {  // of the rounded angle, turned by what the rounding left
        const float half = (float)(2.0 * u), rest = (float)(2.0 * u - (double)half) * 3.14159265f;
        float s0, c0;
        sincospif(half, &s0, &c0);
        sine = fmaf(rest, c0, s0);
        cosine = fmaf(-rest, s0, c0);
      }
      if (p < l.half) {
        shared[p] = cosine;
        shared[N + p] = sine;
      }
    }
    wave_fence();
#pragma unroll
    for (int i = 0; i < VEC * C; i++) {
      c[i] = 1.0f;
      s[i] = 0.0f;
      if (l.turned(i)) {
        c[i] = shared[l.pair(i)];
        s[i] = shared[N + l.pair(i)];
      }
    }
    wave_fence();
  }
};

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
// Bound by memory where there are many tokens: 2048 of 64 + 8 heads of 128 in bf16 16.5 us
// (4.6 TB/s), 30 us with an angle formed for every head; one token takes 3.5 us in a
// graph, of which one access and the launch are some three.
// A wave takes one token, or one of `parts` shares of a token's heads, so that the
// angles are formed once for all of them; 64 / LG heads a round, the next round's
// asked for before the present one's are worked on.  A round's heads are all queries, all
// keys or, with a cache (KIND >= 0), all values.  Keys and values then pass through
// shared memory to lanes of eight channels each, as the cache's stores take them, after
// the rounding to T that k_out would have had: the cache holds what a write of k_out
// would have put there.
template <typename T, int VEC, int LG, int C, int KIND>
__global__ void __launch_bounds__(256) head_fwd_kernel(HeadArgs a, int parts) {
  constexpr int N = VEC * C, SLOTS = 64 / LG;
  constexpr bool WRITE = KIND >= 0;
  __shared__ float turns[4][2 * LG * N];
  __shared__ float turn_over[4][WRITE ? 512 : 1];
  const int lane = threadIdx.x & 63, slot = lane / LG, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long long job = (long long)blockIdx.x * 4 + wave;
  if (job >= (long long)a.tokens * parts) return;
  const int t = (int)(job / parts), part = (int)(job % parts);
  const HeadLanes<VEC, LG, C> l{lane % LG, a.D, a.rot / 2, a.interleaved};
  const int rq = (a.q_heads + SLOTS - 1) / SLOTS, rk = (a.k_heads + SLOTS - 1) / SLOTS, rounds = rq + (WRITE ? 2 : 1) * rk;
  auto fetch = [&](HeadRow<T, VEC, LG, C>& to, int r) {
    const int kind = (r >= rq) + (r >= rq + rk);
    const T* row = static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                   t * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride);
    const int u = (r - (kind ? rq : 0) - (kind == 2 ? rk : 0)) * SLOTS + slot;
    to.load(l, row, u * a.D, u < (kind ? a.k_heads : a.q_heads));
  };
  HeadRow<T, VEC, LG, C> next;
  HeadAngles<VEC, LG, C, true> angles;
  HeadWeights<VEC, LG, C> wq, wk;
  const int last = part + (rounds - 1 - part) / parts * parts;  // keys there, or not at all
  angles.load(l, a, t);
  int64_t in = -1;
  if (WRITE && last >= rq) in = a.slots[t];
  fetch(next, part);
  if (part < rq) wq.load(l, a, a.w_q);
  if (last >= rq) wk.load(l, a, a.w_k);
  float c[N], s[N], w[2 * N];
  angles.get(l, turns[wave], c, s);
  const KvPlace at = WRITE && last >= rq ? kv_place(a.cache, a.data, in) : KvPlace{nullptr, 0, 0};
  bool keys = part >= rq;
  if (keys) wk.get(l, a.weight_offset, w);
  else wq.get(l, a.weight_offset, w);
  for (int k = part; k < rounds; k += parts) {
    if (!keys && k >= rq) {
      keys = true;
      wk.get(l, a.weight_offset, w);
    }
    const int kind = (k >= rq) + (k >= rq + rk), u = (k - (kind ? rq : 0) - (kind == 2 ? rk : 0)) * SLOTS + slot;
    const bool on = u < (kind ? a.k_heads : a.q_heads);
    float x[2 * N], y[2 * N];
    next.get(l, x);
    if (k + parts < rounds) fetch(next, k + parts);
    float r = 1.0f;
    if (a.norm && !(WRITE && kind == 2)) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * N; i++) ss = fmaf(x[i], x[i], ss);
      r = 1.0f / sqrtf(head_sum<LG>(ss) / (float)a.D + a.eps);
#pragma unroll
      for (int i = 0; i < 2 * N; i++) y[i] = x[i] * r * w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 2 * N; i++) y[i] = x[i];
    }
    if (!(WRITE && kind == 2)) {
#pragma unroll
      for (int i = 0; i < N; i++) {
        const float na = y[i], nb = y[N + i];
        const bool turn = l.turned(i);
        y[i] = turn ? na * c[i] - nb * s[i] : na;
        y[N + i] = turn ? na * s[i] + nb * c[i] : nb;
      }
    }
    if (kind == 0) {
      if (on) head_put(l, static_cast<T*>(a.q_out) + (size_t)t * a.q_heads * a.D, u * a.D, y);
    } else if constexpr (!WRITE) {
      if (on) head_put(l, static_cast<T*>(a.k_out) + (size_t)t * a.k_heads * a.D, u * a.D, y);
    } else {
      float* mine = turn_over[wave] + slot * a.D;
      wave_fence();
#pragma unroll
      for (int i = 0; i < N; i++)
        if (l.in(i)) {
          mine[l.first(i)] = round_to(y[i], (const T*)nullptr);
          mine[l.second(i)] = round_to(y[N + i], (const T*)nullptr);
        }
      wave_fence();
      const bool held = on && 8 * l.m < a.D;
      float e[8] = {};
      if (held) {
#pragma unroll
        for (int i = 0; i < 8; i++) e[i] = mine[8 * l.m + i];
      }
      if (kind == 1) kv_store<KIND, LG, false>(a.cache, at, held ? u : 0, l.m, held, e);
      else kv_store<KIND, LG, true>(a.cache, at, held ? u : 0, l.m, held, e);
    }
  }
}

// ------------------------------------------------------------------ backward
// Shares of tokens as in the forward; the waves of the grid take them in turn.  The
// sums for both weights stay in registers over all of a wave's tokens and are joined
// over a head's slots, the workgroup's waves and (head_join_kernel) the workgroups in
// a fixed order.  Bound by memory: 4096 tokens of 64 + 8 heads of 128 in bf16 47 us (4.8
// TB/s) and the join 4 us.  Odd heads above 128 channels (C = 4) take eight waves a
// workgroup, which may have 256 registers each: 2048 tokens of 24 heads of 510 in fp32 75 us, where
// sixteen with 128 registers spill 300 bytes a lane and take 90.
constexpr int head_bwd_waves(int C) { return C == 4 ? 8 : 16; }
template <typename T, int VEC, int LG, int C>
__global__ void __launch_bounds__(64 * head_bwd_waves(C)) head_bwd_kernel(HeadArgs a, int parts) {
  constexpr int N = VEC * C, SLOTS = 64 / LG, TURNS = 2 * LG * N, WAVES = head_bwd_waves(C);
  __shared__ float red[WAVES][TURNS > HEAD_MAX_DIM ? TURNS : HEAD_MAX_DIM];  // first the waves' angles, then their sums
  const int lane = threadIdx.x & 63, slot = lane / LG, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const HeadLanes<VEC, LG, C> l{lane % LG, a.D, a.rot / 2, a.interleaved};
  float sums[2][2 * N];
#pragma unroll
  for (int i = 0; i < 2 * N; i++) sums[0][i] = sums[1][i] = 0.0f;
  const long long jobs = (long long)a.tokens * parts;
  for (long long job = (long long)blockIdx.x * WAVES + wave; job < jobs; job += (long long)gridDim.x * WAVES) {
    const int t = (int)(job / parts), part = (int)(job % parts);
    float c[N], s[N];
    HeadAngles<VEC, LG, C, false> angles;
    angles.load(l, a, t);
    angles.get(l, red[wave], c, s);
#pragma unroll
    for (int kind = 0; kind < 2; kind++) {
      const int heads = kind ? a.k_heads : a.q_heads, step = parts * SLOTS;
      const T* xs = kind ? static_cast<const T*>(a.k) + t * a.k_stride : static_cast<const T*>(a.q) + t * a.q_stride;
      const T* gs = static_cast<const T*>(kind ? a.dk : a.dq) + (size_t)t * heads * a.D;
      T* out = static_cast<T*>(kind ? a.k_out : a.q_out) + (size_t)t * heads * a.D;
      if (part * SLOTS >= heads) continue;
      float w[2 * N];
      HeadRow<T, VEC, LG, C> x, d;
      int u = part * SLOTS + slot;
      x.load(l, xs, u * a.D, a.norm && u < heads);
      d.load(l, gs, u * a.D, u < heads);
      head_weights(l, a, kind ? a.w_k : a.w_q, w);
      for (int base = part * SLOTS; base < heads; base += step) {
        float g[2 * N], n[2 * N];
        x.get(l, n);
        d.get(l, g);
        const int v = u + step;
        if (base + step < heads) {
          x.load(l, xs, v * a.D, a.norm && v < heads);
          d.load(l, gs, v * a.D, v < heads);
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
          const float da = g[i], db = g[N + i];
          const bool turn = l.turned(i);
          g[i] = turn ? da * c[i] + db * s[i] : da;
          g[N + i] = turn ? db * c[i] - da * s[i] : db;
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
        if (u < heads) head_put(l, out, u * a.D, g);
        u = v;
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
      for (int i = 0; i < WAVES; i++) v += red[i][threadIdx.x];
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
    using Two = std::integral_constant<int, 2>;
    using Four = std::integral_constant<int, 4>;
    if (a.D % 8 == 0 && a.rot % 8 == 0) {
      if (a.D <= 64) f(t, Four{}, std::integral_constant<int, 8>{}, One{});
      else if (a.D <= 128) f(t, Four{}, std::integral_constant<int, 16>{}, One{});
      else if (a.D <= 256) f(t, Four{}, std::integral_constant<int, 32>{}, One{});
      else f(t, Four{}, std::integral_constant<int, 64>{}, One{});
    } else if (a.D % 4 == 0 && a.D <= 256 && (a.interleaved || a.rot % 4 == 0)) {
      if (a.D <= 64) f(t, Two{}, std::integral_constant<int, 16>{}, One{});
      else if (a.D <= 128) f(t, Two{}, std::integral_constant<int, 32>{}, One{});
      else f(t, Two{}, std::integral_constant<int, 64>{}, One{});
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
int head_parts(int tokens, int rounds, int waves) {
  const int want = ceil_div(waves, tokens);
  return ceil_div(rounds, ceil_div(rounds, want < rounds ? want : rounds));
}
// Waves of the forward: 64 / 8 heads of 128, 2048 tokens of bf16 19.0 us with 6144 (three shares
// of six rounds a token), 20.5 with 4096, 19.0 with 8192, 21.9 with 16384 (at that step).
constexpr int HEAD_WAVES = 6144;

template <typename Kind>
hipError_t head_launch(const HeadArgs& a, Kind) {
  constexpr int KIND = Kind::value;
  head_dispatch(a, [&](auto t, auto vec, auto lg, auto c) {
    constexpr int LG = decltype(lg)::value, VEC = decltype(vec)::value, C = decltype(c)::value;
    if constexpr (KIND < 0 || VEC < 4 || LG < 64) {  // a cache's heads have 256 channels at most
      constexpr int SLOTS = 64 / LG;
      const int rounds = ceil_div(a.q_heads, SLOTS) + ceil_div(a.k_heads, SLOTS) * (KIND < 0 ? 1 : 2);
      const int parts = head_parts(a.tokens, rounds, HEAD_WAVES);
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
      constexpr int LG = decltype(lg)::value, C = decltype(c)::value, WAVES = head_bwd_waves(C);
      const int heads = a.q_heads > a.k_heads ? a.q_heads : a.k_heads;
      const int parts = head_parts(a.tokens, ceil_div(heads, 64 / LG), 256 * WAVES);
      const long long jobs = (long long)a.tokens * parts;
      blocks = (int)(jobs < 256 * WAVES ? (jobs + WAVES - 1) / WAVES : 256);
      hipLaunchKernelGGL((head_bwd_kernel<decltype(t), decltype(vec)::value, LG, C>), dim3(blocks), dim3(64 * WAVES), 0,
                         a.stream, a, parts);
    });
  }
  if (a.part || !a.tokens) hipLaunchKernelGGL(head_join_kernel, dim3(ceil_div(a.D, 64), 2), dim3(1024), 0, a.stream, a, blocks);
  return hipGetLastError();
}

}  // namespace nq
