// The paged cache of keys and values: writing tokens to their slots and reading
// slots back.  A held value is bf16(x), or s c with c = x / s to the nearest whole
// number and s = bf16(max |x| / 127) over a head's channels (8 bits) or bf16(max |x| / 7)
// over 32 of them (4 bits): off by at most half of s, s within 2^-8 of the quotient.
// Both kernels are bound by memory; 8 heads of 128, bf16 in and out: 8192 tokens of 8 bits
// are written in 20.8 us (2.4 TB/s) and read in 12.5 us (4.0), 32768 of bf16 in 79 (3.4) and
// 58 us (4.6), where a large copy moves 5.2; 64 tokens take 4 us either way, of which a launch
// and two dependent accesses (slot, place) are three.
#include "nq_kv.h"
#include "nq_internal.h"

#include <type_traits>

namespace nq {

namespace {

typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));

// Eight elements from `at` on, fp32 (F32) or bf16; rows start at any element.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, size_t at, float (&v)[8]) {
  if constexpr (F32) {
    const u32x4_at2* q = reinterpret_cast<const u32x4_at2*>(static_cast<const float*>(p) + at);
    const u32x4_at2 a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = __uint_as_float(a[i]), v[4 + i] = __uint_as_float(b[i]);
  } else {
    const u32x4_at2 a = *reinterpret_cast<const u32x4_at2*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __uint_as_float(i & 1 ? a[i / 2] & 0xffff0000u : a[i / 2] << 16);
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, size_t at, const float (&v)[8]) {
  if constexpr (F32) {
    u32x4_at2* q = reinterpret_cast<u32x4_at2*>(static_cast<float*>(p) + at);
    u32x4_at2 a, b;
#pragma unroll
    for (int i = 0; i < 4; i++) a[i] = __float_as_uint(v[i]), b[i] = __float_as_uint(v[4 + i]);
    q[0] = a;
    q[1] = b;
  } else {
    u32x4_at2 a;
#pragma unroll
    for (int i = 0; i < 4; i++) a[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<u32x4_at2*>(static_cast<uint16_t*>(p) + at) = a;
  }
}

// ------------------------------------------------------------------ four values at once
// A value tile holds four slots of a channel side by side.  Four tokens whose slots are
// those four (a prompt's are) are stored and read together, a word or two a channel,
// where one after the other each would take a store of one or two bytes a channel.
__device__ inline bool kv_quad(const KvArgs& a, long long t, int64_t (&slots)[4]) {
#pragma unroll
  for (int j = 0; j < 4; j++) slots[j] = t + j < a.tokens ? a.slots[t + j] : -1;
  return slots[0] >= 0 && slots[0] < (int64_t)a.cache.pages * a.cache.page && slots[0] % 4 == 0 &&
         slots[1] == slots[0] + 1 && slots[2] == slots[0] + 2 && slots[3] == slots[0] + 3;
}

// `at`: the place of the first; otherwise as kv_store.
template <int KIND, int LG>
__device__ inline void kv_store_quad(const KvLayout& l, const KvPlace& at, int head, int m, bool on, const float (&v)[4][8]) {
  const int D = l.D, lb = kv_lane_bytes(KIND, D), x = m >> 1, lane = 8 * (m & 1) + 16 * (at.row >> 2);
  uint8_t* half = at.page + l.tile(head, at.tile) + kv_half_bytes(KIND, D);
  if constexpr (KIND == KV_BF16) {
    if (!on) return;
#pragma unroll
    for (int e = 0; e < 8; e++)
      *reinterpret_cast<uint2*>(half + kv_byte(lane + e, 8 * x, lb)) =
          make_uint2(pack_bf16(v[0][e], v[1][e]), pack_bf16(v[2][e], v[3][e]));
  } else {
    constexpr bool wide = KIND == KV_INT8;
    constexpr int most = wide ? 127 : 7, groups = wide ? LG : 4;
    uint32_t words[8] = {}, s16[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const uint32_t bits = on ? __float_as_uint(v[j][e]) & 0x7fffffffu : 0u;
        top = bits > top ? bits : top;
      }
      const float s = kv_scale(kv_top<groups>(top), (float)most);
      s16[j] = __float_as_uint(s) >> 16;
      int q[8];
      kv_codes(v[j], s, most, q);
#pragma unroll
      for (int e = 0; e < 8; e++)
        words[e] |= wide ? (uint32_t)(q[e] & 255) << (8 * j) : (uint32_t)(q[e] + 8) << (8 * (j == 1 ? 2 : j == 2 ? 1 : j));
    }
    uint16_t* scales = reinterpret_cast<uint16_t*>(at.page + l.scales(head, at.tile));
    if (on && m % groups == 0)
      *reinterpret_cast<uint2*>(scales + kv_scale_at(at.row, 1, wide ? 0 : m >> 2, kv_groups(KIND, D))) =
          make_uint2(s16[0] | s16[1] << 16, s16[2] | s16[3] << 16);
#pragma unroll
    for (int e = 0; e < 8; e++) {
      if constexpr (!wide) words[e] |= __shfl_xor(words[e], 2) << 4;  // to the lane of the lower sixteen channels
      if (on && (wide || !(m & 2)))
        *reinterpret_cast<uint32_t*>(half + kv_byte(lane + e, 4 * (wide ? x : m >> 2), lb)) = words[e];
    }
  }
}

template <int KIND>
__device__ inline void kv_load_quad(const KvLayout& l, const KvPlace& at, int head, int m, float (&v)[4][8]) {
  const int D = l.D, lb = kv_lane_bytes(KIND, D), x = m >> 1, lane = 8 * (m & 1) + 16 * (at.row >> 2);
  const uint8_t* half = at.page + l.tile(head, at.tile) + kv_half_bytes(KIND, D);
  if constexpr (KIND == KV_BF16) {
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const uint2 u = *reinterpret_cast<const uint2*>(half + kv_byte(lane + e, 8 * x, lb));
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const uint32_t w = j < 2 ? u.x : u.y;
        v[j][e] = __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
      }
    }
  } else {
    constexpr bool wide = KIND == KV_INT8;
    const uint16_t* scales = reinterpret_cast<const uint16_t*>(at.page + l.scales(head, at.tile));
    const uint2 u = *reinterpret_cast<const uint2*>(scales + kv_scale_at(at.row, 1, wide ? 0 : m >> 2, kv_groups(KIND, D)));
    const float s[4] = {__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                        __uint_as_float(u.y & 0xffff0000u)};
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(half + kv_byte(lane + e, 4 * (wide ? x : m >> 2), lb));
#pragma unroll
      for (int j = 0; j < 4; j++)
        v[j][e] = s[j] * (wide ? (float)(int8_t)(w >> (8 * j))
                               : (float)((int)(w >> (8 * (j == 1 ? 2 : j == 2 ? 1 : j) + (m & 2 ? 4 : 0)) & 15) - 8));
    }
  }
}

// ------------------------------------------------------------------ kernels
// LG lanes a head of one token, or with QUADS of four, eight channels each; the first
// `key_blocks` workgroups take the keys.
template <int KIND, bool F32, int LG, bool QUADS>
__global__ void __launch_bounds__(256) kv_write_kernel(KvArgs a, unsigned key_blocks) {
  const bool values = blockIdx.x >= key_blocks;
  const long long unit = ((long long)(blockIdx.x - (values ? key_blocks : 0)) * 256 + threadIdx.x) / LG;
  const int m = threadIdx.x % LG, head = (int)(unit % a.cache.heads);
  const bool in = 8 * m < a.cache.D;
  const size_t from = (size_t)head * a.cache.D + 8 * m;
  if constexpr (!QUADS) {
    const long long t = unit / a.cache.heads;
    const bool on = t < a.tokens && in;
    KvPlace at{nullptr, 0, 0};
    float v[8] = {};
    if (on) {
      at = kv_place(a.cache, a.data, a.slots[t]);
      load8<F32>(values ? a.v : a.k, t * (values ? a.v_stride : a.k_stride) + from, v);
    }
    if (values) kv_store<KIND, LG, true>(a.cache, at, head, m, on, v);
    else kv_store<KIND, LG, false>(a.cache, at, head, m, on, v);
  } else {
    const long long t = unit / a.cache.heads * 4;
    int64_t slots[4];
    const bool quad = kv_quad(a, t, slots);
    float v[4][8] = {};
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (t + j < a.tokens && in) load8<F32>(values ? a.v : a.k, (t + j) * (values ? a.v_stride : a.k_stride) + from, v[j]);
    if (!values) {
#pragma unroll
      for (int j = 0; j < 4; j++) kv_store<KIND, LG, false>(a.cache, kv_place(a.cache, a.data, slots[j]), head, m, in, v[j]);
      return;
    }
    // whole waves go through either store: its exchanges want every lane of a head
    if (__any(quad)) kv_store_quad<KIND, LG>(a.cache, kv_place(a.cache, a.data, quad ? slots[0] : 0), head, m, quad && in, v);
    if (__any(!quad)) {
#pragma unroll 1
      for (int j = 0; j < 4; j++) {
        float one[8];
#pragma unroll
        for (int e = 0; e < 8; e++) one[e] = j < 2 ? j ? v[1][e] : v[0][e] : j == 2 ? v[2][e] : v[3][e];
        kv_store<KIND, LG, true>(a.cache, kv_place(a.cache, a.data, quad ? -1 : j < 2 ? j ? slots[1] : slots[0] : j == 2 ? slots[2] : slots[3]),
                                 head, m, !quad && in, one);
      }
    }
  }
}

template <int KIND, bool F32, int LG, bool QUADS>
__global__ void __launch_bounds__(256) kv_read_kernel(KvArgs a, unsigned key_blocks) {
  const bool values = blockIdx.x >= key_blocks;
  const long long unit = ((long long)(blockIdx.x - (values ? key_blocks : 0)) * 256 + threadIdx.x) / LG;
  const int m = threadIdx.x % LG, head = (int)(unit % a.cache.heads);
  if (8 * m >= a.cache.D) return;
  const size_t to = (size_t)head * a.cache.D + 8 * m, row = (size_t)a.cache.heads * a.cache.D;
  if constexpr (!QUADS) {
    const long long t = unit / a.cache.heads;
    if (t >= a.tokens) return;
    const KvPlace at = kv_place(a.cache, a.data, a.slots[t]);
    float v[8] = {};
    if (at.page) {
      if (values) kv_load<KIND, true>(a.cache, at, head, m, v);
      else kv_load<KIND, false>(a.cache, at, head, m, v);
    }
    store8<F32>(values ? a.v_out : a.k_out, t * row + to, v);
  } else {
    const long long t = unit / a.cache.heads * 4;
    if (t >= a.tokens) return;
    int64_t slots[4];
    float v[4][8] = {};
    if (kv_quad(a, t, slots) && values) {
      kv_load_quad<KIND>(a.cache, kv_place(a.cache, a.data, slots[0]), head, m, v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const KvPlace at = kv_place(a.cache, a.data, slots[j]);
        if (!at.page) continue;
        if (values) kv_load<KIND, true>(a.cache, at, head, m, v[j]);
        else kv_load<KIND, false>(a.cache, at, head, m, v[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (t + j < a.tokens) store8<F32>(values ? a.v_out : a.k_out, (t + j) * row + to, v[j]);
  }
}

// Calls f with the kind of cache, fp32 or bf16 tokens and the lanes of a head.
template <typename F>
void kv_dispatch(const KvArgs& a, F f) {
  auto by_lg = [&](auto kind, auto f32) {
    if (a.cache.D <= 64) f(kind, f32, std::integral_constant<int, 8>{});
    else if (a.cache.D <= 128) f(kind, f32, std::integral_constant<int, 16>{});
    else f(kind, f32, std::integral_constant<int, 32>{});
  };
  auto by_type = [&](auto kind) {
    if (a.dtype == 0) by_lg(kind, std::true_type{});
    else by_lg(kind, std::false_type{});
  };
  if (a.cache.kind == KV_BF16) by_type(std::integral_constant<int, KV_BF16>{});
  else if (a.cache.kind == KV_INT8) by_type(std::integral_constant<int, KV_INT8>{});
  else by_type(std::integral_constant<int, KV_INT4>{});
}

unsigned kv_blocks(const KvArgs& a, int LG, int each) {
  return (unsigned)((((long long)a.tokens + each - 1) / each * a.cache.heads * LG + 255) / 256);
}

// Whether tokens go four at a time: where there are many, for a prompt's slots
// follow each other.  8 heads of 128: 8192 tokens of 8 bits written in 20.8 us so and 28.1 us
// one by one, read in 12.5 and 20.8; but 512 tokens written in 6.9 us so and 4.8 one by one,
// 61 scattered ones of 4 bits in 6.0 and 4.0.
bool kv_quads(const KvArgs& a) { return (long long)a.tokens * a.cache.heads >= 16384; }

template <typename F>
void kv_launch(const KvArgs& a, F kernel) {
  kv_dispatch(a, [&](auto kind, auto f32, auto lg) {
    constexpr int LG = decltype(lg)::value;
    const bool quads = kv_quads(a);
    const unsigned keys = kv_blocks(a, LG, quads ? 4 : 1);
    if (quads) hipLaunchKernelGGL(kernel(kind, f32, lg, std::true_type{}), dim3(2 * keys), dim3(256), 0, a.stream, a, keys);
    else hipLaunchKernelGGL(kernel(kind, f32, lg, std::false_type{}), dim3(2 * keys), dim3(256), 0, a.stream, a, keys);
  });
}

}  // namespace

hipError_t kv_write(const KvArgs& a) {
  kv_launch(a, [](auto kind, auto f32, auto lg, auto quads) {
    return kv_write_kernel<decltype(kind)::value, decltype(f32)::value, decltype(lg)::value, decltype(quads)::value>;
  });
  return hipGetLastError();
}

hipError_t kv_read(const KvArgs& a) {
  kv_launch(a, [](auto kind, auto f32, auto lg, auto quads) {
    return kv_read_kernel<decltype(kind)::value, decltype(f32)::value, decltype(lg)::value, decltype(quads)::value>;
  });
  return hipGetLastError();
}

}  // namespace nq
