// The paged cache of keys and values: writing tokens to their slots and reading
// slots back.  A held value is bf16(x), or s c with c = x / s to the nearest whole
// number and s = bf16(max |x| / 127) over a head's channels (8 bits) or bf16(max |x| / 7)
// over 32 of them (4 bits): off by at most half of s, s within 2^-9 of the quotient.
// Both kernels are bound by memory.
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
    for (int i = 0; i < 4; i++) a[i] = f32_to_bf16(v[2 * i]) | (uint32_t)f32_to_bf16(v[2 * i + 1]) << 16;
    *reinterpret_cast<u32x4_at2*>(static_cast<uint16_t*>(p) + at) = a;
  }
}

// LG lanes a (token, head), eight channels each; blockIdx.y = 0 keys, 1 values.
template <int KIND, bool F32, int LG>
__global__ void __launch_bounds__(256) kv_write_kernel(KvArgs a) {
  const long long unit = ((long long)blockIdx.x * 256 + threadIdx.x) / LG;
  const int m = threadIdx.x % LG, head = (int)(unit % a.cache.heads);
  const long long t = unit / a.cache.heads;
  const bool on = t < a.tokens && 8 * m < a.cache.D;
  KvPlace at{nullptr, 0, 0};
  float v[8] = {};
  if (on) {
    at = kv_place(a.cache, a.data, a.slots[t]);
    const size_t from = (size_t)head * a.cache.D + 8 * m;
    if (blockIdx.y) load8<F32>(a.v, t * a.v_stride + from, v);
    else load8<F32>(a.k, t * a.k_stride + from, v);
  }
  if (blockIdx.y) kv_store<KIND, LG, true>(a.cache, at, head, m, on, v);
  else kv_store<KIND, LG, false>(a.cache, at, head, m, on, v);
}

template <int KIND, bool F32, int LG>
__global__ void __launch_bounds__(256) kv_read_kernel(KvArgs a) {
  const long long unit = ((long long)blockIdx.x * 256 + threadIdx.x) / LG;
  const int m = threadIdx.x % LG, head = (int)(unit % a.cache.heads);
  const long long t = unit / a.cache.heads;
  if (t >= a.tokens || 8 * m >= a.cache.D) return;
  const KvPlace at = kv_place(a.cache, a.data, a.slots[t]);
  float v[8] = {};
  const size_t to = (size_t)unit * a.cache.D + 8 * m;
  if (blockIdx.y) {
    if (at.page) kv_load<KIND, true>(a.cache, at, head, m, v);
    store8<F32>(a.v_out, to, v);
  } else {
    if (at.page) kv_load<KIND, false>(a.cache, at, head, m, v);
    store8<F32>(a.k_out, to, v);
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

unsigned kv_blocks(const KvArgs& a, int LG) {
  return (unsigned)(((long long)a.tokens * a.cache.heads * LG + 255) / 256);
}

}  // namespace

hipError_t kv_write(const KvArgs& a) {
  kv_dispatch(a, [&](auto kind, auto f32, auto lg) {
    auto kernel = kv_write_kernel<decltype(kind)::value, decltype(f32)::value, decltype(lg)::value>;
    hipLaunchKernelGGL(kernel, dim3(kv_blocks(a, decltype(lg)::value), 2), dim3(256), 0, a.stream, a);
  });
  return hipGetLastError();
}

hipError_t kv_read(const KvArgs& a) {
  kv_dispatch(a, [&](auto kind, auto f32, auto lg) {
    auto kernel = kv_read_kernel<decltype(kind)::value, decltype(f32)::value, decltype(lg)::value>;
    hipLaunchKernelGGL(kernel, dim3(kv_blocks(a, decltype(lg)::value), 2), dim3(256), 0, a.stream, a);
  });
  return hipGetLastError();
}

}  // namespace nq
