// Norms between two blocks of a transformer, with the block's gate and the
// scales of the residual sum, forward and backward.  For each row, d columns:
//
//   u  = y ry (w_post + o),  ry = (mean y^2 + eps)^-1/2        (u = y without the post norm)
//   h' = a h + b gate u
//   x  = h' rh (w_pre + o),  rh = (mean h'^2 + eps)^-1/2
//
// Backward, from dx and dh' (the gradients of x and of h'), with yn = y ry,
// hn = h' rh and means over the row:
//   t  = dx (w_pre + o),  g = dh' + rh (t - hn mean(t hn)),  dw_pre = sum of dx hn over rows
//   dh = a g,  v = b g,  dgate = v u (summed over rows for one gate a channel)
//   s  = v gate (w_post + o),  dy = ry (s - yn mean(s yn)),  dw_post = sum of v gate yn over rows
//
// All arithmetic is fp32; each output is rounded once, to its type (x is formed
// from h' before its rounding).  The row stays in registers from its one read
// to its one write.
#include "nq_common.h"
#include "nq_internal.h"

#include <type_traits>

namespace nq {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ memory
// Thread t of NT holds C x 8 elements of the row.  V = 8: the eight of chunk c
// are columns 8 (c NT + t) .. + 7, read and written in 16-byte pieces (d a
// multiple of 8, every row 16-byte aligned).  V = 1: element e of chunk c is
// column (8 c + e) NT + t, so that neighbouring threads take neighbouring columns.
template <int V>
__device__ __forceinline__ int norm_col(int c, int e, int NT) {
  return V == 8 ? 8 * (c * NT + (int)threadIdx.x) + e : (8 * c + e) * NT + (int)threadIdx.x;
}

template <int V, int C, typename T>
__device__ __forceinline__ void norm_load(const T* p, int d, int NT, float (&v)[8 * C]) {
#pragma unroll
  for (int c = 0; c < C; c++) {
    if constexpr (V == 8) {
      const int k = norm_col<8>(c, 0, NT);
      if (k < d) {
        if constexpr (sizeof(T) == 4) {
          const v4f a = *reinterpret_cast<const v4f*>(p + k), b = *reinterpret_cast<const v4f*>(p + k + 4);
#pragma unroll
          for (int e = 0; e < 4; e++) v[8 * c + e] = a[e], v[8 * c + 4 + e] = b[e];
        } else {
          const uint4 a = *reinterpret_cast<const uint4*>(p + k);
          const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int e = 0; e < 4; e++) {
            if constexpr (std::is_same<T, _Float16>::value) {
              v[8 * c + 2 * e] = (float)__builtin_bit_cast(_Float16, (uint16_t)u[e]);
              v[8 * c + 2 * e + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[e] >> 16));
            } else {
              v[8 * c + 2 * e] = __uint_as_float(u[e] << 16);
              v[8 * c + 2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; e++) v[8 * c + e] = 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const int k = norm_col<1>(c, e, NT);
        v[8 * c + e] = k < d ? to_f32<T>(p[k]) : 0.0f;
      }
    }
  }
}

__device__ __forceinline__ void norm_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void norm_put(uint16_t* p, float v) { *p = f32_to_bf16(v); }

template <int V, int C, typename T>
__device__ __forceinline__ void norm_store(T* p, int d, int NT, const float (&v)[8 * C]) {
#pragma unroll
  for (int c = 0; c < C; c++) {
    if constexpr (V == 8) {
      const int k = norm_col<8>(c, 0, NT);
      if (k < d) {
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<v4f*>(p + k) = v4f{v[8 * c], v[8 * c + 1], v[8 * c + 2], v[8 * c + 3]};
          *reinterpret_cast<v4f*>(p + k + 4) = v4f{v[8 * c + 4], v[8 * c + 5], v[8 * c + 6], v[8 * c + 7]};
        } else {
          uint32_t u[4];
#pragma unroll
          for (int e = 0; e < 4; e++)
            u[e] = (uint32_t)f32_to_bf16(v[8 * c + 2 * e]) | (uint32_t)f32_to_bf16(v[8 * c + 2 * e + 1]) << 16;
          *reinterpret_cast<uint4*>(p + k) = uint4{u[0], u[1], u[2], u[3]};
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const int k = norm_col<1>(c, e, NT);
        if (k < d) norm_put(p + k, v[8 * c + e]);
      }
    }
  }
}

// A norm's weights plus their offset; all ones (and no offset) without weights.
template <int V, int C, typename PT>
__device__ __forceinline__ void norm_weights(const void* p, float offset, int d, int NT, float (&w)[8 * C]) {
  if (p) {
    norm_load<V, C>(static_cast<const PT*>(p), d, NT, w);
#pragma unroll
    for (int i = 0; i < 8 * C; i++) w[i] += offset;
  } else {
#pragma unroll
    for (int i = 0; i < 8 * C; i++) w[i] = 1.0f;
  }
}

// Sum over the workgroup, in a fixed order, to every thread.  `red` holds 16
// floats; two calls in a row use different ones.
__device__ __forceinline__ float norm_sum(float v, float* red) {
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  const int W = blockDim.x >> 6;
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
  for (int w = 1; w < W; w++) s += red[w];
  return s;
}

template <int C>
__device__ __forceinline__ float norm_dot(const float (&a)[8 * C], const float (&b)[8 * C]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8 * C; i++) s = fmaf(a[i], b[i], s);
  return s;
}

__device__ __forceinline__ float norm_rstd(float ss, int d, float eps) { return 1.0f / sqrtf(ss / (float)d + eps); }

// ------------------------------------------------------------------ forward
template <typename HT, typename AT, typename PT, int V, int C>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(NormArgs a) {
  __shared__ float red[32];
  const int NT = blockDim.x, d = a.d;
  const size_t row = blockIdx.x, at = row * d;
  float h[8 * C];
  norm_load<V, C>(static_cast<const HT*>(a.h) + at, d, NT, h);
  if (a.y) {
    float y[8 * C], w[8 * C];
    norm_load<V, C>(static_cast<const AT*>(a.y) + at, d, NT, y);
    if (a.post) {
      norm_weights<V, C, PT>(a.w_post, a.weight_offset, d, NT, w);
      const float r = norm_rstd(norm_sum(norm_dot<C>(y, y), red), d, a.eps);
      if (a.stats && threadIdx.x == 0) a.stats[row] = r;
#pragma unroll
      for (int i = 0; i < 8 * C; i++) y[i] = y[i] * r * w[i];
    }
    if (a.gate || a.gate_rows) {
      if (a.gate) norm_load<V, C>(static_cast<const PT*>(a.gate), d, NT, w);
      else norm_load<V, C>(static_cast<const AT*>(a.gate_rows) + at, d, NT, w);
#pragma unroll
      for (int i = 0; i < 8 * C; i++) y[i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < 8 * C; i++) h[i] = fmaf(a.res_scale, h[i], a.block_scale * y[i]);
    norm_store<V, C>(static_cast<HT*>(a.h_out) + at, d, NT, h);
  }
  if (a.pre) {
    float w[8 * C];
    norm_weights<V, C, PT>(a.w_pre, a.weight_offset, d, NT, w);
    const float r = norm_rstd(norm_sum(norm_dot<C>(h, h), red + 16), d, a.eps);
    if (a.stats && threadIdx.x == 0) a.stats[a.rows + row] = r;
#pragma unroll
    for (int i = 0; i < 8 * C; i++) h[i] = h[i] * r * w[i];
    norm_store<V, C>(static_cast<AT*>(a.x) + at, d, NT, h);
  }
}

// ------------------------------------------------------------------ backward
// Workgroup k takes rows k, k + grid, ...; its sums over rows stay in registers
// and are written once, to part[k][0] (dx hn) and part[k][1] (v yn, times a
// token's gate), for norm_join_kernel.
template <typename HT, typename AT, typename PT, int V, int C>
__global__ void __launch_bounds__(1024) norm_bwd_kernel(NormArgs a) {
  __shared__ float red[32];
  const int NT = blockDim.x, d = a.d;
  float sum_pre[8 * C], sum_post[8 * C];
#pragma unroll
  for (int i = 0; i < 8 * C; i++) sum_pre[i] = sum_post[i] = 0.0f;
  for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x) {
    const size_t at = row * d;
    float g[8 * C];
    if (a.dh_out) {
      norm_load<V, C>(static_cast<const HT*>(a.dh_out) + at, d, NT, g);
    } else {
#pragma unroll
      for (int i = 0; i < 8 * C; i++) g[i] = 0.0f;
    }
    if (a.pre) {
      float hn[8 * C], t[8 * C], w[8 * C];
      norm_load<V, C>(static_cast<const HT*>(a.h) + at, d, NT, hn);
      norm_load<V, C>(static_cast<const AT*>(a.dx) + at, d, NT, t);
      norm_weights<V, C, PT>(a.w_pre, a.weight_offset, d, NT, w);
      const float r = a.stats[a.rows + row];
#pragma unroll
      for (int i = 0; i < 8 * C; i++) {
        hn[i] *= r;
        sum_pre[i] = fmaf(t[i], hn[i], sum_pre[i]);
        t[i] *= w[i];
      }
      const float mean = norm_sum(norm_dot<C>(t, hn), red) / (float)d;
#pragma unroll
      for (int i = 0; i < 8 * C; i++) g[i] = fmaf(r, t[i] - hn[i] * mean, g[i]);
    }
    if (!a.y) {
      norm_store<V, C>(static_cast<HT*>(a.dh) + at, d, NT, g);
      if (NT > 64) __syncthreads();
      continue;
    }
    float y[8 * C], w[8 * C];
    norm_load<V, C>(static_cast<const AT*>(a.y) + at, d, NT, y);
    {
      float dh[8 * C];
#pragma unroll
      for (int i = 0; i < 8 * C; i++) {
        dh[i] = a.res_scale * g[i];
        g[i] *= a.block_scale;
      }
      norm_store<V, C>(static_cast<HT*>(a.dh) + at, d, NT, dh);
    }
    const float r = a.post ? a.stats[row] : 1.0f;
#pragma unroll
    for (int i = 0; i < 8 * C; i++) y[i] *= r;  // yn
    norm_weights<V, C, PT>(a.post ? a.w_post : nullptr, a.weight_offset, d, NT, w);
    if (a.gate_rows) {
      float gate[8 * C], dg[8 * C];
      norm_load<V, C>(static_cast<const AT*>(a.gate_rows) + at, d, NT, gate);
#pragma unroll
      for (int i = 0; i < 8 * C; i++) {
        dg[i] = g[i] * y[i] * w[i];
        g[i] *= gate[i];
      }
      norm_store<V, C>(static_cast<AT*>(a.dgate_rows) + at, d, NT, dg);
    }
#pragma unroll
    for (int i = 0; i < 8 * C; i++) sum_post[i] = fmaf(g[i], y[i], sum_post[i]);
    if (a.gate) {
      float gate[8 * C];
      norm_load<V, C>(static_cast<const PT*>(a.gate), d, NT, gate);
#pragma unroll
      for (int i = 0; i < 8 * C; i++) g[i] *= gate[i];
    }
    if (a.post) {
#pragma unroll
      for (int i = 0; i < 8 * C; i++) g[i] *= w[i];
      const float mean = norm_sum(norm_dot<C>(g, y), red + 16) / (float)d;
#pragma unroll
      for (int i = 0; i < 8 * C; i++) g[i] = r * (g[i] - y[i] * mean);
    }
    norm_store<V, C>(static_cast<AT*>(a.dy) + at, d, NT, g);
    // with both sums in a row, the barrier of one keeps a wave from overwriting
    // what the other still reads; with one sum (or none) it is put here
    if (!(a.pre && a.post) && NT > 64) __syncthreads();
  }
  if (a.part) {
    norm_store<V, C>(a.part + (size_t)blockIdx.x * 2 * d, d, NT, sum_pre);
    norm_store<V, C>(a.part + ((size_t)blockIdx.x * 2 + 1) * d, d, NT, sum_post);
  }
}

// Sums of the workgroups' partial sums, 64 columns a workgroup: wave w adds the
// partials w, w + 4, ... and the four sums are added in order.
template <typename PT>
__global__ void __launch_bounds__(256) norm_join_kernel(NormArgs a, int parts) {
  __shared__ float red[4][2][64];
  const int d = a.d, lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
  float s0 = 0.0f, s1 = 0.0f;
  if (col < d)
    for (int k = w; k < parts; k += 4) {
      s0 += a.part[(size_t)k * 2 * d + col];
      s1 += a.part[((size_t)k * 2 + 1) * d + col];
    }
  red[w][0][lane] = s0;
  red[w][1][lane] = s1;
  __syncthreads();
  if (w || col >= d) return;
  s0 = red[0][0][lane] + red[1][0][lane] + red[2][0][lane] + red[3][0][lane];
  s1 = red[0][1][lane] + red[1][1][lane] + red[2][1][lane] + red[3][1][lane];
  if (a.dw_pre) a.dw_pre[col] = s0;
  if (a.dw_post) a.dw_post[col] = a.gate && parts ? s1 * to_f32<PT>(static_cast<const PT*>(a.gate)[col]) : s1;
  if (a.dgate)
    a.dgate[col] = a.post && a.w_post && parts ? s1 * (to_f32<PT>(static_cast<const PT*>(a.w_post)[col]) + a.weight_offset) : s1;
}

// ------------------------------------------------------------------ host
// Threads and chunks of a row: few rows take one chunk a thread, so that the
// row's latency is one load deep; many rows take up to four, so that the sums
// over the row cross fewer waves.
void norm_shape(int d, int rows, int* NT, int* C) {
  const int chunks = ceil_div(d, 8);
  const int want = rows <= 512 ? 1024 : 256;
  *C = chunks <= want ? 1 : chunks <= 2 * want ? 2 : 4;
  *NT = (int)align_up(ceil_div(chunks, *C), 64);
}

// Calls f with the compile-time types, vector width and chunk count.
template <typename F>
void norm_dispatch(const NormArgs& a, bool vec, int C, F f) {
  auto by_c = [&](auto ht, auto at, auto pt, auto v) {
    if (C == 1) f(ht, at, pt, v, std::integral_constant<int, 1>{});
    else if (C == 2) f(ht, at, pt, v, std::integral_constant<int, 2>{});
    else f(ht, at, pt, v, std::integral_constant<int, 4>{});
  };
  auto by_v = [&](auto ht, auto at, auto pt) {
    if (vec) by_c(ht, at, pt, std::integral_constant<int, 8>{});
    else by_c(ht, at, pt, std::integral_constant<int, 1>{});
  };
  auto by_p = [&](auto ht, auto at) {
    if (a.param_dtype == 0) by_v(ht, at, float{});
    else if (a.param_dtype == 1) by_v(ht, at, _Float16{});
    else by_v(ht, at, uint16_t{});
  };
  if (a.act_dtype == 0) by_p(float{}, float{});
  else if (a.res_dtype == 0) by_p(float{}, uint16_t{});
  else by_p(uint16_t{}, uint16_t{});
}

bool norm_vec(const NormArgs& a) {
  const void* ps[] = {a.h,  a.y,  a.h_out, a.x,    a.gate_rows, a.w_post, a.w_pre,
                      a.gate, a.dx, a.dh_out, a.dh, a.dy,        a.dgate_rows};
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return a.d % 8 == 0;
}

}  // namespace

int norm_bwd_parts(int rows) { return rows < 512 ? rows : 512; }

hipError_t norm_forward(const NormArgs& a) {
  int NT, C;
  norm_shape(a.d, a.rows, &NT, &C);
  norm_dispatch(a, norm_vec(a), C, [&](auto ht, auto at, auto pt, auto v, auto c) {
    auto kernel = norm_fwd_kernel<decltype(ht), decltype(at), decltype(pt), decltype(v)::value, decltype(c)::value>;
    hipLaunchKernelGGL(kernel, dim3(a.rows), dim3(NT), 0, a.stream, a);
  });
  return hipGetLastError();
}

hipError_t norm_backward(const NormArgs& a) {
  const int parts = norm_bwd_parts(a.rows);
  if (a.rows) {
    int NT, C;
    norm_shape(a.d, 1, &NT, &C);
    norm_dispatch(a, norm_vec(a), C, [&](auto ht, auto at, auto pt, auto v, auto c) {
      auto kernel = norm_bwd_kernel<decltype(ht), decltype(at), decltype(pt), decltype(v)::value, decltype(c)::value>;
      hipLaunchKernelGGL(kernel, dim3(parts), dim3(NT), 0, a.stream, a);
    });
  }
  if (a.dw_pre || a.dw_post || a.dgate) {
    const dim3 grid(ceil_div(a.d, 64));
    if (a.param_dtype == 0) hipLaunchKernelGGL((norm_join_kernel<float>), grid, dim3(256), 0, a.stream, a, parts);
    else if (a.param_dtype == 1) hipLaunchKernelGGL((norm_join_kernel<_Float16>), grid, dim3(256), 0, a.stream, a, parts);
    else hipLaunchKernelGGL((norm_join_kernel<uint16_t>), grid, dim3(256), 0, a.stream, a, parts);
  }
  return hipGetLastError();
}

}  // namespace nq
