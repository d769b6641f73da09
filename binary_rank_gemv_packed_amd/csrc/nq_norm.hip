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
// from h' before its rounding).  The row stays in registers from its one read to
// its one write: forward up to 16384 columns, backward up to 4096, and up to 8192 but
// for a few registers of some types.  Wider rows pass through scratch memory in part,
// see the kernels.
#include "nq_common.h"
#include "nq_internal.h"

#include <type_traits>

namespace nq {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ memory
// Thread t of NT holds C x 8 elements of the row, chunk c being columns
// 8 (c NT + t) .. + 7, read and written in 16-byte pieces.  WHOLE: d is a multiple
// of 8 and every row 16-byte aligned.  Else the pieces need not be aligned (a row
// of an odd width starts anywhere), and the chunk across the row's end goes
// element by element.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
template <bool WHOLE>
using piece = typename std::conditional<WHOLE, u32x4, u32x4_at2>::type;

__device__ __forceinline__ int norm_col(int c, int NT) { return 8 * (c * NT + (int)threadIdx.x); }

// Column k of a row as a byte offset of 32 bits from the row's address, which is
// the same for the workgroup: one register for all the rows at that column, where
// 64-bit addresses of every row would take two each.
template <typename U, typename T>
__device__ __forceinline__ U* norm_at(T* p, int k) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type byte;
  return reinterpret_cast<U*>(reinterpret_cast<byte*>(p) + (uint32_t)k * (uint32_t)sizeof(T));
}

// A thread's part of a row as it is stored, until get(): what is asked for early
// takes no more registers than its bytes.  Columns from d on are zero.
template <bool WHOLE, int C, typename T>
struct NormRow {
  static constexpr int Q = sizeof(T) / 2;  // pieces of a chunk
  u32x4 u[Q * C];
  __device__ __forceinline__ void load(const void* base, size_t at, int d, int NT) {
    const T* p = static_cast<const T*>(base) + at;
#pragma unroll
    for (int c = 0; c < C; c++) {
      const int k = norm_col(c, NT);
#pragma unroll
      for (int i = 0; i < Q; i++) u[Q * c + i] = u32x4{0u, 0u, 0u, 0u};
      if (k + 8 <= d) {
#pragma unroll
        for (int i = 0; i < Q; i++) u[Q * c + i] = norm_at<const piece<WHOLE>>(p, k)[i];
      } else if (!WHOLE && k < d) {
#pragma unroll
        for (int e = 0; e < 7; e++)
          if (k + e < d) {
            if constexpr (Q == 2) u[Q * c + e / 4][e % 4] = *norm_at<const uint32_t>(p, k + e);
            else u[c][e / 2] |= (uint32_t)*norm_at<const uint16_t>(p, k + e) << (16 * (e & 1));
          }
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (Q == 2) {
      return __uint_as_float(u[i / 4][i % 4]);
    } else {
      const uint32_t w = u[i / 8][i % 8 / 2];
      if constexpr (std::is_same<T, _Float16>::value)
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(i & 1 ? w >> 16 : w));
      else
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
  }
};

template <bool WHOLE, int C, typename T>
__device__ __forceinline__ void norm_store(T* p, int d, int NT, const float (&v)[8 * C]) {
  constexpr int Q = sizeof(T) / 2;
#pragma unroll
  for (int c = 0; c < C; c++) {
    const int k = norm_col(c, NT);
    u32x4 u[Q];
#pragma unroll
    for (int i = 0; i < 4 * Q; i++) {
      if constexpr (Q == 2) u[i / 4][i % 4] = __float_as_uint(v[8 * c + i]);
      else u[0][i] = (uint32_t)f32_to_bf16(v[8 * c + 2 * i]) | (uint32_t)f32_to_bf16(v[8 * c + 2 * i + 1]) << 16;
    }
    if (k + 8 <= d) {
#pragma unroll
      for (int i = 0; i < Q; i++) norm_at<piece<WHOLE>>(p, k)[i] = u[i];
    } else if (!WHOLE && k < d) {
#pragma unroll
      for (int e = 0; e < 7; e++)
        if (k + e < d) {
          if constexpr (Q == 2) *norm_at<uint32_t>(p, k + e) = u[e / 4][e % 4];
          else *norm_at<uint16_t>(p, k + e) = (uint16_t)(u[0][e / 2] >> (16 * (e & 1)));
        }
    }
  }
}

// A norm's weights, asked for by load(): w[i] + offset, or 1 without weights.
template <bool WHOLE, int C, typename PT>
struct NormWeights {
  NormRow<WHOLE, C, PT> row;
  float offset;
  bool given;
  __device__ __forceinline__ void load(const void* p, float weight_offset, int d, int NT) {
    given = p != nullptr;
    offset = weight_offset;
    if (given) row.load(p, 0, d, NT);
  }
  __device__ __forceinline__ float get(int i) const { return given ? row.get(i) + offset : 1.0f; }
};

// Sum over the wavefront to every lane: within sixteen lanes by exchanges that
// cost an instruction each, then the four sixteens in order.
__device__ __forceinline__ float wave_sum(float v) {
#define NQ_DPP_ADD(ctrl) v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, false))
  NQ_DPP_ADD(0xB1);   // lane ^ 1
  NQ_DPP_ADD(0x4E);   // lane ^ 2
  NQ_DPP_ADD(0x141);  // the other four of eight
  NQ_DPP_ADD(0x140);  // the other eight of sixteen
#undef NQ_DPP_ADD
  const int u = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(u, 0)) + __int_as_float(__builtin_amdgcn_readlane(u, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(u, 32)) + __int_as_float(__builtin_amdgcn_readlane(u, 48)));
}

// Sum over the workgroup, in a fixed order, to every thread.  `red` holds 16
// floats; two calls in a row use different ones.
__device__ __forceinline__ float norm_sum(float v, float* red) {
  v = wave_sum(v);
  const int W = blockDim.x >> 6;
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; w++) s += w < W ? red[w] : 0.0f;
  return s;
}

__device__ __forceinline__ float norm_rstd(float ss, int d, float eps) { return 1.0f / sqrtf(ss / (float)d + eps); }

// ------------------------------------------------------------------ forward
// While the registers hold it, everything is asked for before the first sum: with
// few rows the kernel's time is that of one read.  One row of 8192: 4.85 us (5.4 us
// with each read where it is used); 2048 rows with an fp32 stream: 42.2 us a call
// among others, 4.8 TB/s (38.6 us by itself in a kernel trace), where a 1 GiB copy
// moves 5.2; 1024 x 16384 50 us, 4.0 TB/s.  Four chunks a thread (above 16384 columns)
// spill 28 to 436 bytes a lane in 9 of their 18 variants: 512 x 28672 46 us, 3.8 TB/s.
template <typename HT, typename AT, typename PT, bool WHOLE, int C>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(NormArgs a) {
  constexpr bool EARLY = C == 1 || (C == 2 && sizeof(AT) == 2);
  __shared__ float red[32];
  const int NT = blockDim.x, d = a.d;
  const size_t row = blockIdx.x, at = row * d;
  NormRow<WHOLE, C, HT> h0;
  NormRow<WHOLE, C, AT> y0, gr;
  NormRow<WHOLE, C, PT> gc;
  NormWeights<WHOLE, C, PT> wp, wq;
  auto load_branch = [&]() {
    if (a.gate_rows) gr.load(a.gate_rows, at, d, NT);
    wp.load(a.post ? a.w_post : nullptr, a.weight_offset, d, NT);
    if (a.gate) gc.load(a.gate, 0, d, NT);
  };
  auto load_pre = [&]() { wq.load(a.pre ? a.w_pre : nullptr, a.weight_offset, d, NT); };
  h0.load(a.h, at, d, NT);
  if (a.y) {
    y0.load(a.y, at, d, NT);
    if (EARLY) load_branch();
  }
  if (EARLY) load_pre();
  float h[8 * C];
  if (a.y) {
    float r = 1.0f;
    if (a.post) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8 * C; i++) ss = fmaf(y0.get(i), y0.get(i), ss);
      r = norm_rstd(norm_sum(ss, red), d, a.eps);
      if (a.stats && threadIdx.x == 0) a.stats[row] = r;
    }
    if (!EARLY) load_branch();
#pragma unroll
    for (int i = 0; i < 8 * C; i++) {
      float u = y0.get(i) * r * wp.get(i);
      if (a.gate) u *= gc.get(i);
      if (a.gate_rows) u *= gr.get(i);
      h[i] = fmaf(a.res_scale, h0.get(i), a.block_scale * u);
    }
    norm_store<WHOLE, C>(static_cast<HT*>(a.h_out) + at, d, NT, h);
  } else {
#pragma unroll
    for (int i = 0; i < 8 * C; i++) h[i] = h0.get(i);
  }
  if (a.pre) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8 * C; i++) ss = fmaf(h[i], h[i], ss);
    const float r = norm_rstd(norm_sum(ss, red + 16), d, a.eps);
    if (a.stats && threadIdx.x == 0) a.stats[a.rows + row] = r;
    if (!EARLY) load_pre();
#pragma unroll
    for (int i = 0; i < 8 * C; i++) h[i] = h[i] * r * wq.get(i);
    norm_store<WHOLE, C>(static_cast<AT*>(a.x) + at, d, NT, h);
  }
}

// ------------------------------------------------------------------ backward
// What a row of the backward pass reads, in two parts.
template <typename HT, typename AT, bool WHOLE, int C>
struct NormBwdRow {
  NormRow<WHOLE, C, HT> h, dh;
  NormRow<WHOLE, C, AT> dx, y;
  float ry, rh;
  __device__ __forceinline__ void load_pre(const NormArgs& a, size_t row, int NT) {
    if (a.pre) {
      h.load(a.h, row * a.d, a.d, NT);
      dx.load(a.dx, row * a.d, a.d, NT);
      rh = a.stats[a.rows + row];
    }
    if (a.dh_out) dh.load(a.dh_out, row * a.d, a.d, NT);
  }
  __device__ __forceinline__ void load_post(const NormArgs& a, size_t row, int NT) {
    if (a.y) {
      y.load(a.y, row * a.d, a.d, NT);
      ry = a.post ? a.stats[row] : 1.0f;
    }
  }
};

// Workgroup k takes rows k, k + grid, ...; its sums over rows stay in registers
// and are written once, to part[k][0] (dx hn) and part[k][1] (v yn, times a
// token's gate), for norm_join_kernel.  With one chunk a thread (C = 1) the next
// row is asked for before this one is worked on, for two sums over the row with
// a barrier each would leave the memory idle; the weights then lie in shared
// memory (w_pre, w_post, gate, each [thread][8]), for a read of them from memory
// would have to wait for the next row's, which is ahead of it.
// Up to 512 threads (4096 columns) a thread may have 256 registers, and none of
// this leaves them.  4096 x 8192 with an fp32 stream: 123 us with the join, 4.9 TB/s
// (149 us with 512 workgroups, no row ahead and the weights read from memory).
// 1024 threads have 128 registers each.  One chunk a thread then spills 12 bytes a lane
// with an fp32 stream and weights, 48 to 52 with an fp32 branch, and 68 to 160 where
// rows are not whole 16-byte pieces (1024 x 6001, 52 us, 2.1 TB/s).  Two and four
// chunks, whose two sums over rows alone are 32 and 64 registers beside the row and its
// gradients, spill 348 to 1960 bytes inside the row loop: 1024 x 16384 with an fp32
// stream 235 us, four times its bytes' time, and 1209 us with all of it bf16, where
// elementary operations take 791 us.
template <typename HT, typename AT, typename PT, bool WHOLE, int C, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_bwd_kernel(NormArgs a) {
  constexpr bool AHEAD = C == 1;
  extern __shared__ __align__(16) float held[];
  __shared__ float red[32];
  const int NT = blockDim.x, d = a.d;
  float sum_pre[8 * C], sum_post[8 * C];
#pragma unroll
  for (int i = 0; i < 8 * C; i++) sum_pre[i] = sum_post[i] = 0.0f;
  const void* w_pre = a.pre ? a.w_pre : nullptr;
  const void* w_post = a.post ? a.w_post : nullptr;
  // the weights as factors: which = 0 w_pre, 1 w_post, 2 a channel's gate
  auto factor = [&](int which, float (&w)[8 * C]) {
    const void* p = which == 0 ? w_pre : which == 1 ? w_post : a.gate;
    if (!p) {
#pragma unroll
      for (int i = 0; i < 8 * C; i++) w[i] = 1.0f;
    } else if (AHEAD) {
      const v4f* q = reinterpret_cast<const v4f*>(held + which * 8 * NT) + threadIdx.x;
      const v4f lo = q[0], hi = q[NT];
#pragma unroll
      for (int i = 0; i < 4; i++) w[i] = lo[i], w[4 + i] = hi[i];
    } else {
      NormRow<WHOLE, C, PT> r;
      r.load(p, 0, d, NT);
#pragma unroll
      for (int i = 0; i < 8 * C; i++) w[i] = r.get(i) + (which == 2 ? 0.0f : a.weight_offset);
    }
  };
  NormBwdRow<HT, AT, WHOLE, C> next;
  if (AHEAD) {
    next.load_pre(a, blockIdx.x, NT);
    next.load_post(a, blockIdx.x, NT);
    for (int which = 0; which < 3; which++) {  // each thread reads back what it wrote
      const void* p = which == 0 ? w_pre : which == 1 ? w_post : a.gate;
      if (!p) continue;
      const float o = which == 2 ? 0.0f : a.weight_offset;
      NormRow<WHOLE, C, PT> r;
      r.load(p, 0, d, NT);
      v4f* q = reinterpret_cast<v4f*>(held + which * 8 * NT) + threadIdx.x;
      q[0] = v4f{r.get(0) + o, r.get(1) + o, r.get(2) + o, r.get(3) + o};
      q[NT] = v4f{r.get(4) + o, r.get(5) + o, r.get(6) + o, r.get(7) + o};
    }
  }
  for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x) {
    const size_t at = row * d;
    // behind the last row this one is read again, from the caches
    const size_t after = row + gridDim.x < (size_t)a.rows ? row + gridDim.x : row;
    if (!AHEAD) next.load_pre(a, row, NT);
    NormRow<WHOLE, C, AT> gate;
    if (AHEAD && a.gate_rows) gate.load(a.gate_rows, at, d, NT);
    float g[8 * C], w[8 * C];
#pragma unroll
    for (int i = 0; i < 8 * C; i++) g[i] = a.dh_out ? next.dh.get(i) : 0.0f;
    if (a.pre) {
      float hn[8 * C], t[8 * C], dot = 0.0f;
      const float r = next.rh;
      factor(0, w);
#pragma unroll
      for (int i = 0; i < 8 * C; i++) {
        hn[i] = next.h.get(i) * r;
        t[i] = next.dx.get(i);
        sum_pre[i] = fmaf(t[i], hn[i], sum_pre[i]);
        t[i] *= w[i];
        dot = fmaf(t[i], hn[i], dot);
      }
      if (AHEAD) next.load_pre(a, after, NT);
      const float mean = norm_sum(dot, red) / (float)d;
#pragma unroll
      for (int i = 0; i < 8 * C; i++) g[i] = fmaf(r, t[i] - hn[i] * mean, g[i]);
    } else if (AHEAD) {
      next.load_pre(a, after, NT);
    }
    if (a.y) {
      if (!AHEAD) next.load_post(a, row, NT);
      float s[8 * C], yn[8 * C], dot = 0.0f;
      const float r = next.ry;
#pragma unroll
      for (int i = 0; i < 8 * C; i++) {
        yn[i] = next.y.get(i) * r;
        s[i] = a.block_scale * g[i];
        g[i] *= a.res_scale;
      }
      norm_store<WHOLE, C>(static_cast<HT*>(a.dh) + at, d, NT, g);
      factor(1, w);
      if (a.gate_rows) {
        float dg[8 * C];
        if (!AHEAD) gate.load(a.gate_rows, at, d, NT);
#pragma unroll
        for (int i = 0; i < 8 * C; i++) {
          dg[i] = s[i] * yn[i] * w[i];
          s[i] *= gate.get(i);
        }
        norm_store<WHOLE, C>(static_cast<AT*>(a.dgate_rows) + at, d, NT, dg);
      }
      if (AHEAD) next.load_post(a, after, NT);
#pragma unroll
      for (int i = 0; i < 8 * C; i++) {
        sum_post[i] = fmaf(s[i], yn[i], sum_post[i]);
        s[i] *= w[i];
      }
      if (a.gate) {
        factor(2, w);
#pragma unroll
        for (int i = 0; i < 8 * C; i++) s[i] *= w[i];
      }
      if (a.post) {
#pragma unroll
        for (int i = 0; i < 8 * C; i++) dot = fmaf(s[i], yn[i], dot);
        const float mean = norm_sum(dot, red + 16) / (float)d;
#pragma unroll
        for (int i = 0; i < 8 * C; i++) s[i] = r * (s[i] - yn[i] * mean);
      }
      norm_store<WHOLE, C>(static_cast<AT*>(a.dy) + at, d, NT, s);
    } else {
      norm_store<WHOLE, C>(static_cast<HT*>(a.dh) + at, d, NT, g);
    }
    // with both sums in a row, the barrier of one keeps a wave from overwriting
    // what the other still reads; with one sum (or none) it is put here
    if (!(a.pre && a.y && a.post) && NT > 64) __syncthreads();
  }
  if (a.part) {
    norm_store<WHOLE, C>(a.part + (size_t)blockIdx.x * 2 * d, d, NT, sum_pre);
    norm_store<WHOLE, C>(a.part + ((size_t)blockIdx.x * 2 + 1) * d, d, NT, sum_post);
  }
}

// Sums of the workgroups' partial sums, 64 columns of one of the two sums
// (blockIdx.y) a workgroup: wave w adds the partials w, w + 16, ..., eight reads
// under way at a time, and the sixteen sums are added in order.
template <typename PT>
__global__ void __launch_bounds__(1024) norm_join_kernel(NormArgs a, int parts) {
  __shared__ float red[16][64];
  const int d = a.d, lane = threadIdx.x & 63, w = threadIdx.x >> 6, col = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (col < d) {
    const float* p = a.part + (size_t)blockIdx.y * d + col;
#pragma unroll 8
    for (int k = w; k < parts; k += 16) s += p[(size_t)k * 2 * d];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w || col >= d) return;
#pragma unroll
  for (int i = 1; i < 16; i++) s += red[i][lane];
  if (blockIdx.y == 0) {
    if (a.dw_pre) a.dw_pre[col] = s;
    return;
  }
  if (a.dw_post) a.dw_post[col] = a.gate && parts ? s * to_f32<PT>(static_cast<const PT*>(a.gate)[col]) : s;
  if (a.dgate)
    a.dgate[col] =
        a.post && a.w_post && parts ? s * (to_f32<PT>(static_cast<const PT*>(a.w_post)[col]) + a.weight_offset) : s;
}

// ------------------------------------------------------------------ host
// Threads and chunks of a row: one chunk a thread while 1024 threads hold the row, so
// that its latency is one load deep.  Four chunks on a quarter of the threads are
// slower or equal: 1 x 8192 4.8 -> 6.5 us, 2048 x 8192 46.3 -> 54.4 us, 2048 x 4096
// (two chunks) 25.4 us either way.
void norm_shape(int d, int* NT, int* C) {
  const int chunks = ceil_div(d, 8);
  const int want = 1024;
  *C = chunks <= want ? 1 : chunks <= 2 * want ? 2 : 4;
  *NT = (int)align_up(ceil_div(chunks, *C), 64);
}

// Calls f with the compile-time types, whether rows are whole, and chunk count.
template <typename F>
void norm_dispatch(const NormArgs& a, bool whole, int C, F f) {
  auto by_c = [&](auto ht, auto at, auto pt, auto v) {
    if (C == 1) f(ht, at, pt, v, std::integral_constant<int, 1>{});
    else if (C == 2) f(ht, at, pt, v, std::integral_constant<int, 2>{});
    else f(ht, at, pt, v, std::integral_constant<int, 4>{});
  };
  auto by_v = [&](auto ht, auto at, auto pt) {
    if (whole) by_c(ht, at, pt, std::true_type{});
    else by_c(ht, at, pt, std::false_type{});
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

bool norm_whole(const NormArgs& a) {
  const void* ps[] = {a.h,  a.y,  a.h_out, a.x,    a.gate_rows, a.w_post, a.w_pre,
                      a.gate, a.dx, a.dh_out, a.dh, a.dy,        a.dgate_rows};
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return a.d % 8 == 0;
}

}  // namespace

// Workgroups of the backward pass: one a CU.  512 are slower at most sizes (1024 x
// 4096 24.6 -> 28.4 us, 4096 x 8192 126 -> 134 us, 512 x 1024 10.9 -> 11.8 us) and
// faster at few (333 x 1619 18.6 -> 16.8 us, 4096 x 2048 39.8 -> 38.7 us).
int norm_bwd_parts(int rows) { return rows < 256 ? rows : 256; }

hipError_t norm_forward(const NormArgs& a) {
  int NT, C;
  norm_shape(a.d, &NT, &C);
  norm_dispatch(a, norm_whole(a), C, [&](auto ht, auto at, auto pt, auto v, auto c) {
    auto kernel = norm_fwd_kernel<decltype(ht), decltype(at), decltype(pt), decltype(v)::value, decltype(c)::value>;
    hipLaunchKernelGGL(kernel, dim3(a.rows), dim3(NT), 0, a.stream, a);
  });
  return hipGetLastError();
}

hipError_t norm_backward(const NormArgs& a) {
  const int parts = norm_bwd_parts(a.rows);
  if (a.rows) {
    int NT, C;
    norm_shape(a.d, &NT, &C);
    norm_dispatch(a, norm_whole(a), C, [&](auto ht, auto at, auto pt, auto v, auto c) {
      constexpr int CC = decltype(c)::value;
      using H = decltype(ht);
      using A = decltype(at);
      using Q = decltype(pt);
      auto kernel = norm_bwd_kernel<H, A, Q, decltype(v)::value, CC, 1024>;
      if constexpr (CC == 1)
        if (NT <= 512) kernel = norm_bwd_kernel<H, A, Q, decltype(v)::value, CC, 512>;
      hipLaunchKernelGGL(kernel, dim3(parts), dim3(NT), C == 1 ? (size_t)3 * 8 * NT * 4 : 0, a.stream, a);
    });
  }
  if (a.dw_pre || a.dw_post || a.dgate) {
    const dim3 grid(ceil_div(a.d, 64), 2), block(1024);
    if (a.param_dtype == 0) hipLaunchKernelGGL((norm_join_kernel<float>), grid, block, 0, a.stream, a, parts);
    else if (a.param_dtype == 1) hipLaunchKernelGGL((norm_join_kernel<_Float16>), grid, block, 0, a.stream, a, parts);
    else hipLaunchKernelGGL((norm_join_kernel<uint16_t>), grid, block, 0, a.stream, a, parts);
  }
  return hipGetLastError();
}

}  // namespace nq
