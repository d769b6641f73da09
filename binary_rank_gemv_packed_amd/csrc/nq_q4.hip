// Linears with 4-bit weights and group scales: packing and the forward.
//
//   y[b, i] = sum_j W[i, j] x[b, j],   W[i, j] = s[i, j / G] (q[i, j] - z[i, j / G])
//
// with codes q in 0..15, one scale s and one zero point z (8 without zero
// points) for G = 32, 64 or 128 consecutive columns of a row.
//
// Arithmetic.  q - z is a whole number of at most five bits, exact in fp16: the
// codes become fp16 by setting them into the mantissa of 1024 (0x6400 | q) and
// subtracting 1024 + z.  An activation becomes fp16 too, after a power of two
// has put the largest magnitude of its block (128 columns of a row in the
// decode kernel, the row in the prompt kernel) into [2^14, 2^15): a bf16 value
// keeps its eight bits down to 2^-32 of the block's largest, and what is lost
// below is under 2^-39 of it.  An fp32 value is taken as two fp16 pieces, the
// rounded value and its rounded remainder, off by at most 2^-22 of itself.  So
// the products are exact or nearly so, the sums over a group are held by the
// fp16 MFMA in fp32, and s times the block's power of two multiplies the group's
// sum in fp32.  y is rounded once.
#include "nq_common.h"
#include "nq_internal.h"

#include <type_traits>

namespace nq {

namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ pack / unpack
// Column (inside a word's eight) of nibble p: nibbles p and p + 4 are the two
// halves that one mask takes out of the word, columns 2p and 2p + 1.
__device__ inline int q4_nibble_col(int p) { return p < 4 ? 2 * p : 2 * (p - 4) + 1; }

// One thread per 32-bit word of codes.
__global__ void __launch_bounds__(256) q4_pack_codes_kernel(const uint8_t* __restrict__ q, int m, int n, int KT,
                                                            long long words, uint32_t* __restrict__ out,
                                                            int* __restrict__ bad_flag) {
  for (long long id = (long long)blockIdx.x * 256 + threadIdx.x; id < words; id += (long long)gridDim.x * 256) {
    const int t = (int)(id & 3), lane = (int)(id >> 2) & 63;
    const long long tile = id >> 8;
    const int kt = (int)(tile % KT), row = (int)(tile / KT) * 16 + (lane & 15);
    const int col0 = kt * 128 + 32 * t + 8 * (lane >> 4);
    uint32_t word = 0;
    bool bad = false;
    if (row < m)
      for (int p = 0; p < 8; p++) {
        const int col = col0 + q4_nibble_col(p);
        if (col >= n) continue;
        const uint32_t c = q[(size_t)row * n + col];
        bad |= c > 15;
        word |= (c & 15u) << (4 * p);
      }
    out[id] = word;
    if (bad) atomicOr(bad_flag, 1);
  }
}

// One thread per (row tile, column tile, group, row) entry of scales or zero points.
template <typename T>
__global__ void __launch_bounds__(256) q4_pack_groups_kernel(const T* __restrict__ in, int m, int ng, int KT, int SG,
                                                             long long entries, T* __restrict__ out, int limit,
                                                             int* __restrict__ bad_flag) {
  for (long long id = (long long)blockIdx.x * 256 + threadIdx.x; id < entries; id += (long long)gridDim.x * 256) {
    const long long rest = id >> 4;
    const int g = (int)(rest % (KT * SG)), row = (int)(rest / (KT * SG)) * 16 + (int)(id & 15);
    T v = 0;
    if (row < m && g < ng) v = in[(size_t)row * ng + g];
    if (limit && (int)v > limit) atomicOr(bad_flag, 1);
    out[id] = v;
  }
}

__global__ void __launch_bounds__(256) q4_unpack_kernel(const uint32_t* __restrict__ in, int m, int n, int KT,
                                                        long long words, uint8_t* __restrict__ q) {
  for (long long id = (long long)blockIdx.x * 256 + threadIdx.x; id < words; id += (long long)gridDim.x * 256) {
    const int t = (int)(id & 3), lane = (int)(id >> 2) & 63;
    const long long tile = id >> 8;
    const int kt = (int)(tile % KT), row = (int)(tile / KT) * 16 + (lane & 15);
    const int col0 = kt * 128 + 32 * t + 8 * (lane >> 4);
    if (row >= m) continue;
    const uint32_t word = in[id];
    for (int p = 0; p < 8; p++) {
      const int col = col0 + q4_nibble_col(p);
      if (col < n) q[(size_t)row * n + col] = (uint8_t)((word >> (4 * p)) & 15u);
    }
  }
}

__global__ void __launch_bounds__(256) q4_unpack_zeros_kernel(const uint8_t* __restrict__ in, int m, int ng, int KT,
                                                              int SG, long long entries, uint8_t* __restrict__ z) {
  for (long long id = (long long)blockIdx.x * 256 + threadIdx.x; id < entries; id += (long long)gridDim.x * 256) {
    const long long rest = id >> 4;
    const int g = (int)(rest % (KT * SG)), row = (int)(rest / (KT * SG)) * 16 + (int)(id & 15);
    if (row < m && g < ng) z[(size_t)row * ng + g] = in[id];
  }
}

// ------------------------------------------------------------------ shared pieces
// The eight codes of a word less their zero point, as an MFMA operand: column
// order 0..7.  zc holds -(1024 + z) twice.
__device__ __forceinline__ h8 q4_expand(uint32_t w, h2 zc) {
  union {
    h2 p[4];
    h8 v;
  } u;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t c = ((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
    u.p[i] = __builtin_bit_cast(h2, c) + zc;
  }
  return u.v;
}

__device__ __forceinline__ h2 q4_zero(uint32_t z) { return __builtin_bit_cast(h2, (z | (z << 16)) | 0xE400E400u); }

// Four neighbouring scales as floats.
__device__ __forceinline__ v4f q4_scales(const _Float16* p) {
  return __builtin_convertvector(*reinterpret_cast<const h4*>(p), v4f);
}
__device__ __forceinline__ v4f q4_scales(const float* p) { return *reinterpret_cast<const v4f*>(p); }

// Columns k .. k+7 of a row of x (zero from column n on) as floats; vec: the
// eight can be read in 16-byte pieces.
__device__ __forceinline__ void q4_load8(const float* x, int k, int n, bool vec, float* v) {
  if (vec && k + 8 <= n) {
    const v4f a = *reinterpret_cast<const v4f*>(x + k), b = *reinterpret_cast<const v4f*>(x + k + 4);
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = a[i], v[4 + i] = b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = k + i < n ? x[k + i] : 0.0f;
  }
}
__device__ __forceinline__ void q4_load8(const uint16_t* x, int k, int n, bool vec, float* v) {
  if (vec && k + 8 <= n) {
    const uint4 a = *reinterpret_cast<const uint4*>(x + k);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = k + i < n ? to_f32<uint16_t>(x[k + i]) : 0.0f;
  }
}

// Largest finite magnitude of eight values (0 if there is none).
__device__ __forceinline__ float q4_max8(const float* v) {
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float a = fabsf(v[i]);
    mx = fmaxf(mx, a < INFINITY ? a : 0.0f);
  }
  return mx;
}

// Power of two that puts a block whose largest magnitude is mx into fp16: mx 2^e
// in [2^14, 2^15).  e <= 120 keeps 2^-e a normal number.
__device__ __forceinline__ int q4_block_exp(float mx) {
  if (!(mx > 0.0f)) return 0;
  const int e = 14 - floor_log2(mx);
  return e < 120 ? e : 120;
}

template <int P>
__device__ __forceinline__ void q4_to_f16(const float* v, int e, h8* hi, h8* lo) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float s = __builtin_ldexpf(v[i], e);
    const _Float16 h = (_Float16)s;
    (*hi)[i] = h;
    // an infinity or NaN has no remainder
    if (P == 2) (*lo)[i] = fabsf(s) < INFINITY ? (_Float16)(s - (float)h) : (_Float16)0.0f;
  }
}

// Maximum over the 16 lanes of a row of the wavefront.
__device__ __forceinline__ float row16_max(float v) {
#define NQ_ROR_MAX(n)                                                                                           \
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + (n), 0xf, 0xf, false)))
  NQ_ROR_MAX(8);
  NQ_ROR_MAX(4);
  NQ_ROR_MAX(2);
  NQ_ROR_MAX(1);
#undef NQ_ROR_MAX
  return v;
}

__device__ __forceinline__ void q4_store(void* y, int ydt, size_t i, float v) {
  if (ydt == 0) reinterpret_cast<float*>(y)[i] = v;
  else reinterpret_cast<uint16_t*>(y)[i] = f32_to_bf16(v);
}

// Orders a wavefront's own shared-memory accesses before and after it.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ------------------------------------------------------------------ decode: B <= 16
struct Q4DecArgs {
  const uint8_t* blob[GROUP_MAX];
  void* y[GROUP_MAX];
  int m[GROUP_MAX], wg_end[GROUP_MAX];
  int L, n, KT, B;
  int tpw;     // column tiles per wave
  int region;  // bytes of shared memory per wave
  int xvec, ydt;
  const void* x;
};

// One workgroup computes R row tiles (16 R rows) of one layer for all B <= 16
// rows of x; its waves take contiguous runs of tpw column tiles each and their
// sums meet in shared memory.  A wave goes through its run T column tiles at a
// time: it asks for the codes, scales and zero points of R x T tiles, turns the
// same columns of x into fp16 in its own part of shared memory while they
// come, and multiplies.  Lane layout of the 16x16x32 MFMA: the first operand
// has row lane & 15 and columns 8 (lane >> 4) .. + 7, the second row b = lane & 15
// of x and the same columns; the result has row 4 (lane >> 4) + v of the tile
// for b = lane & 15.  Lanes with b >= B repeat row B - 1 and are not stored.
template <typename XT, typename ST, int SG, bool ZERO, int T, int R>
__global__ void __launch_bounds__(1024) q4_dec_kernel(Q4DecArgs a) {
  constexpr int P = sizeof(XT) == 4 ? 2 : 1;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, W = blockDim.x >> 6, B = a.B, KT = a.KT;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* mine = smem + wave * a.region;
  _Float16* img = reinterpret_cast<_Float16*>(mine);                        // [P][T][B][128]
  float* xfac = reinterpret_cast<float*>(mine + (size_t)P * T * B * 256);  // [T][B]

  int l = 0, wg = blockIdx.x;
  while (l + 1 < a.L && (int)blockIdx.x >= a.wg_end[l]) l++;
  if (l) wg -= a.wg_end[l - 1];
  const int m = a.m[l], RT = ceil_div(m, 16), rt0 = wg * R;
  const Q4Layout lay = q4_layout(m, a.n, 128 / SG, sizeof(ST), ZERO);
  const uint8_t* blob = a.blob[l];
  const XT* x = reinterpret_cast<const XT*>(a.x);

  const uint4* codes[R];
  const ST* scales[R];
  const uint8_t* zeros[R];
#pragma unroll
  for (int r = 0; r < R; r++) {
    const size_t rt = min(rt0 + r, RT - 1);
    codes[r] = reinterpret_cast<const uint4*>(blob + lay.off_codes) + rt * KT * 64 + lane;
    scales[r] = reinterpret_cast<const ST*>(blob + lay.off_scales) + rt * KT * SG * 16 + 4 * (lane >> 4);
    zeros[r] = blob + lay.off_zeros + rt * KT * SG * 16 + (lane & 15);
  }
  v4f acc[R];
#pragma unroll
  for (int r = 0; r < R; r++) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};

  const int kbeg = wave * a.tpw, kend = min(KT, kbeg + a.tpw);
  const int bc = min(lane & 15, B - 1);
  for (int k0 = kbeg; k0 < kend; k0 += T) {
    uint4 w[R][T];
    v4f sc[R][T][SG];
    uint32_t z[R][T][SG];
#pragma unroll
    for (int t = 0; t < T; t++) {
      const int kt = min(k0 + t, kend - 1);
#pragma unroll
      for (int r = 0; r < R; r++) {
        w[r][t] = codes[r][(size_t)kt * 64];
#pragma unroll
        for (int g = 0; g < SG; g++) {
          sc[r][t][g] = q4_scales(scales[r] + (kt * SG + g) * 16);
          if (ZERO) z[r][t][g] = zeros[r][(kt * SG + g) * 16];
        }
      }
    }
    // x: sixteen lanes take the 128 columns of one (row, tile), eight each; the
    // 16-byte pieces of row b are stored exchanged by b so that the sixteen rows
    // of an operand read lie in different banks
    for (int u = lane >> 4; u < T * B; u += 4) {
      const int t = u % T, b = u / T, j = lane & 15, kt = k0 + t;
      if (kt >= kend) continue;
      float v[8];
      q4_load8(x + (size_t)b * a.n, kt * 128 + 8 * j, a.n, a.xvec, v);
      const int e = q4_block_exp(row16_max(q4_max8(v)));
      h8 hi, lo;
      q4_to_f16<P>(v, e, &hi, &lo);
      const int at = ((t * B + b) * 16 + (j ^ (b & 15))) * 8;
      *reinterpret_cast<h8*>(img + at) = hi;
      if (P == 2) *reinterpret_cast<h8*>(img + T * B * 128 + at) = lo;
      if (j == 0) xfac[t * B + b] = __builtin_ldexpf(1.0f, -e);
    }
    wave_lds_order();
#pragma unroll
    for (int t = 0; t < T; t++) {
      if (k0 + t >= kend) break;
      h8 bh[4], bl[4];
#pragma unroll
      for (int s = 0; s < 4; s++) {
        const int at = ((t * B + bc) * 16 + ((4 * s + (lane >> 4)) ^ (bc & 15))) * 8;
        bh[s] = *reinterpret_cast<const h8*>(img + at);
        if (P == 2) bl[s] = *reinterpret_cast<const h8*>(img + T * B * 128 + at);
      }
      const float f = xfac[t * B + bc];
#pragma unroll
      for (int r = 0; r < R; r++) {
        const uint32_t ww[4] = {w[r][t].x, w[r][t].y, w[r][t].z, w[r][t].w};
#pragma unroll
        for (int g = 0; g < SG; g++) {
          const h2 zc = q4_zero(ZERO ? z[r][t][g] : 8u);
          v4f d{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = g * 4 / SG; s < (g + 1) * 4 / SG; s++) {
            const h8 av = q4_expand(ww[s], zc);
            d = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, bh[s], d, 0, 0, 0);
            if (P == 2) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, bl[s], d, 0, 0, 0);
          }
          const v4f sf = sc[r][t][g] * f;
#pragma unroll
          for (int v = 0; v < 4; v++) acc[r][v] = fmaf(sf[v], d[v], acc[r][v]);
        }
      }
    }
    wave_lds_order();
  }

  // the waves' sums: [row][b] in each wave's own region, added in wave order
  float* red = reinterpret_cast<float*>(mine);
  if ((lane & 15) < B) {
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
      for (int v = 0; v < 4; v++) red[(r * 16 + 4 * (lane >> 4) + v) * B + (lane & 15)] = acc[r][v];
  }
  __syncthreads();
  for (int id = threadIdx.x; id < 16 * R * B; id += blockDim.x) {
    const int row = id % (16 * R), b = id / (16 * R), i = rt0 * 16 + row;
    if (i >= m) continue;
    float s = 0.0f;
    for (int w = 0; w < W; w++) s += *reinterpret_cast<const float*>(smem + w * a.region + (row * B + b) * 4);
    q4_store(a.y[l], a.ydt, (size_t)b * m + i, s);
  }
}

// ------------------------------------------------------------------ prompts: any B
// x as fp16 rows of Kpad columns (zero from column n on) with one power of two a
// row; for fp32 x the remainders follow as a second image.
template <typename XT>
__global__ void __launch_bounds__(256) q4_rows_kernel(const XT* __restrict__ x, int n, int Kpad, int xvec,
                                                      _Float16* __restrict__ hi, _Float16* __restrict__ lo,
                                                      float* __restrict__ fac) {
  constexpr int P = sizeof(XT) == 4 ? 2 : 1;
  __shared__ float red[4];
  const size_t row = blockIdx.x;
  const XT* src = x + row * n;
  float mx = 0.0f, v[8];
  for (int k = 8 * threadIdx.x; k < n; k += 2048) {
    q4_load8(src, k, n, xvec, v);
    mx = fmaxf(mx, q4_max8(v));
  }
  for (int o = 32; o; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const int e = q4_block_exp(mx);
  for (int k = 8 * threadIdx.x; k < Kpad; k += 2048) {
    h8 h, r;
    q4_load8(src, k, n, xvec, v);
    q4_to_f16<P>(v, e, &h, &r);
    *reinterpret_cast<h8*>(hi + row * Kpad + k) = h;
    if (P == 2) *reinterpret_cast<h8*>(lo + row * Kpad + k) = r;
  }
  if (threadIdx.x == 0) fac[row] = __builtin_ldexpf(1.0f, -e);
}

struct Q4GemmArgs {
  const uint8_t* blob;
  const _Float16* img[2];
  const float* fac;
  void* y;      // S == 1: the output; else fp32 partial sums, [S][B][m]
  int m, n, B, KT, ydt, S;
};

constexpr int QM = 128, QB = 128;  // rows of W and of x per workgroup

// One workgroup of four waves: 128 rows of W times 128 rows of x, a wave 64 x 64
// as 4 x 4 MFMA tiles.  A K step is one column tile (128 columns): its x goes
// from memory straight to shared memory one step ahead, the codes of the wave's
// four row tiles to registers one step ahead.
template <typename ST, int SG, bool ZERO, int P>
__global__ void __launch_bounds__(256) q4_gemm_kernel(Q4GemmArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  _Float16* lds = reinterpret_cast<_Float16*>(smem);  // [2][P][QB][128]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int MB = ceil_div(a.m, QM), BB = ceil_div(a.B, QB);
  const long long tiles = (long long)MB * BB * a.S, per = (tiles + 7) / 8;
  // the 8 XCDs take contiguous runs of tiles, rows of W slowest, so that the
  // workgroups that one XCD runs together share their codes
  const long long ts = (long long)(blockIdx.x % 8) * per + blockIdx.x / 8;
  if ((int)(blockIdx.x / 8) >= per || ts >= tiles) return;
  const int split = (int)(ts / ((long long)MB * BB)), t0 = (int)(ts % ((long long)MB * BB));
  const int i0 = t0 / BB * QM, b0 = t0 % BB * QB;
  const int KT = a.KT, Kpad = KT * 128, RT = ceil_div(a.m, 16);
  const int per_split = ceil_div(KT, a.S), kbeg = split * per_split, kend = min(KT, kbeg + per_split);
  const Q4Layout lay = q4_layout(a.m, a.n, 128 / SG, sizeof(ST), ZERO);
  const int wm = (wave >> 1) * 64, wb = (wave & 1) * 64;

  const uint4* codes[4];
  const ST* scales[4];
  const uint8_t* zeros[4];
#pragma unroll
  for (int r = 0; r < 4; r++) {
    const size_t rt = min((i0 + wm) / 16 + r, RT - 1);
    codes[r] = reinterpret_cast<const uint4*>(a.blob + lay.off_codes) + rt * KT * 64 + lane;
    scales[r] = reinterpret_cast<const ST*>(a.blob + lay.off_scales) + rt * KT * SG * 16 + 4 * (lane >> 4);
    zeros[r] = a.blob + lay.off_zeros + rt * KT * SG * 16 + (lane & 15);
  }
  // x tile: 128 rows x 16 pieces of 16 bytes; piece c of row b lies at place
  // c ^ (b & 15) of the row (see the decode kernel), so the place is fixed by the
  // thread and the column it reads from by the exchange
  auto stage = [&](int kt, int buf) {
#pragma unroll
    for (int p = 0; p < P; p++)
#pragma unroll
      for (int c = 0; c < 8; c++) {
        const int id = c * 256 + threadIdx.x, row = id >> 4, col = ((id & 15) ^ (row & 15)) * 8;
        const int b = min(b0 + row, a.B - 1);
        const h8 v = *reinterpret_cast<const h8*>(a.img[p] + (size_t)b * Kpad + kt * 128 + col);
        *reinterpret_cast<h8*>(lds + ((size_t)(buf * P + p) * QB * 16 + id) * 8) = v;
      }
  };

  v4f acc[4][4];
#pragma unroll
  for (int r = 0; r < 4; r++)
#pragma unroll
    for (int c = 0; c < 4; c++) acc[r][c] = v4f{0.f, 0.f, 0.f, 0.f};

  if (kbeg < kend) stage(kbeg, 0);
  __syncthreads();
  for (int kt = kbeg; kt < kend; kt++) {
    const int buf = (kt - kbeg) & 1;
    uint4 w[4];
#pragma unroll
    for (int r = 0; r < 4; r++) w[r] = codes[r][(size_t)kt * 64];
    if (kt + 1 < kend) stage(kt + 1, buf ^ 1);
#pragma unroll
    for (int g = 0; g < SG; g++) {
      v4f d[4][4];
#pragma unroll
      for (int r = 0; r < 4; r++)
#pragma unroll
        for (int c = 0; c < 4; c++) d[r][c] = v4f{0.f, 0.f, 0.f, 0.f};
      h2 zc[4];
#pragma unroll
      for (int r = 0; r < 4; r++) zc[r] = q4_zero(ZERO ? zeros[r][(kt * SG + g) * 16] : 8u);
#pragma unroll
      for (int s = g * 4 / SG; s < (g + 1) * 4 / SG; s++) {
        h8 bv[P][4];
#pragma unroll
        for (int p = 0; p < P; p++)
#pragma unroll
          for (int c = 0; c < 4; c++) {
            const int row = wb + 16 * c + (lane & 15);
            bv[p][c] = *reinterpret_cast<const h8*>(
                lds + ((size_t)(buf * P + p) * QB * 16 + row * 16 + ((4 * s + (lane >> 4)) ^ (row & 15))) * 8);
          }
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const h8 av = q4_expand(s == 0 ? w[r].x : s == 1 ? w[r].y : s == 2 ? w[r].z : w[r].w, zc[r]);
#pragma unroll
          for (int p = 0; p < P; p++)
#pragma unroll
            for (int c = 0; c < 4; c++) d[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, bv[p][c], d[r][c], 0, 0, 0);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const v4f sc = q4_scales(scales[r] + (kt * SG + g) * 16);
#pragma unroll
        for (int c = 0; c < 4; c++)
#pragma unroll
          for (int v = 0; v < 4; v++) acc[r][c][v] = fmaf(sc[v], d[r][c][v], acc[r][c][v]);
      }
    }
    __syncthreads();
  }

#pragma unroll
  for (int c = 0; c < 4; c++) {
    const int b = b0 + wb + 16 * c + (lane & 15);
    if (b >= a.B) continue;
    const float f = a.fac[b];
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const int i = i0 + wm + 16 * r + 4 * (lane >> 4) + v;
        if (i >= a.m) continue;
        if (a.S > 1) reinterpret_cast<float*>(a.y)[((size_t)split * a.B + b) * a.m + i] = acc[r][c][v] * f;
        else q4_store(a.y, a.ydt, (size_t)b * a.m + i, acc[r][c][v] * f);
      }
  }
}

// y = the S partial sums added in order.
__global__ void __launch_bounds__(256) q4_join_kernel(const float* __restrict__ part, int S, size_t count, void* y,
                                                      int ydt) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= count) return;
  float s = part[i];
  for (int k = 1; k < S; k++) s += part[k * count + i];
  q4_store(y, ydt, i, s);
}

// ------------------------------------------------------------------ host
template <typename XT, typename ST, int SG, bool ZERO, int T>
hipError_t launch_dec(const Q4DecArgs& a, int R, dim3 grid, int W, hipStream_t s) {
  const size_t lds = (size_t)W * a.region;
  if (R == 2) hipLaunchKernelGGL((q4_dec_kernel<XT, ST, SG, ZERO, T, 2>), grid, dim3(64 * W), lds, s, a);
  else hipLaunchKernelGGL((q4_dec_kernel<XT, ST, SG, ZERO, T, 1>), grid, dim3(64 * W), lds, s, a);
  return hipGetLastError();
}

// Calls f with the compile-time scale type, groups per tile and zero points.
template <typename F>
auto q4_dispatch(int scale_dtype, int group, bool zeros, F f) {
  auto by_zero = [&](auto st, auto sg) {
    return zeros ? f(st, sg, std::true_type{}) : f(st, sg, std::false_type{});
  };
  auto by_group = [&](auto st) {
    return group == 32   ? by_zero(st, std::integral_constant<int, 4>{})
           : group == 64 ? by_zero(st, std::integral_constant<int, 2>{})
                         : by_zero(st, std::integral_constant<int, 1>{});
  };
  return scale_dtype == 1 ? by_group(_Float16{}) : by_group(float{});
}

// Workgroups of a pack kernel: its threads stride over the words, so that the
// launch stays far below 2^32 threads for every weight.
dim3 q4_pack_grid(long long items) {
  const long long g = (items + 255) / 256;
  return dim3((unsigned)(g < (1 << 20) ? g : (1 << 20)));
}

template <typename XT>
hipError_t dec_chunk(const Q4Args& a, int b0, int B) {
  constexpr int P = sizeof(XT) == 4 ? 2 : 1;
  Q4DecArgs k{};
  k.L = a.L;
  k.n = a.n;
  k.KT = ceil_div(a.n, 128);
  k.B = B;
  k.ydt = a.y_dtype;
  const XT* x = static_cast<const XT*>(a.x) + (size_t)b0 * a.n;
  k.x = x;
  k.xvec = a.n % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  int RT = 0;
  for (int l = 0; l < a.L; l++) RT += ceil_div(a.m[l], 16);
  const int R = RT >= 512 ? 2 : 1;
  const int W = k.KT >= 16 ? 16 : k.KT;
  const int T = B * P <= 8 ? 4 : B * P <= 16 ? 2 : 1;
  k.tpw = ceil_div(k.KT, W);
  const int image = T * B * (256 * P + 4), sums = 16 * R * B * 4;
  k.region = (int)align_up(image > sums ? image : sums, 16);
  int end = 0;
  for (int l = 0; l < a.L; l++) {
    k.blob[l] = a.blob[l];
    k.y[l] = static_cast<uint8_t*>(a.y[l]) + (size_t)b0 * a.m[l] * (a.y_dtype == 0 ? 4 : 2);
    k.m[l] = a.m[l];
    end += ceil_div(ceil_div(a.m[l], 16), R);
    k.wg_end[l] = end;
  }
  return q4_dispatch(a.scale_dtype, a.group, a.zeros, [&](auto st, auto sg, auto zero) {
    using ST = decltype(st);
    constexpr int SG = decltype(sg)::value;
    constexpr bool Z = decltype(zero)::value;
    return T == 4   ? launch_dec<XT, ST, SG, Z, 4>(k, R, dim3(end), W, a.stream)
           : T == 2 ? launch_dec<XT, ST, SG, Z, 2>(k, R, dim3(end), W, a.stream)
                    : launch_dec<XT, ST, SG, Z, 1>(k, R, dim3(end), W, a.stream);
  });
}

}  // namespace

Q4GemmPlan q4_gemm_plan(int m, int n, int B, int x_dtype) {
  Q4GemmPlan p{};
  const int KT = ceil_div(n, 128), P = x_dtype == 0 ? 2 : 1;
  const long long tiles = (long long)ceil_div(m, QM) * ceil_div(B, QB);
  int S = 1;
  while (tiles * S < 384 && S < 8 && KT / (2 * S) >= 4) S *= 2;
  p.S = ceil_div(KT, ceil_div(KT, S));
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  p.off_hi = take((size_t)B * KT * 256);
  p.off_lo = take(P == 2 ? (size_t)B * KT * 256 : 0);
  p.off_fac = take((size_t)B * 4);
  p.off_part = take(p.S > 1 ? (size_t)p.S * B * m * 4 : 0);
  p.bytes = o;
  return p;
}

size_t q4_workspace(const int* m, int L, int n, int B, int x_dtype) {
  if (B <= Q4_DEC_MAX) return 0;
  size_t need = 0;
  for (int l = 0; l < L; l++) {
    const size_t b = q4_gemm_plan(m[l], n, B, x_dtype).bytes;
    need = b > need ? b : need;
  }
  return need;
}

template <typename XT>
static hipError_t gemm_layer(const Q4Args& a, int l, bool image) {
  constexpr int P = sizeof(XT) == 4 ? 2 : 1;
  const Q4GemmPlan p = q4_gemm_plan(a.m[l], a.n, a.B, a.x_dtype);
  Q4GemmArgs k{};
  k.blob = a.blob[l];
  k.img[0] = reinterpret_cast<const _Float16*>(a.ws + p.off_hi);
  k.img[1] = reinterpret_cast<const _Float16*>(a.ws + p.off_lo);
  k.fac = reinterpret_cast<const float*>(a.ws + p.off_fac);
  k.m = a.m[l];
  k.n = a.n;
  k.B = a.B;
  k.KT = ceil_div(a.n, 128);
  k.ydt = a.y_dtype;
  k.S = p.S;
  k.y = p.S > 1 ? static_cast<void*>(a.ws + p.off_part) : a.y[l];
  if (image) {
    const int xvec = a.n % 8 == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
    hipLaunchKernelGGL((q4_rows_kernel<XT>), dim3(a.B), dim3(256), 0, a.stream, static_cast<const XT*>(a.x), a.n,
                       k.KT * 128, xvec, reinterpret_cast<_Float16*>(a.ws + p.off_hi),
                       reinterpret_cast<_Float16*>(a.ws + p.off_lo), reinterpret_cast<float*>(a.ws + p.off_fac));
  }
  const long long tiles = (long long)ceil_div(k.m, QM) * ceil_div(k.B, QB) * k.S;
  const dim3 grid((unsigned)(8 * ((tiles + 7) / 8)));
  q4_dispatch(a.scale_dtype, a.group, a.zeros, [&](auto st, auto sg, auto zero) {
    using ST = decltype(st);
    auto kernel = q4_gemm_kernel<ST, decltype(sg)::value, decltype(zero)::value, P>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 2 * P * QB * 256, a.stream, k);
    return 0;
  });
  if (p.S > 1) {
    const size_t count = (size_t)a.B * a.m[l];
    hipLaunchKernelGGL(q4_join_kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, a.stream,
                       reinterpret_cast<const float*>(a.ws + p.off_part), p.S, count, a.y[l], a.y_dtype);
  }
  return hipGetLastError();
}

hipError_t q4_forward(const Q4Args& a) {
  hipError_t e = hipSuccess;
  if (a.B <= Q4_DEC_MAX) {
    for (int b0 = 0; b0 < a.B && e == hipSuccess; b0 += 16) {
      const int B = a.B - b0 < 16 ? a.B - b0 : 16;
      e = a.x_dtype == 0 ? dec_chunk<float>(a, b0, B) : dec_chunk<uint16_t>(a, b0, B);
    }
    return e;
  }
  // the image of x lies at the same place for every layer of the group
  for (int l = 0; l < a.L && e == hipSuccess; l++)
    e = a.x_dtype == 0 ? gemm_layer<float>(a, l, l == 0) : gemm_layer<uint16_t>(a, l, l == 0);
  return e;
}

hipError_t q4_pack(const Q4Layout& lay, int m, int n, int group, int scale_bytes, const uint8_t* q, const void* s,
                   const uint8_t* z, uint8_t* blob, int* bad, hipStream_t st) {
  const int KT = ceil_div(n, 128), SG = 128 / group, ng = ceil_div(n, group);
  const long long words = (long long)ceil_div(m, 16) * KT * 256, entries = (long long)ceil_div(m, 16) * KT * SG * 16;
  const dim3 gw = q4_pack_grid(words), ge = q4_pack_grid(entries);
  hipLaunchKernelGGL(q4_pack_codes_kernel, gw, dim3(256), 0, st, q, m, n, KT, words,
                     reinterpret_cast<uint32_t*>(blob + lay.off_codes), bad);
  if (scale_bytes == 2)
    hipLaunchKernelGGL((q4_pack_groups_kernel<uint16_t>), ge, dim3(256), 0, st, static_cast<const uint16_t*>(s), m, ng,
                       KT, SG, entries, reinterpret_cast<uint16_t*>(blob + lay.off_scales), 0, bad);
  else
    hipLaunchKernelGGL((q4_pack_groups_kernel<uint32_t>), ge, dim3(256), 0, st, static_cast<const uint32_t*>(s), m, ng,
                       KT, SG, entries, reinterpret_cast<uint32_t*>(blob + lay.off_scales), 0, bad);
  if (z)
    hipLaunchKernelGGL((q4_pack_groups_kernel<uint8_t>), ge, dim3(256), 0, st, z, m, ng, KT, SG, entries,
                       blob + lay.off_zeros, 15, bad);
  return hipGetLastError();
}

hipError_t q4_unpack(const Q4Layout& lay, int m, int n, int group, const uint8_t* blob, uint8_t* q, uint8_t* z,
                     hipStream_t st) {
  const int KT = ceil_div(n, 128), SG = 128 / group, ng = ceil_div(n, group);
  const long long words = (long long)ceil_div(m, 16) * KT * 256, entries = (long long)ceil_div(m, 16) * KT * SG * 16;
  hipLaunchKernelGGL(q4_unpack_kernel, q4_pack_grid(words), dim3(256), 0, st,
                     reinterpret_cast<const uint32_t*>(blob + lay.off_codes), m, n, KT, words, q);
  if (z)
    hipLaunchKernelGGL(q4_unpack_zeros_kernel, q4_pack_grid(entries), dim3(256), 0, st,
                       blob + lay.off_zeros, m, ng, KT, SG, entries, z);
  return hipGetLastError();
}

}  // namespace nq
