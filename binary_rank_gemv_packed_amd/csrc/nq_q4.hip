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
// below is under 2^-39 of it, or under 2^-144.  An fp32 value is taken as two fp16 pieces, the
// rounded value and its rounded remainder, off by at most 2^-22 of itself.  So
// the products are exact or nearly so, the sums over a group are held by the
// fp16 MFMA in fp32; s multiplies the group's sum and then the block's power of two
// the product, both in fp32 (in the prompt kernel once for the whole row, whose
// sum of s times integers stays below 2^119 by Q4_SCALE_LIMIT).  y is rounded once.
#include "nq_common.h"
#include "nq_internal.h"
#include "nq_q4_lds.h"

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

// Row of W and group of its row that an entry of the scales (quad = 4) or zero
// points (quad = 1) belongs to.
__device__ inline void q4_group_entry(long long id, int KT, int SG, int quad, int* row, int* g) {
  const int within = (int)(id % (16 * SG));
  const long long tile = id / (16 * SG);
  *row = (int)(tile / KT) * 16 + within / (quad * SG) * quad + within % quad;
  *g = (int)(tile % KT) * SG + within / quad % SG;
}

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
    if (bad) atomicOr(bad_flag, Q4_BAD_CODE);
  }
}

// One thread per entry of the scales (quad = 4: four rows of a group together)
// or the zero points (quad = 1: a row's groups together).  Zero points above 15
// and fp32 scales of a finite magnitude of Q4_SCALE_LIMIT or more are reported.
template <typename T>
__global__ void __launch_bounds__(256) q4_pack_groups_kernel(const T* __restrict__ in, int m, int ng, int KT, int SG,
                                                             int quad, long long entries, T* __restrict__ out,
                                                             int* __restrict__ bad_flag) {
  for (long long id = (long long)blockIdx.x * 256 + threadIdx.x; id < entries; id += (long long)gridDim.x * 256) {
    int row, g;
    q4_group_entry(id, KT, SG, quad, &row, &g);
    T v = 0;
    if (row < m && g < ng) v = in[(size_t)row * ng + g];
    if (sizeof(T) == 1 && v > 15) atomicOr(bad_flag, Q4_BAD_CODE);
    if (sizeof(T) == 4) {
      const float scale = fabsf(__uint_as_float((uint32_t)v));
      if (scale >= Q4_SCALE_LIMIT && scale < INFINITY) atomicOr(bad_flag, Q4_BAD_SCALE);
    }
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
    int row, g;
    q4_group_entry(id, KT, SG, 1, &row, &g);
    if (row < m && g < ng) z[(size_t)row * ng + g] = in[id];
  }
}

// ------------------------------------------------------------------ shared pieces
// A zero point ready for both places a code can have in a half: -(1024 + z) for
// the four lowest bits of the mantissa, -(64 + z) for the four above them.
struct Q4Zero {
  h2 low, high;
};
__device__ __forceinline__ Q4Zero q4_zero(uint32_t z) {
  const uint32_t zz = z | (z << 16);
  return {__builtin_bit_cast(h2, zz | 0xE400E400u), __builtin_bit_cast(h2, (zz << 4) | 0xD400D400u)};
}

// The magic numbers of q4_expand, out of the compiler's sight: as constants they
// would cost an instruction of their own at each use (an instruction takes one
// constant; and-then-or would need two).
struct Q4Magic {
  uint32_t low = 0x64006400u, high = 0x54005400u;
  __device__ __forceinline__ Q4Magic() { asm("" : "+v"(low), "+v"(high)); }
};

// The eight codes of a word less their zero point, as an MFMA operand: column
// order 0..7.  1024 + q is 0x6400 with q in the lowest bits, 64 + q is 0x5400
// with q four bits up, so that of a word's four pairs only two need a shift:
// nine instructions a word.
__device__ __forceinline__ h8 q4_expand(uint32_t w, const Q4Zero& z, const Q4Magic& magic) {
  union {
    h2 p[4];
    h8 v;
  } u;
  const uint32_t v = w >> 8;
  u.p[0] = __builtin_bit_cast(h2, (w & 0x000F000Fu) | magic.low) + z.low;
  u.p[1] = __builtin_bit_cast(h2, (w & 0x00F000F0u) | magic.high) + z.high;
  u.p[2] = __builtin_bit_cast(h2, (v & 0x000F000Fu) | magic.low) + z.low;
  u.p[3] = __builtin_bit_cast(h2, (v & 0x00F000F0u) | magic.high) + z.high;
  return u.v;
}

// A lane's four rows of scales of every group of a tile, kept as they are stored
// until they are used, and its row's zero points.
template <typename ST, int SG>
struct Q4Scales {
  typedef ST v4 __attribute__((ext_vector_type(4)));
  v4 v[SG];
  __device__ __forceinline__ void load(const uint8_t* base, size_t tile, int lane) {
    typedef ST row __attribute__((ext_vector_type(4 * SG)));
    const row r = reinterpret_cast<const row*>(base)[tile * 4 + (lane >> 4)];
#pragma unroll
    for (int g = 0; g < SG; g++)
#pragma unroll
      for (int i = 0; i < 4; i++) v[g][i] = r[4 * g + i];
  }
  __device__ __forceinline__ float get(int g, int i) const { return (float)v[g][i]; }
};
template <int SG, bool ZERO>
struct Q4Zeros {
  uint32_t z;
  __device__ __forceinline__ void load(const uint8_t* base, size_t tile, int lane) {
    if (!ZERO) return;
    const size_t at = tile * 16 + (lane & 15);
    z = SG == 1 ? base[at]
        : SG == 2 ? reinterpret_cast<const uint16_t*>(base)[at] : reinterpret_cast<const uint32_t*>(base)[at];
  }
  __device__ __forceinline__ uint32_t get(int g) const { return !ZERO ? 8u : SG == 1 ? z : (z >> (8 * g)) & 255u; }
};

// Columns k .. k+7 of a row of x (zero from column n on), as they are stored
// until get().  The 16-byte reads need not be aligned: a row of an odd width starts
// anywhere.
typedef float v4f_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
template <typename XT>
struct Q4X;
template <>
struct Q4X<float> {
  v4f a, b;
  __device__ __forceinline__ void load(const float* x, int k, int n) {
    if (k + 8 <= n) {
      a = *reinterpret_cast<const v4f_at4*>(x + k);
      b = *reinterpret_cast<const v4f_at4*>(x + k + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        a[i] = k + i < n ? x[k + i] : 0.0f;
        b[i] = k + 4 + i < n ? x[k + 4 + i] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = a[i], v[4 + i] = b[i];
  }
  // bits of the largest magnitude; FINITE: of the largest below infinity
  template <bool FINITE>
  __device__ __forceinline__ uint32_t top() const {
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t u = __float_as_uint(i < 4 ? a[i & 3] : b[i & 3]) & 0x7fffffffu;
      mx = max(mx, FINITE && u >= 0x7f800000u ? 0u : u);
    }
    return mx;
  }
};
template <>
struct Q4X<uint16_t> {
  u32x4 a;
  __device__ __forceinline__ void load(const uint16_t* x, int k, int n) {
    if (k + 8 <= n) {
      a = *reinterpret_cast<const u32x4_at2*>(x + k);
    } else {
      uint32_t u[8];
#pragma unroll
      for (int i = 0; i < 8; i++) u[i] = k + i < n ? x[k + i] : 0u;
      a = u32x4{u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16};
    }
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
  template <bool FINITE>
  __device__ __forceinline__ uint32_t top() const {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 mx = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      u16x2 v = __builtin_bit_cast(u16x2, a[i] & 0x7fff7fffu);
      if (FINITE) {
        v[0] = v[0] >= 0x7f80 ? 0 : v[0];
        v[1] = v[1] >= 0x7f80 ? 0 : v[1];
      }
      mx = __builtin_elementwise_max(mx, v);
    }
    return (uint32_t)max(mx[0], mx[1]) << 16;
  }
};

// Power of two that puts a block whose largest magnitude has these bits (of an
// fp32 number, below infinity) into fp16: the largest times 2^e lies in
// [2^14, 2^15).  e <= 120 keeps 2^-e a normal number; fp16 then ends at 2^-24-120.
__device__ __forceinline__ int q4_block_exp(uint32_t mx) {
  const int e = 14 + 127 - (int)(mx >> 23);
  return mx == 0 ? 0 : e < 120 ? e : 120;
}

// 2^e as a float, -126 <= e <= 127.
__device__ __forceinline__ float q4_exp2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// v 2^e as fp16 (f = 2^e), with P = 2 its remainder too.
template <int P>
__device__ __forceinline__ void q4_to_f16(const float* v, float f, h8* hi, h8* lo) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float s = v[i] * f;
    const _Float16 h = (_Float16)s;
    (*hi)[i] = h;
    // an infinity or NaN has no remainder
    if (P == 2) (*lo)[i] = fabsf(s) < INFINITY ? (_Float16)(s - (float)h) : (_Float16)0.0f;
  }
}

// Maximum over the 16 lanes of a row of the wavefront.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
#define NQ_ROR_MAX(n) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + (n), 0xf, 0xf, false))
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

// ------------------------------------------------------------------ decode: B <= 16
struct Q4DecLayer {
  const uint8_t *codes, *scales, *zeros;
  void* out;    // y, or with S > 1 the first split's partial sums
  int m, rt_end;  // rows; row tiles up to this layer's end, counted through
};
struct Q4DecArgs {
  Q4DecLayer layer[GROUP_MAX];
  const void* x;
  int n, KT, B, rows;     // rows: row tiles of all layers
  int range, tpw, steps;  // column tiles of a split, of a wave; units of a wave's row tile
  int shared;             // the waves share each row tile; else each has its own
  int groups;             // workgroups of one split
  int tw;                 // log2 of the tiles that the workgroup turns over side by side
  int keep;               // row tiles whose shared sums are kept before they are added
  int odt;                // dtype of out
  size_t part_split;      // values between the splits' partial sums
};

// The codes, scales and zero points of one tile, as one lane holds them.
template <typename ST, int SG, bool ZERO>
struct Q4Tile {
  u32x4 w;
  Q4Scales<ST, SG> sc;
  Q4Zeros<SG, ZERO> z;
};

// A workgroup of W waves holds the columns of its split of x as fp16 in shared
// memory and goes through row tiles.  Either all waves share a row tile, each a
// run of tpw column tiles, and their sums meet in shared memory, or (shared = 0)
// each wave has a row tile to itself.  A wave's tiles, row tile after row tile,
// are one sequence of units of U tiles; a ring of D units is in flight, and a
// place of the ring is asked for anew as soon as its unit has been multiplied, so
// that the reads do not pause for the sums at the end of a row tile.  Lane layout
// of the 16x16x32 MFMA: the first operand has row lane & 15 and columns
// 8 (lane >> 4) .. + 7, the second row b = lane & 15 of x and the same columns; the
// result has row 4 (lane >> 4) + v of the tile for b = lane & 15.  Lanes with
// b >= B repeat row B - 1 and are not stored.
// Bound by the reads: gate and up of a 70B block (2 x 28672 x 8192, one row) take
// 45 to 47 us over runs, 5.2 TB/s, a bare read of as many bytes 37.9 us; one 8192 x
// 8192 9.7 to 10.2 us.
// A tile costs a wave about 70 vector instructions, half the issue slots.
// STREAM: codes that no cache will hold until the next call are read past the
// caches' replacement (host side: q4_streams).
template <typename XT, typename ST, int SG, bool ZERO, int U, int D, bool STREAM>
__global__ void __launch_bounds__(1024) q4_dec_kernel(Q4DecArgs a) {
  constexpr int P = sizeof(XT) == 4 ? 2 : 1;
  constexpr int XN = 8 / P;  // pieces of x that a thread reads at a time
  constexpr int PRE = (U + 1) / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 63, W = blockDim.x >> 6, B = a.B, KT = a.KT;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x / a.groups, group = blockIdx.x % a.groups;
  const int k_lo = split * a.range, k_hi = min(KT, k_lo + a.range), KR = a.range;
  _Float16* img = reinterpret_cast<_Float16*>(smem);                        // [P][KR][B][128]
  float* xfac = reinterpret_cast<float*>(smem + (size_t)P * KR * B * 256);  // [KR][B]
  float* red = xfac + q4_dec_fac_floats(B, KR);                             // [keep][W][B][16]

  const bool shared = a.shared;
  const int wr = shared ? 0 : wave, WR = shared ? 1 : W;
  const int kbeg = k_lo + (shared ? wave * a.tpw : 0), kend = min(k_hi, kbeg + a.tpw);
  const int rows = a.rows, stride = a.groups * WR, first = group * WR;
  // row tiles that the workgroup goes through (wave 0 has most) and units of a
  // wave's sequence, the same for every wave: the barriers are met by all
  const int turns = (rows - first + stride - 1) / stride;
  int to_ask = turns * a.steps;

  // ---- the sequence of units to be asked for.  A layer's pointers are read anew
  // only where one layer ends and the next begins.
  Q4Tile<ST, SG, ZERO> ring[D][U];
  const uint8_t *codes = a.layer[0].codes, *scales = a.layer[0].scales, *zeros = a.layer[0].zeros;
  int ask_l = 0, ask_lo = 0, ask_hi = a.layer[0].rt_end, ask_rt = first + wr, ask_step = 0;
  size_t ask_tile;
  auto seek = [&]() {
    const int rt = min(ask_rt, rows - 1);
    while (rt >= ask_hi) {
      ask_l++;
      ask_lo = ask_hi;
      ask_hi = a.layer[ask_l].rt_end;
      codes = a.layer[ask_l].codes;
      scales = a.layer[ask_l].scales;
      zeros = a.layer[ask_l].zeros;
    }
    ask_tile = (size_t)(rt - ask_lo) * KT;
  };
  auto load = [&](Q4Tile<ST, SG, ZERO>& q, int t) {
    // past the run its last tile is asked for again
    const size_t tile = ask_tile + max(min(kbeg + ask_step * U + t, kend - 1), 0);
    const u32x4* w = reinterpret_cast<const u32x4*>(codes + tile * 1024) + lane;
    q.w = STREAM ? __builtin_nontemporal_load(w) : *w;
    q.sc.load(scales, tile, lane);
    q.z.load(zeros, tile, lane);
  };
  auto asked = [&]() {  // a whole unit
    to_ask--;
    if (++ask_step == a.steps) {
      ask_step = 0;
      ask_rt += stride;
      seek();
    }
  };
  // ---- x: sixteen lanes take the 128 columns of one (tile, row), eight each; the
  // 16-byte pieces of row b are stored exchanged by b so that the sixteen rows
  // of an operand read lie in different banks.  All of x is asked for before any
  // code: behind the codes of the other waves it would come microseconds later.
  const int units = turns * a.steps;
  {
    const XT* x = reinterpret_cast<const XT*>(a.x);
    // the workgroup's groups of sixteen lanes as TW tiles x BW rows; a group goes
    // through rows b0, b0 + BW, ... of tiles t0, t0 + TW, ... (powers of two: a
    // division by B would cost as much as the turning over)
    const int j = lane & 15, g = threadIdx.x >> 4, span = k_hi - k_lo;
    const int TW = 1 << a.tw, BW = max((int)(blockDim.x >> 4) >> a.tw, 1);
    const int t0 = g & (TW - 1), b0 = g >> a.tw;
    const int pieces = ceil_div(span, TW) * ceil_div(B, BW);
    Q4X<XT> raw[XN];
    int tf = t0, bf = b0, tt = t0, bt = b0;  // the next to fetch and to turn over
    auto advance = [&](int& t, int& b) {
      b += BW;
      if (b >= B) {
        b = b0;
        t += TW;
      }
    };
    auto fetch = [&](int count) {
#pragma unroll
      for (int i = 0; i < XN; i++) {
        if (i >= count) break;
        raw[i].load(x + (size_t)min(bf, B - 1) * a.n, (k_lo + min(tf, span - 1)) * 128 + 8 * j, a.n);
        advance(tf, bf);
      }
    };
    auto turn_over = [&](int count) {
#pragma unroll
      for (int i = 0; i < XN; i++) {
        if (i >= count) break;
        uint32_t mx = row16_max(raw[i].template top<false>());
        if (mx >= 0x7f800000u) mx = row16_max(raw[i].template top<true>());
        const int e = q4_block_exp(mx);
        float v[8];
        raw[i].get(v);
        h8 hi, lo;
        q4_to_f16<P>(v, q4_exp2(e), &hi, &lo);
        const int t = tt, b = bt;
        advance(tt, bt);
        if (t >= span || b >= B) continue;
        const int u = t * B + b, at = (u * 16 + (j ^ (b & 15))) * 8;
        *reinterpret_cast<h8*>(img + at) = hi;
        if (P == 2) *reinterpret_cast<h8*>(img + (size_t)KR * B * 128 + at) = lo;
        if (j == 0) xfac[u] = q4_exp2(-e);
      }
    };
    int left = pieces;
    for (; left > XN; left -= XN) {
      fetch(XN);
      turn_over(XN);
    }
    fetch(left);
    __builtin_amdgcn_s_barrier();
    seek();
#pragma unroll
    for (int t = 0; t < PRE; t++) load(ring[0][t], t);
    turn_over(left);
  }
#pragma unroll
  for (int t = PRE; t < U; t++) load(ring[0][t], t);
  asked();
  __syncthreads();
#pragma unroll
  for (int i = 1; i < D; i++) {
#pragma unroll
    for (int t = 0; t < U; t++) load(ring[i][t], t);
    asked();
  }

  // ---- the sequence of units to be multiplied
  const Q4Magic magic;
  const int bc = min(lane & 15, B - 1);
  int step = 0, rt = first + wr, kept = 0;
  v4f acc{0.f, 0.f, 0.f, 0.f};
  int out_l = 0, out_lo = 0, out_hi = a.layer[0].rt_end, out_m = a.layer[0].m;
  void* out = a.layer[0].out;
  const size_t out_split = split * a.part_split;
  auto put = [&](int rt, int row, int b, float v) {
    while (rt >= out_hi) {
      out_l++;
      out_lo = out_hi;
      out_hi = a.layer[out_l].rt_end;
      out_m = a.layer[out_l].m;
      out = a.layer[out_l].out;
    }
    const int i = (rt - out_lo) * 16 + row;
    if (i < out_m) q4_store(out, a.odt, out_split + (size_t)b * out_m + i, v);
  };
  // The end of a row tile.  A wave that has it to itself stores its sums.  Shared
  // sums are kept in shared memory, a.keep row tiles of them, and added when it is
  // full or all row tiles are done, so that the waves seldom wait for each other:
  // four lanes add a quarter of the waves' sums each, then the four.
  auto finish = [&]() {
    if (!shared) {
      if (rt < rows)
#pragma unroll
        for (int v = 0; v < 4; v++)
          if ((lane & 15) < B) put(rt, 4 * (lane >> 4) + v, lane & 15, acc[v]);
    } else {
      if ((lane & 15) < B)
        *reinterpret_cast<v4f*>(red + ((kept * W + wave) * B + (lane & 15)) * 16 + 4 * (lane >> 4)) = acc;
      kept++;
      if (kept == a.keep || rt + stride >= rows) {
        __syncthreads();
        const int rt0 = rt - (kept - 1) * stride;
        for (int id = wave; id < kept * B; id += W) {
          const int i = id / B, b = id % B;
          const float* r = red + (i * W * B + b) * 16 + (lane & 15);
          float s = 0.0f;
#pragma unroll
          for (int q = 0; q < 4; q++) {
            const int w = 4 * q + (lane >> 4);
            if (w < W) s += r[w * B * 16];
          }
          s += __shfl_xor(s, 16);
          s += __shfl_xor(s, 32);
          if (lane < 16) put(rt0 + i * stride, lane, b, s);
        }
        kept = 0;
        __syncthreads();
      }
    }
    acc = v4f{0.f, 0.f, 0.f, 0.f};
    rt += stride;
  };
  auto multiply = [&](const Q4Tile<ST, SG, ZERO>& q, int t) {
    const int kt = kbeg + step * U + t;
    if (kt >= kend) return;
    const int u = (kt - k_lo) * B + bc;
    h8 bh[4], bl[4];
#pragma unroll
    for (int s = 0; s < 4; s++) {
      const int at = (u * 16 + ((4 * s + (lane >> 4)) ^ (bc & 15))) * 8;
      bh[s] = *reinterpret_cast<const h8*>(img + at);
      if (P == 2) bl[s] = *reinterpret_cast<const h8*>(img + (size_t)KR * B * 128 + at);
    }
    const float f = xfac[u];
    const uint32_t ww[4] = {q.w.x, q.w.y, q.w.z, q.w.w};
#pragma unroll
    for (int g = 0; g < SG; g++) {
      const Q4Zero zc = q4_zero(q.z.get(g));
      v4f d{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = g * 4 / SG; s < (g + 1) * 4 / SG; s++) {
        const h8 av = q4_expand(ww[s], zc, magic);
        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, bh[s], d, 0, 0, 0);
        if (P == 2) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, bl[s], d, 0, 0, 0);
      }
      // The scale first, though that rounds once more: f (2^-120 .. 2^113) times d
      // alone passes fp32 where x is large and the scale small, and loses bits
      // where x is tiny.  (fmaf with 0, for a scale in fp16 is an operand of it.)
#pragma unroll
      for (int v = 0; v < 4; v++) acc[v] = fmaf(fmaf(q.sc.get(g, v), d[v], 0.0f), f, acc[v]);
    }
  };
  auto multiplied = [&]() {  // a whole unit
    if (++step == a.steps) {
      step = 0;
      finish();
    }
  };

  // rounds of the ring, then the units that are left in it.  What a last round
  // asks for past the end is the last row tile, which the L2 holds by then.
  int left = units;
  for (; to_ask > 0; left -= D)
#pragma unroll
    for (int i = 0; i < D; i++) {
#pragma unroll
      for (int t = 0; t < U; t++) {
        multiply(ring[i][t], t);
        load(ring[i][t], t);
      }
      asked();
      multiplied();
    }
#pragma unroll
  for (int i = 0; i < D; i++)
    if (i < left) {
#pragma unroll
      for (int t = 0; t < U; t++) multiply(ring[i][t], t);
      multiplied();
    }
}

// ------------------------------------------------------------------ prompts: any B
// x as fp16 rows of Kpad columns (zero from column n on) with one power of two a
// row; for fp32 x the remainders follow as a second image.
template <typename XT>
__global__ void __launch_bounds__(256) q4_rows_kernel(const XT* __restrict__ x, int n, int Kpad,
                                                      _Float16* __restrict__ hi, _Float16* __restrict__ lo,
                                                      float* __restrict__ fac) {
  constexpr int P = sizeof(XT) == 4 ? 2 : 1;
  __shared__ uint32_t red[4];
  const size_t row = blockIdx.x;
  const XT* src = x + row * n;
  uint32_t mx = 0;
  Q4X<XT> raw;
  for (int k = 8 * threadIdx.x; k < n; k += 2048) {
    raw.load(src, k, n);
    mx = max(mx, raw.template top<true>());
  }
  for (int o = 32; o; o >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
  __syncthreads();
  const int e = q4_block_exp(max(max(red[0], red[1]), max(red[2], red[3])));
  for (int k = 8 * threadIdx.x; k < Kpad; k += 2048) {
    float v[8];
    h8 h, r;
    raw.load(src, k, n);
    raw.get(v);
    q4_to_f16<P>(v, q4_exp2(e), &h, &r);
    *reinterpret_cast<h8*>(hi + row * Kpad + k) = h;
    if (P == 2) *reinterpret_cast<h8*>(lo + row * Kpad + k) = r;
  }
  if (threadIdx.x == 0) fac[row] = q4_exp2(-e);
}

struct Q4GemmArgs {
  const uint8_t* blob;
  const _Float16* img[2];
  const float* fac;
  void* y;      // S == 1: the output; else fp32 partial sums, [S][B][m]
  int m, n, B, KT, ydt, S;
  int quads;    // m a multiple of 4 and y aligned to four values
};

constexpr int QM = 128;  // rows of W per workgroup

// Waits for every read of this wave, those straight to shared memory among them;
// no access to memory moves across.
__device__ __forceinline__ void wait_vmem() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// One workgroup of four waves: 128 rows of W times QB = 16 NC rows of x (128, or 64
// for batches of up to 64), a wave 32 rows of W times all of x as 2 x NC MFMA
// tiles: no two waves expand the same codes.  (Waves of 64 x 64, which read half
// as much from shared memory but expand every code twice: 2048 x 4096 -> 11008,
// 215 us against 200 us; 34 x 9728 -> 8832 with groups of 32, 78 against 41 us.)
// A K step is one column tile (128 columns): its x goes from memory straight to
// shared memory one step ahead, the codes of the wave's two row tiles to registers
// one step ahead.  2048 x 4096 -> 11008, groups of 128: 199 to 205 us with
// q4_rows_kernel over runs, 900 to 930 TFLOP/s (each launch by itself in a kernel
// trace: 217 and 8.5 us); matrix unit busy 0.39 of the time, vector issue 0.38.
// The launch bound fits groups of 128.  Groups of 64 with fp16 scales need about
// 340 registers and have 256: 192 to 216 bytes a lane go through scratch memory in
// the K loop, 849 us for the same product (groups of 32, 483 us; fp32 x, one wave a
// SIMD, 498 us).
template <typename ST, int SG, bool ZERO, int P, int NC>
__global__ void __launch_bounds__(256, NC == 4 || (P == 1 && SG * sizeof(ST) <= 4) ? 2 : 1)
    q4_gemm_kernel(Q4GemmArgs a) {
  constexpr int QB = 16 * NC;  // rows of x per workgroup
  // two arrays of their own, so that reads of one do not wait for writes to the other
  __shared__ __align__(16) _Float16 lds0[P * QB * 128], lds1[P * QB * 128];
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
  const int wm = wave * 32;

  const uint8_t *codes = a.blob + lay.off_codes, *scales = a.blob + lay.off_scales, *zeros = a.blob + lay.off_zeros;
  size_t row_tile[2];  // first tile of the wave's row tiles
#pragma unroll
  for (int r = 0; r < 2; r++) row_tile[r] = (size_t)min((i0 + wm) / 16 + r, RT - 1) * KT;
  // x tile: 128 rows x 16 pieces of 16 bytes; piece c of row b lies at place
  // c ^ (b & 15) of the row (see the decode kernel), so the place is fixed by the
  // thread and the column it reads from by the exchange
  auto fetch = [&](int kt, _Float16* to) {
#pragma unroll
    for (int p = 0; p < P; p++)
#pragma unroll
      for (int c = 0; c < QB / 16; c++) {
        const int id = c * 256 + threadIdx.x, row = id >> 4, col = ((id & 15) ^ (row & 15)) * 8;
        const int b = min(b0 + row, a.B - 1);
        // 16 bytes a lane straight to shared memory, a wavefront's 64 in a row
        __builtin_amdgcn_global_load_lds(
            reinterpret_cast<const __attribute__((address_space(1))) void*>(
                reinterpret_cast<uintptr_t>(a.img[p] + (size_t)b * Kpad + kt * 128 + col)),
            (__attribute__((address_space(3))) void*)(to + (p * QB * 16 + c * 256 + wave * 64) * 8), 16, 0, 0);
      }
  };
  Q4Tile<ST, SG, ZERO> w[2], wn[2];
  auto codes_of = [&](int kt) {
#pragma unroll
    for (int r = 0; r < 2; r++) {
      wn[r].w = reinterpret_cast<const u32x4*>(codes + (row_tile[r] + kt) * 1024)[lane];
      wn[r].sc.load(scales, row_tile[r] + kt, lane);
      wn[r].z.load(zeros, row_tile[r] + kt, lane);
    }
  };

  v4f acc[2][NC];
#pragma unroll
  for (int r = 0; r < 2; r++)
#pragma unroll
    for (int c = 0; c < NC; c++) acc[r][c] = v4f{0.f, 0.f, 0.f, 0.f};

  const Q4Magic magic;
  // one column tile: multiplies what `from` and wn hold while the next tile comes
  // to `to` and wn.  The reads stay in front of the products (the compiler would
  // move them to where their results are used, and wait there).
  auto step = [&](int kt, const _Float16* from, _Float16* to) {
    const int next = min(kt + 1, kend - 1);
#pragma unroll
    for (int r = 0; r < 2; r++) w[r] = wn[r];
    codes_of(next);
    fetch(next, to);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < SG; g++) {
      v4f d[2][NC];
#pragma unroll
      for (int r = 0; r < 2; r++)
#pragma unroll
        for (int c = 0; c < NC; c++) d[r][c] = v4f{0.f, 0.f, 0.f, 0.f};
      Q4Zero zc[2];
#pragma unroll
      for (int r = 0; r < 2; r++) zc[r] = q4_zero(w[r].z.get(g));
#pragma unroll
      for (int s = g * 4 / SG; s < (g + 1) * 4 / SG; s++) {
        h8 bv[P][NC];
#pragma unroll
        for (int p = 0; p < P; p++)
#pragma unroll
          for (int c = 0; c < NC; c++) {
            const int row = 16 * c + (lane & 15);
            bv[p][c] =
                *reinterpret_cast<const h8*>(from + (p * QB * 16 + row * 16 + ((4 * s + (lane >> 4)) ^ (row & 15))) * 8);
          }
#pragma unroll
        for (int r = 0; r < 2; r++) {
          const h8 av = q4_expand(s == 0 ? w[r].w.x : s == 1 ? w[r].w.y : s == 2 ? w[r].w.z : w[r].w.w, zc[r], magic);
#pragma unroll
          for (int p = 0; p < P; p++)
#pragma unroll
            for (int c = 0; c < NC; c++) d[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, bv[p][c], d[r][c], 0, 0, 0);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; r++) {
#pragma unroll
        for (int c = 0; c < NC; c++)
#pragma unroll
          for (int v = 0; v < 4; v++) acc[r][c][v] = fmaf(w[r].sc.get(g, v), d[r][c][v], acc[r][c][v]);
      }
      if (SG > 1) __builtin_amdgcn_sched_barrier(0);  // one group's sums at a time
    }
    wait_vmem();  // this wave's part of the next tile has come
    __syncthreads();
  };
  if (kbeg < kend) {
    codes_of(kbeg);
    fetch(kbeg, lds0);
    wait_vmem();
    __syncthreads();
    for (int kt = kbeg; kt < kend; kt += 2) {
      step(kt, lds0, lds1);
      if (kt + 1 < kend) step(kt + 1, lds1, lds0);
    }
  }

  // a lane's four rows of W lie side by side in y: one store where m lets it
  const int odt = a.S > 1 ? 0 : a.ydt;
  const size_t first = a.S > 1 ? (size_t)split * a.B * a.m : 0;
#pragma unroll
  for (int c = 0; c < NC; c++) {
    const int b = b0 + 16 * c + (lane & 15);
    if (b >= a.B) continue;
    const float f = a.fac[b];
#pragma unroll
    for (int r = 0; r < 2; r++) {
      const int i = i0 + wm + 16 * r + 4 * (lane >> 4);
      const size_t at = first + (size_t)b * a.m + i;
      const v4f v = acc[r][c] * f;
      if (a.quads) {
        if (i >= a.m) continue;
        if (odt == 0) {
          *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.y) + at) = v;
        } else {
          const uint32_t lo = (uint32_t)f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16;
          const uint32_t hi = (uint32_t)f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16;
          *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + at) = uint2{lo, hi};
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
          if (i + k < a.m) q4_store(a.y, odt, at + k, v[k]);
      }
    }
  }
}

// y = the S partial sums, `stride` values apart, added in order.
__global__ void __launch_bounds__(256) q4_join_kernel(const float* __restrict__ part, int S, size_t stride,
                                                      size_t count, void* y, int ydt) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= count) return;
  float s = part[i];
  for (int k = 1; k < S; k++) s += part[k * stride + i];
  q4_store(y, ydt, i, s);
}

// ------------------------------------------------------------------ host
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

constexpr size_t MAX_LDS = 160 * 1024;

// Workgroups of a pack kernel: its threads stride over the words, so that the
// launch stays far below 2^32 threads for every weight.
dim3 q4_pack_grid(long long items) {
  const long long g = (items + 255) / 256;
  return dim3((unsigned)(g < (1 << 20) ? g : (1 << 20)));
}

// Splits and shared memory of the decode kernel for B <= 16 rows of x.
struct Q4DecPlan {
  int W, S, range, tpw, groups, keep;
  bool shared;
  size_t lds, part;  // bytes: shared memory of a workgroup, partial sums
};

Q4DecPlan q4_dec_plan(const int* m, int L, int n, int B, int P) {
  Q4DecPlan p{};
  const int KT = ceil_div(n, 128);
  int RT = 0;
  size_t out = 0;
  for (int l = 0; l < L; l++) {
    RT += ceil_div(m[l], 16);
    out += (size_t)B * m[l];
  }
  const size_t per_tile = (size_t)B * (256 * P + 4);  // of the image of x
  const bool small = per_tile * KT <= 40 * 1024;
  // An image of 64 to 128 KB is turned over whole by every workgroup, or split.  us
  // shared / split, for 7 rows of 4099 fp32, 7 of 8192 and 5 of 11008 bf16:
  //   69 row tiles  11.6 / 10.8  10.7 / 10.9  12.9 / 11.6
  //   127           11.6 / 10.9  10.7 / 11.0  13.1 / 12.9
  //   129           11.6 / 10.9  10.7 / 11.5  13.1 / 13.1
  //   256           11.7 / 13.6  11.8 / 12.6  13.7 / 13.2
  //   512           14.5 / 13.9  14.1 / 14.7  18.5 / 18.9
  // so few row tiles are split and many share; no size of the three is best all along.
  p.shared = per_tile * KT <= (RT < 128 ? 64 : 128) * 1024;
  if (p.shared) {
    // the whole row of x fits: the waves of a workgroup share each row tile, four
    // column tiles a wave where there are as many.  A small image (one row of x, two
    // of 8192) is turned over twice rather than once, and two workgroups of 8 waves
    // a CU do not wait for each other: 8192 x 8192, 11.2 -> 10.2 us, 57344 x 8192
    // 45.3 -> 44 us, two rows 11.5 -> 11.3 us.  Four rows of 8192 gain nothing: 8192
    // rows of W 11.8 us against 12.0 us with two workgroups, 32000 29.7 us either way.
    const int most = small ? 8 : 16, w = ceil_div(KT, 4);
    p.W = w < most ? w : most;
    p.S = 1;
    // 16 waves a CU
    const int fill = 256 * (16 / p.W);
    p.groups = RT < fill ? RT : fill;
  } else {
    // a wave keeps its row tile; the columns are split so that the image fits
    // and the workgroups fill the CUs
    p.W = RT >= 256 ? 16 : 4;
    const int row_groups = ceil_div(RT, p.W);
    p.S = (int)((per_tile * KT + 144 * 1024 - 1) / (144 * 1024));
    while (row_groups * p.S < 256 && ceil_div(KT, p.S) >= 8) p.S++;
    p.groups = row_groups;
  }
  p.range = ceil_div(KT, p.S);
  p.S = ceil_div(KT, p.range);
  p.tpw = p.shared ? ceil_div(p.range, p.W) : p.range;
  if (p.shared) {
    const size_t most = small ? MAX_LDS / 2 : MAX_LDS, row_tile = q4_dec_lds(P, B, 0, p.W, 1).total;
    const int turns = ceil_div(RT, p.groups);
    const int fit = (int)((most - q4_dec_lds(P, B, p.range, p.W, 0).total) / row_tile);  // at least 2
    p.keep = turns < fit ? turns : fit;
  }
  p.lds = q4_dec_lds(P, B, p.range, p.W, p.keep).total;
  p.part = p.S > 1 ? p.S * out * 4 : 0;
  return p;
}

// Codes of 16 MB or more are read as a stream.  One row, us as a stream / not, over
// 1 GiB of weights in turn: 32000 x 8192 (131 MB) 27.6 / 28.4, 8192 x 8192 (34 MB)
// 10.2 / 10.5, 11008 x 4096 (23 MB) 8.55 / 8.42, 4096 x 8192 (17 MB) 7.1 / 7.3, 4096 x
// 4096 (8 MB) 5.9 / 5.8, 2048 x 4096 5.4 / 5.3; with weights that stay in the 256 MB
// cache 4096 x 4096 5.6 / 5.5 and 2048 x 4096 5.3 / 4.9.
bool q4_streams(const Q4DecArgs& k) { return (size_t)k.rows * k.KT * 1024 >= (size_t)16 << 20; }

template <typename XT>
hipError_t dec_forward(const Q4Args& a) {
  const int B = a.B;
  constexpr int P = sizeof(XT) == 4 ? 2 : 1;
  const Q4DecPlan p = q4_dec_plan(a.m, a.L, a.n, B, P);
  Q4DecArgs k{};
  k.n = a.n;
  k.KT = ceil_div(a.n, 128);
  k.B = B;
  k.range = p.range;
  k.tpw = p.tpw;
  k.shared = p.shared;
  k.groups = p.groups;
  k.keep = p.keep;
  while ((1 << k.tw) < p.range && (1 << k.tw) < 4 * p.W) k.tw++;
  k.odt = p.S > 1 ? 0 : a.y_dtype;
  k.x = a.x;
  float* part = reinterpret_cast<float*>(a.ws);
  for (int l = 0; l < a.L; l++) {
    const Q4Layout lay = q4_layout(a.m[l], a.n, a.group, a.scale_dtype == 1 ? 2 : 4, a.zeros);
    Q4DecLayer& c = k.layer[l];
    c.codes = a.blob[l] + lay.off_codes;
    c.scales = a.blob[l] + lay.off_scales;
    c.zeros = a.blob[l] + lay.off_zeros;
    c.out = p.S > 1 ? static_cast<void*>(part + k.part_split) : a.y[l];
    c.m = a.m[l];
    k.rows += ceil_div(a.m[l], 16);
    c.rt_end = k.rows;
    k.part_split += (size_t)B * a.m[l];
  }
  q4_dispatch(a.scale_dtype, a.group, a.zeros, [&](auto st, auto sg, auto zero) {
    using ST = decltype(st);
    constexpr int SG = decltype(sg)::value, bytes = SG * sizeof(ST);
    // tiles in flight (U D): as many as the registers of 16 waves a CU hold beside
    // the operands of a bf16 x (groups of 32 with fp32 scales and zero points: 12
    // bytes a lane spill).  fp32 x has twice the operands, and 14 of its 24 variants
    // spill 8 to 80 bytes a lane.
    constexpr int U = bytes == 2 ? 4 : bytes <= 8 ? 2 : 1, D = bytes == 4 || bytes == 16 ? 3 : 2;
    k.steps = ceil_div(p.tpw, U);
    constexpr bool Z = decltype(zero)::value;
    auto kernel = q4_streams(k) ? q4_dec_kernel<XT, ST, SG, Z, U, D, true> : q4_dec_kernel<XT, ST, SG, Z, U, D, false>;
    hipLaunchKernelGGL(kernel, dim3(p.groups * p.S), dim3(64 * p.W), p.lds, a.stream, k);
    return 0;
  });
  if (p.S > 1)
    for (int l = 0; l < a.L; l++) {
      const size_t count = (size_t)B * a.m[l];
      hipLaunchKernelGGL(q4_join_kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, a.stream,
                         static_cast<const float*>(k.layer[l].out), p.S, k.part_split, count, a.y[l],
                         a.y_dtype);
    }
  return hipGetLastError();
}

}  // namespace

Q4GemmPlan q4_gemm_plan(int m, int n, int B, int x_dtype) {
  Q4GemmPlan p{};
  const int KT = ceil_div(n, 128), P = x_dtype == 0 ? 2 : 1;
  // up to 64 rows one tile of 64 columns: 8192 x 8192, 20 rows 28.5 -> 22.0 us, 64 rows
  // 31.9 -> 25.9 us against tiles of 128
  p.NC = B <= 64 ? 4 : 8;
  const long long tiles = (long long)ceil_div(m, QM) * ceil_div(B, 16 * p.NC);
  // K splits while the tiles leave CUs idle, each of at least four steps: 8192 x 8192,
  // 20 rows 64 -> 22 us, 128 rows 92 -> 38 us.  (The floor of such a batch, one read
  // of the codes, is 5 to 7 us: three launches, a K step's latency and the partial
  // sums' way through memory are in the rest.)
  int S = 1;
  while (tiles * S < 384 && S < 32 && KT / (2 * S) >= 4) S *= 2;
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
  const int P = x_dtype == 0 ? 2 : 1;
  size_t need = 0;
  if (B <= Q4_DEC_MAX) return q4_dec_plan(m, L, n, B, P).part;
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
  k.quads = k.m % 4 == 0 && reinterpret_cast<uintptr_t>(k.y) % 16 == 0;
  if (image) {
    hipLaunchKernelGGL((q4_rows_kernel<XT>), dim3(a.B), dim3(256), 0, a.stream, static_cast<const XT*>(a.x), a.n,
                       k.KT * 128, reinterpret_cast<_Float16*>(a.ws + p.off_hi),
                       reinterpret_cast<_Float16*>(a.ws + p.off_lo), reinterpret_cast<float*>(a.ws + p.off_fac));
  }
  const long long tiles = (long long)ceil_div(k.m, QM) * ceil_div(k.B, 16 * p.NC) * k.S;
  const dim3 grid((unsigned)(8 * ((tiles + 7) / 8)));
  q4_dispatch(a.scale_dtype, a.group, a.zeros, [&](auto st, auto sg, auto zero) {
    using ST = decltype(st);
    auto kernel = p.NC == 4 ? q4_gemm_kernel<ST, decltype(sg)::value, decltype(zero)::value, P, 4>
                            : q4_gemm_kernel<ST, decltype(sg)::value, decltype(zero)::value, P, 8>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, a.stream, k);
    return 0;
  });
  if (p.S > 1) {
    const size_t count = (size_t)a.B * a.m[l];
    hipLaunchKernelGGL(q4_join_kernel, dim3((unsigned)((count + 255) / 256)), dim3(256), 0, a.stream,
                       reinterpret_cast<const float*>(a.ws + p.off_part), p.S, count, count, a.y[l], a.y_dtype);
  }
  return hipGetLastError();
}

hipError_t q4_forward(const Q4Args& a) {
  if (a.B <= Q4_DEC_MAX) return a.x_dtype == 0 ? dec_forward<float>(a) : dec_forward<uint16_t>(a);
  hipError_t e = hipSuccess;
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
                       KT, SG, 4, entries, reinterpret_cast<uint16_t*>(blob + lay.off_scales), bad);
  else
    hipLaunchKernelGGL((q4_pack_groups_kernel<uint32_t>), ge, dim3(256), 0, st, static_cast<const uint32_t*>(s), m, ng,
                       KT, SG, 4, entries, reinterpret_cast<uint32_t*>(blob + lay.off_scales), bad);
  if (z)
    hipLaunchKernelGGL((q4_pack_groups_kernel<uint8_t>), ge, dim3(256), 0, st, z, m, ng, KT, SG, 1, entries,
                       blob + lay.off_zeros, bad);
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
