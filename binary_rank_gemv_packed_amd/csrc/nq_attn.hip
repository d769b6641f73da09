// Attention of one new token a sequence over the paged cache of keys and values:
//
//   y[b, h] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q[b, h] . k_t - max),
//
// t over the sequence's last `window` tokens (all without a window), keys and
// values of head h / (q_heads / heads).  A sequence without tokens gives zeros.
//
// One pass over the cache: a wave holds 16 query heads of one key head as the
// columns of an MFMA 16x16x32 and takes 32 tokens at a time.  The product of keys
// and queries leaves a lane with 2 x 4 tokens of one head, which are, without any
// exchange, its operand of the product of values and weights (the cache's tiles are
// laid out for it).  The running maximum of a head is raised, and the sums are scaled
// down, only where a weight would pass 2^8: until then lanes do not talk to each other.
//
// Arithmetic.  Keys and values enter as bf16: held values, or whole numbers (exact),
// whose scale multiplies the product of keys and queries in fp32 and, for values, the
// weight.  4-bit codes enter as c + 24 (set into the mantissa of 16) and 24 times
// the sum of what they are multiplied with is taken off by the same MFMA.  Scores, maximum, sum and
// output are fp32.  Weights are rounded to bf16 (2^-9 each, and the sum of bf16 values
// is taken over the rounded ones, so that a token that outweighs the others is exact);
// FINE, for fp32 queries or outputs, takes weights and queries as three bf16 pieces,
// exactly, and 4-bit codes as c, for 24 times the sum of the weights would cost some of
// the bits that are asked for.
#include "nq_common.h"
#include "nq_internal.h"

#include <type_traits>

namespace nq {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x3 __attribute__((ext_vector_type(3), aligned(4)));

constexpr int ATTN_WAVES = 4;
constexpr int ATTN_GRID = 512;    // workgroups that share the tokens of all sequences
constexpr int ATTN_PAIR = 32;     // tokens of a wave's step: two tiles
constexpr float ATTN_RISE = 8.0f;  // a maximum is raised by more than this (powers of two)
#define NEG_INF (-__builtin_inff())

__device__ __forceinline__ v4f mfma(u32x4 a, u32x4 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t hi, uint32_t lo) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }
// Two fp32 to bf16, to the nearest.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const bf2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float low_f32(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float high_f32(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }
// Four signed bytes as bf16.
__device__ __forceinline__ u32x2 bytes_bf16(uint32_t w) {
  uint32_t f[4];
#pragma unroll
  for (int i = 0; i < 4; i++) f[i] = __float_as_uint((float)(int8_t)(w >> (8 * i)));
  return u32x2{high_halves(f[1], f[0]), high_halves(f[3], f[2])};
}
// Nibbles p and p + 4 as bf16 of 16 + nibble.
__device__ __forceinline__ uint32_t nibbles_bf16(uint32_t w, int p) {
  return ((p == 0 ? w << 3 : w >> (4 * p - 3)) & 0x00780078u) | 0x41804180u;
}
// Nibbles p and p + 4 as bf16 of nibble - 8.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, int p) {
  const float lo = (float)(w >> (4 * p) & 15u) - 8.0f, hi = (float)(w >> (4 * p + 16) & 15u) - 8.0f;
  return high_halves(__float_as_uint(hi), __float_as_uint(lo));
}
constexpr uint32_t MINUS_24 = 0xc1c0c1c0u;  // two bf16

// ------------------------------------------------------------------ which tokens
struct Span {
  int n, lo;   // tokens lo .. n - 1
  bool bad;    // a length that the table cannot hold
  __device__ __forceinline__ int first_pair() const { return lo / ATTN_PAIR; }
  __device__ __forceinline__ int pairs() const { return n > lo ? (n + ATTN_PAIR - 1) / ATTN_PAIR - first_pair() : 0; }
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
  Span s{a.lengths[b], 0, false};
  s.bad = s.n < 0 || s.n > a.max_length;
  if (s.bad) s.n = 0;
  if (a.window > 0 && s.n > a.window) s.lo = s.n - a.window;
  return s;
}

// Sums over a workgroup of 256 threads: `before` the sum of the threads in front, `total` of all.
__device__ __forceinline__ void block_scan(long long v, long long* before, long long* total, long long* shared) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  long long up = v;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const long long other = __shfl_up(up, o);
    if (lane >= o) up += other;
  }
  if (lane == 63) shared[wave] = up;
  __syncthreads();
  long long b = 0, t = 0;
#pragma unroll
  for (int w = 0; w < 4; w++) {
    if (w < wave) b += shared[w];
    t += shared[w];
  }
  __syncthreads();
  *before = b + up - v;
  *total = t;
}

// Pairs of a workgroup's share of `total`: a multiple of its waves.
__device__ __forceinline__ long long share_of(long long total) {
  const long long even = (total + ATTN_GRID - 1) / ATTN_GRID;
  return (even + ATTN_WAVES - 1) / ATTN_WAVES * ATTN_WAVES;
}

__host__ __device__ inline int head_tiles(int ratio) { return (ratio + 15) / 16; }
__host__ __device__ inline size_t slot_floats(int D) { return 16 * D + 32; }

// ------------------------------------------------------------------ a wave's step
template <int LB>
__device__ __forceinline__ void lane_bytes(const uint8_t* tile, int lane, uint32_t (&w)[LB / 4]) {
#pragma unroll
  for (int p = 0; p < LB / 16; p++) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(tile + p * 1024 + lane * 16);
#pragma unroll
    for (int i = 0; i < 4; i++) w[4 * p + i] = u[i];
  }
  if constexpr (LB % 16 == 8) {
    const u32x2 u = *reinterpret_cast<const u32x2*>(tile + LB / 16 * 1024 + lane * 8);
    w[LB / 4 - 2] = u[0];
    w[LB / 4 - 1] = u[1];
  } else if constexpr (LB % 16 == 12) {
    const u32x3 u = *reinterpret_cast<const u32x3*>(tile + LB / 16 * 1024 + lane * 12);
#pragma unroll
    for (int i = 0; i < 3; i++) w[LB / 4 - 3 + i] = u[i];
  }
}

template <int D, int KIND>
struct Pair {
  static constexpr int LB = kv_lane_bytes(KIND, D), NG = kv_groups(KIND, D), SW = NG ? 4 * NG : 1;
  uint32_t k[2][LB / 4], v[2][LB / 4];
  uint32_t s[2][SW];  // scales of the lane's four slots: keys [NG], values [NG], two words each
  __device__ __forceinline__ void load(int i, const uint8_t* tile, const uint8_t* scales, int lane) {
    lane_bytes<LB>(tile, lane, k[i]);
    lane_bytes<LB>(tile + kv_half_bytes(KIND, D), lane, v[i]);
    if constexpr (NG > 0) {
#pragma unroll
      for (int p = 0; p < NG; p++) {
        const u32x4 u = *reinterpret_cast<const u32x4*>(scales + (lane >> 4) * 16 * NG + 16 * p);
#pragma unroll
        for (int e = 0; e < 4; e++) s[i][4 * p + e] = u[e];
      }
    }
  }
  __device__ __forceinline__ float scale(int i, int value, int group, int j) const {
    const uint32_t w = s[i][(value * NG + group) * 2 + j / 2];
    return j & 1 ? high_f32(w) : low_f32(w);
  }
  // operand of 32 channels of 16 keys
  template <bool FINE>
  __device__ __forceinline__ u32x4 keys(int i, int c) const {
    if constexpr (KIND == KV_BF16) {
      return u32x4{k[i][4 * c], k[i][4 * c + 1], k[i][4 * c + 2], k[i][4 * c + 3]};
    } else if constexpr (KIND == KV_INT8) {
      const u32x2 a = bytes_bf16(k[i][2 * c]), b = bytes_bf16(k[i][2 * c + 1]);
      return u32x4{a[0], a[1], b[0], b[1]};
    } else {
      const uint32_t w = k[i][c];
      if constexpr (FINE) return u32x4{codes_bf16(w, 0), codes_bf16(w, 1), codes_bf16(w, 2), codes_bf16(w, 3)};
      return u32x4{nibbles_bf16(w, 0), nibbles_bf16(w, 1), nibbles_bf16(w, 2), nibbles_bf16(w, 3)};
    }
  }
  // operand of 16 channels of the pair's values
  template <bool FINE>
  __device__ __forceinline__ u32x4 values(int x) const {
    if constexpr (KIND == KV_BF16) {
      return u32x4{v[0][2 * x], v[0][2 * x + 1], v[1][2 * x], v[1][2 * x + 1]};
    } else if constexpr (KIND == KV_INT8) {
      const u32x2 a = bytes_bf16(v[0][x]), b = bytes_bf16(v[1][x]);
      return u32x4{a[0], a[1], b[0], b[1]};
    } else {
      const int h = x & 1;
      const uint32_t a = v[0][x / 2], b = v[1][x / 2];
      if constexpr (FINE) return u32x4{codes_bf16(a, h), codes_bf16(a, 2 + h), codes_bf16(b, h), codes_bf16(b, 2 + h)};
      return u32x4{nibbles_bf16(a, h), nibbles_bf16(a, 2 + h), nibbles_bf16(b, h), nibbles_bf16(b, 2 + h)};
    }
  }
};

template <int D, int KIND, bool FINE>
struct Wave {
  static constexpr int CH = D / 32, XT = D / 16, NG = kv_groups(KIND, D), PIECES = FINE ? 3 : 1;
  u32x4 q[PIECES][CH];
  static constexpr bool BIAS = KIND == KV_INT4 && !FINE;
  v4f less[BIAS ? CH : 1];  // -24 times the sum of the queries' 32 channels
  v4f o[XT];
  float m, safe, l;
  int lane;

  // queries of the lane's head (row null: zeros), eight channels of each 32
  __device__ __forceinline__ void queries(const void* row, int dtype) {
#pragma unroll
    for (int c = 0; c < CH; c++) {
#pragma unroll
      for (int p = 0; p < PIECES; p++) q[p][c] = u32x4{0u, 0u, 0u, 0u};
      if (!row) continue;
      const int at = 32 * c + 8 * (lane >> 4);
      if (dtype == 2) {
        const uint16_t* r = static_cast<const uint16_t*>(row) + at;
#pragma unroll
        for (int i = 0; i < 4; i++) q[0][c][i] = r[2 * i] | (uint32_t)r[2 * i + 1] << 16;
      } else if constexpr (FINE) {  // pieces cut off, not rounded: none passes the largest value
        const float* r = static_cast<const float*>(row) + at;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float a = r[2 * i], b = r[2 * i + 1];
          const bool fine_a = fabsf(a) <= 3.402823466e38f, fine_b = fabsf(b) <= 3.402823466e38f;
#pragma unroll
          for (int p = 0; p < 3; p++) {
            // of an infinity or a NaN only one piece, a quiet one
            const float ha = fine_a ? __uint_as_float(__float_as_uint(a) & 0xffff0000u) : p ? 0.0f : a != a ? __uint_as_float(0x7fc00000u) : a;
            const float hb = fine_b ? __uint_as_float(__float_as_uint(b) & 0xffff0000u) : p ? 0.0f : b != b ? __uint_as_float(0x7fc00000u) : b;
            q[p][c][i] = high_halves(__float_as_uint(hb), __float_as_uint(ha));
            a -= ha;
            b -= hb;
          }
        }
      }
    }
    if constexpr (BIAS) {
      const u32x4 minus = {MINUS_24, MINUS_24, MINUS_24, MINUS_24};
#pragma unroll
      for (int c = 0; c < CH; c++) less[c] = mfma(minus, q[0][c], v4f{0.0f, 0.0f, 0.0f, 0.0f});
    }
  }

  __device__ __forceinline__ void begin() {
    m = NEG_INF;
    safe = l = 0.0f;
#pragma unroll
    for (int x = 0; x < XT; x++) o[x] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // 32 tokens from `first` on; EDGE: some of them are not seen
  template <bool EDGE>
  __device__ __forceinline__ void step(Pair<D, KIND>& t, float c, int first, int lo, int n) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (KIND == KV_INT4) {
#pragma unroll
        for (int ch = 0; ch < CH; ch++) {
          v4f d = {0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (BIAS) d = less[ch];
          const u32x4 key = t.template keys<FINE>(i, ch);
#pragma unroll
          for (int p = PIECES - 1; p >= 0; p--) d = mfma(key, q[p][ch], d);
#pragma unroll
          for (int j = 0; j < 4; j++) s[j] = fmaf(t.scale(i, 0, ch, j), d[j], s[j]);
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < CH; ch++) {
          const u32x4 key = t.template keys<FINE>(i, ch);
#pragma unroll
          for (int p = PIECES - 1; p >= 0; p--) s = mfma(key, q[p][ch], s);
        }
        if constexpr (KIND == KV_INT8) {
#pragma unroll
          for (int j = 0; j < 4; j++) s[j] *= t.scale(i, 0, 0, j);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        x[4 * i + j] = s[j] * c;
        if constexpr (EDGE) {
          const int at = first + 16 * i + 4 * (lane >> 4) + j;
          if (at < lo || at >= n) x[4 * i + j] = NEG_INF;
        }
      }
    }
    if constexpr (EDGE && KIND == KV_BF16) {  // what lies in slots that are not seen may be anything
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const int at = first + 16 * i + 4 * (lane >> 4);
        uint32_t keep[2];
#pragma unroll
        for (int w = 0; w < 2; w++) {
          keep[w] = (at + 2 * w >= lo && at + 2 * w < n ? 0xffffu : 0u) |
                    (at + 2 * w + 1 >= lo && at + 2 * w + 1 < n ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int w = 0; w < D / 8; w++) t.v[i][w] &= keep[w & 1];
      }
    }
    float top = NEG_INF;
#pragma unroll
    for (int j = 0; j < 8; j++) top = fmaxf(top, x[j]);
    if (__any(top > m + ATTN_RISE)) raise(top);
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; j++) p[j] = __builtin_amdgcn_exp2f(x[j] - safe);
    if constexpr (NG == 0) {
      u32x4 w[PIECES];
      weights(p, w);
#pragma unroll
      for (int j = 0; j < 4; j++) l += FINE ? p[2 * j] + p[2 * j + 1] : low_f32(w[0][j]) + high_f32(w[0][j]);
#pragma unroll
      for (int xt = 0; xt < XT; xt++) {
        const u32x4 value = t.template values<FINE>(xt);
#pragma unroll
        for (int i = PIECES - 1; i >= 0; i--) o[xt] = mfma(value, w[i], o[xt]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) l += p[j];
#pragma unroll
      for (int g = 0; g < NG; g++) {
        float ps[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
          ps[j] = p[j] * t.scale(j / 4, 1, g, j & 3);
          if constexpr (EDGE) ps[j] = x[j] == NEG_INF ? 0.0f : ps[j];
        }
        u32x4 w[PIECES];
        weights(ps, w);
#pragma unroll
        for (int xt = g * XT / NG; xt < (g + 1) * XT / NG; xt++) {
          const u32x4 value = t.template values<FINE>(xt);
#pragma unroll
          for (int i = PIECES - 1; i >= 0; i--) o[xt] = mfma(value, w[i], o[xt]);
          if constexpr (BIAS) {
            const u32x4 minus = {MINUS_24, MINUS_24, MINUS_24, MINUS_24};
            o[xt] = mfma(minus, w[0], o[xt]);
          }
        }
      }
    }
  }

  // weights as bf16, or as pieces that add up to them
  __device__ __forceinline__ static void weights(const float (&p)[8], u32x4 (&w)[PIECES]) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      float lo = p[2 * j], hi = p[2 * j + 1];
#pragma unroll
      for (int i = 0; i < PIECES; i++) {
        w[i][j] = pack_bf16(lo, hi);
        lo -= low_f32(w[i][j]);
        hi -= high_f32(w[i][j]);
      }
    }
  }

  __device__ __forceinline__ void raise(float top) {
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float to = fmaxf(m, top);
    const float f = to == m ? 1.0f : __builtin_amdgcn_exp2f(m - to);
    m = to;
    safe = to == NEG_INF ? 0.0f : to;
    l *= f;
#pragma unroll
    for (int x = 0; x < XT; x++) o[x] *= f;
  }
};

// ------------------------------------------------------------------ kernel
// SPLIT: the pairs of all (sequence, key head, 16 query heads) units, one after the
// other, are cut into equal shares, one a workgroup, whose waves take a unit's pairs in turn.
// A unit that lies within a share is finished there; else its parts go to the
// workgroup's two places (place 1: the part that begins a unit, place 0: one that does
// not) and attn_join_kernel adds them in order.  Without SPLIT a workgroup is a unit.
template <int D, int KIND, bool FINE, bool SPLIT>
__global__ void __launch_bounds__(64 * ATTN_WAVES) attn_kernel(AttnArgs a) {
  constexpr int XT = D / 16;
  __shared__ float part_o[ATTN_WAVES - 1][XT][64][4];
  __shared__ float part_m[ATTN_WAVES][16], part_l[ATTN_WAVES][16];
  __shared__ long long shared[4];
  __shared__ int found[2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15;
  const int heads = a.cache.heads, ratio = a.q_heads / heads, tiles = head_tiles(ratio), units = heads * tiles;
  const float c = a.scale * 1.44269504088896341f;
  int b, unit;
  long long from, left;  // the first pair within the unit; pairs of this workgroup's share
  if constexpr (SPLIT) {
    const int each = (a.B + 255) / 256, b0 = threadIdx.x * each, b1 = b0 + each < a.B ? b0 + each : a.B;
    long long mine = 0, before, total;
    for (int i = b0; i < b1; i++) mine += span_of(a, i).pairs();
    block_scan(mine, &before, &total, shared);
    total *= units;
    before *= units;
    const long long share = share_of(total), start = share * blockIdx.x;
    if (start >= total) return;
    left = total - start < share ? total - start : share;
    if (start >= before && start < before + mine * units) {
      long long at = before;
      int i = b0;
      for (;; i++) {
        const long long its = (long long)span_of(a, i).pairs() * units;
        if (start < at + its) break;
        at += its;
      }
      found[0] = i;
      shared[0] = start - at;
    }
    __syncthreads();
    b = found[0];
    from = shared[0];
    const int pairs = span_of(a, b).pairs();
    unit = (int)(from / pairs);
    from -= (long long)unit * pairs;
  } else {
    b = blockIdx.x / units;
    unit = blockIdx.x % units;
    from = 0;
    left = span_of(a, b).pairs();
  }
  b = __builtin_amdgcn_readfirstlane(b);
  unit = __builtin_amdgcn_readfirstlane(unit);
  const int tpp = a.cache.page / KV_TILE;
  Wave<D, KIND, FINE> w;
  w.lane = lane;
  while (true) {
    const Span sp = span_of(a, b);
    const int pairs = sp.pairs(), p0 = (int)from, p1 = left < pairs - p0 ? p0 + (int)left : pairs;
    if (SPLIT && pairs == 0) {  // no unit of this sequence
      if (++b >= a.B) return;
      unit = 0;
      continue;
    }
    const int head = unit / tiles, q0 = head * ratio + unit % tiles * 16;
    const int cols = ratio - unit % tiles * 16 < 16 ? ratio - unit % tiles * 16 : 16;
    const size_t q_row = ((size_t)b * a.q_heads + q0 + col) * D;
    w.queries(col < cols ? static_cast<const uint8_t*>(a.q) + q_row * (a.q_dtype == 2 ? 2 : 4) : nullptr, a.q_dtype);
    w.begin();
    const uint8_t* tiles_at = a.data + a.cache.tile(head, 0);
    const uint8_t* scales_at = a.data + a.cache.scales(head, 0);
    bool bad = false;
    int page[2], tile[2];  // of the pair that this lane looks after
    // the wave's k-th pair: its tiles' places are looked up for 64 pairs at once, a lane each
    auto look = [&](int k) {
      const int pair = p0 + wave + (k + lane) * ATTN_WAVES;
#pragma unroll
      for (int i = 0; i < 2; i++) {
        page[i] = tile[i] = 0;
        if (pair < p1) {
          int t = (sp.first_pair() + pair) * 2 + i;
          // a tile without tokens that are seen may have no page: the pair's other one once more
          if (t * KV_TILE >= sp.n) t--;
          else if ((t + 1) * KV_TILE <= sp.lo) t++;
          const int p = t / tpp;
          tile[i] = t - p * tpp;
          page[i] = a.table[(size_t)b * a.table_width + p];
          if (page[i] < 0 || page[i] >= a.cache.pages) {
            bad = true;
            page[i] = 0;
          }
        }
      }
    };
    auto load = [&](Pair<D, KIND>& t, int k) {
      if ((k & 63) == 0) look(k);
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const size_t at = (size_t)__builtin_amdgcn_readlane(page[i], k & 63) * a.cache.page_bytes;
        const int in = __builtin_amdgcn_readlane(tile[i], k & 63);
        t.load(i, tiles_at + at + (size_t)in * 2 * kv_half_bytes(KIND, D), scales_at + at + (size_t)in * kv_scale_bytes(KIND, D), lane);
      }
    };
    auto take = [&](Pair<D, KIND>& t, int k) {
      const int first = (sp.first_pair() + p0 + wave + k * ATTN_WAVES) * ATTN_PAIR;
      if (first >= sp.lo && first + ATTN_PAIR <= sp.n) w.template step<false>(t, c, first, sp.lo, sp.n);
      else w.template step<true>(t, c, first, sp.lo, sp.n);
    };
    const int count = p1 - p0 > wave ? (p1 - p0 - wave + ATTN_WAVES - 1) / ATTN_WAVES : 0;
    Pair<D, KIND> t;
    for (int k = 0; k < count; k++) {
      load(t, k);
      take(t, k);
    }
    w.l += __shfl_xor(w.l, 16);
    w.l += __shfl_xor(w.l, 32);
    if (__any(bad) || sp.bad) w.l = __uint_as_float(0x7fc00000u);
    // the waves' sums to wave 0, in order
    if (lane < 16) {
      part_m[wave][lane] = w.m;
      part_l[wave][lane] = w.l;
    }
    if (wave) {
#pragma unroll
      for (int x = 0; x < XT; x++) *reinterpret_cast<v4f*>(part_o[wave - 1][x][lane]) = w.o[x];
    }
    __syncthreads();
    if (wave == 0) {
      float m = w.m, f[ATTN_WAVES], l = 0.0f;
#pragma unroll
      for (int i = 1; i < ATTN_WAVES; i++) m = fmaxf(m, part_m[i][col]);
#pragma unroll
      for (int i = 0; i < ATTN_WAVES; i++) {
        f[i] = part_m[i][col] == m ? 1.0f : __builtin_amdgcn_exp2f(part_m[i][col] - m);
        l += f[i] * part_l[i][col];
      }
      const bool whole = p0 == 0 && p1 == pairs;
      const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
      float* place = a.part + ((size_t)blockIdx.x * 2 + (p0 == 0)) * slot_floats(D);
#pragma unroll
      for (int x = 0; x < XT; x++) {
        v4f s = w.o[x] * f[0];
#pragma unroll
        for (int i = 1; i < ATTN_WAVES; i++) s += *reinterpret_cast<const v4f*>(part_o[i - 1][x][lane]) * f[i];
        s *= inv;
        if (col < cols) {
          const int ch = 16 * x + 4 * (lane >> 4);
          if (!whole) *reinterpret_cast<v4f*>(place + col * D + ch) = s;
          else if (a.y_dtype == 0) *reinterpret_cast<v4f*>(static_cast<float*>(a.y) + q_row + ch) = s;
          else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + q_row + ch) = u32x2{pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
        }
      }
      if (!whole && lane < 16) {
        place[16 * D + lane] = m;
        place[16 * D + 16 + lane] = l;
      }
    }
    left -= p1 - p0;
    if (!SPLIT || left <= 0) return;
    __syncthreads();
    from = 0;
    if (++unit == units) {
      unit = 0;
      if (++b >= a.B) return;
    }
  }
}

// Joins the parts of a unit that was cut: one query head a workgroup.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnArgs a) {
  __shared__ long long shared[4];
  const int heads = a.cache.heads, ratio = a.q_heads / heads, tiles = head_tiles(ratio), units = heads * tiles;
  const int b = blockIdx.y, qh = blockIdx.x, unit = qh / ratio * tiles + qh % ratio / 16, col = qh % ratio % 16;
  long long in_front = 0, all = 0, unused;
  for (int i = threadIdx.x; i < a.B; i += 256) {
    const int p = span_of(a, i).pairs();
    all += p;
    if (i < b) in_front += p;
  }
  long long total, front;
  block_scan(all, &unused, &total, shared);
  block_scan(in_front, &unused, &front, shared);
  const Span sp = span_of(a, b);
  const int pairs = sp.pairs(), d = threadIdx.x;
  const size_t at = ((size_t)b * a.q_heads + qh) * D + d;
  float y = sp.bad ? __uint_as_float(0x7fc00000u) : 0.0f;
  if (pairs) {
    const long long share = share_of(total * units), start = front * units + (long long)unit * pairs;
    const int w0 = (int)(start / share), w1 = (int)((start + pairs - 1) / share);
    if (w0 == w1) return;
    if (d >= D) return;
    auto place = [&](int w) { return a.part + ((size_t)w * 2 + (w == w0)) * slot_floats(D); };
    float m = NEG_INF, l = 0.0f;
    for (int w = w0; w <= w1; w++) m = fmaxf(m, place(w)[16 * D + col]);
    for (int w = w0; w <= w1; w++) {
      const float* p = place(w);
      const float pm = p[16 * D + col], f = pm == m ? 1.0f : __builtin_amdgcn_exp2f(pm - m);
      l += f * p[16 * D + 16 + col];
      y += f * p[col * D + d];
    }
    y = l == 0.0f ? 0.0f : y / l;
  }
  if (d >= D) return;
  if (a.y_dtype == 0) static_cast<float*>(a.y)[at] = y;
  else static_cast<uint16_t*>(a.y)[at] = f32_to_bf16(y);
}

// ------------------------------------------------------------------ host
template <int D, int KIND, bool FINE>
void attn_launch(const AttnArgs& a) {
  const int heads = a.cache.heads, units = heads * head_tiles(a.q_heads / heads);
  if (a.max_length <= 512) {
    hipLaunchKernelGGL((attn_kernel<D, KIND, FINE, false>), dim3((unsigned)(a.B * units)), dim3(64 * ATTN_WAVES), 0, a.stream, a);
    return;
  }
  hipLaunchKernelGGL((attn_kernel<D, KIND, FINE, true>), dim3(ATTN_GRID), dim3(64 * ATTN_WAVES), 0, a.stream, a);
  hipLaunchKernelGGL((attn_join_kernel<D>), dim3(a.q_heads, a.B), dim3(256), 0, a.stream, a);
}

template <int D>
void attn_by_kind(const AttnArgs& a) {
  const bool fine = a.q_dtype == 0 || a.y_dtype == 0;
  if (a.cache.kind == KV_BF16) fine ? attn_launch<D, KV_BF16, true>(a) : attn_launch<D, KV_BF16, false>(a);
  else if (a.cache.kind == KV_INT8) fine ? attn_launch<D, KV_INT8, true>(a) : attn_launch<D, KV_INT8, false>(a);
  else fine ? attn_launch<D, KV_INT4, true>(a) : attn_launch<D, KV_INT4, false>(a);
}

}  // namespace

size_t attn_workspace(const KvLayout& l) { return align_up(ATTN_GRID * 2 * slot_floats(l.D) * 4, 256); }

hipError_t attn_forward(const AttnArgs& a) {
  switch (a.cache.D) {
    case 64: attn_by_kind<64>(a); break;
    case 96: attn_by_kind<96>(a); break;
    case 128: attn_by_kind<128>(a); break;
    case 192: attn_by_kind<192>(a); break;
    default: attn_by_kind<256>(a);
  }
  return hipGetLastError();
}

}  // namespace nq
