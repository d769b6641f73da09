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
// down, only where a score is more than 8 (a factor of 2^8) above it: until then lanes do not talk to
// each other.  Weights are 2^-8 at that maximum, so that none passes 1 and the sums are finite
// wherever n |v| is.
//
// Arithmetic.  Keys and values enter as bf16: held values, or whole numbers (exact),
// whose scale multiplies the product of keys and queries in fp32 and, for values, the
// weight.  4-bit codes enter as c + 24 or c + 136 (set into the mantissa of 16 or 128) and as
// many times the sum of what they are multiplied with is taken off by another MFMA: both products
// are rounded at the size of 144 s sum |q| (values: 144 s times the weights), an instruction's few
// roundings of 2^-24 of that, which is 21 times what a group's largest code makes of it and so some
// 2^-18 of such a score or value, whatever the result is, where a weight's rounding is 2^-8 of its
// value.  Scores, maximum, sum and output are fp32.  Weights (with codes times their scale) enter as two
// bf16 pieces, off by 2^-16, so that a bf16 output is off by its own rounding: with one, 2^-8 each,
// the error of 131072 tokens was 2.2e-3 where the output's rounding is 1.7e-3 (8 bits 55.1 -> 55.6 us; 64 x
// 4096 of 4 key heads of 64 35.8 -> 38.1, of 96 and more within 2 %, bf16 within 1 %, heads of 256 59.4 ->
// 61.3).  For 4 bits one piece, which is far below their own step: two cost them a tenth (131072 tokens 42.3
// -> 46.0 us, 64 x 4096 75 -> 83).  FINE, for fp32 queries or outputs, takes weights and queries as three
// bf16 pieces, exactly, and 4-bit codes as c / 16, for many times the sum of the weights would
// cost some of the bits that are asked for.
//
// Bound by memory where sequences are long: 32 of up to 16384 tokens (675 MB of bf16) 111
// us with the join, 6.1 TB/s, where a large copy moves 5.2 and reads alone 6.9; 131072 tokens
// of 8 bits 55 us, of which the join and its launch are 7 and the way to the first keys
// (lengths, places, tiles, one access behind the other) 4; of 4 bits 43 us, where vector
// instructions take half of the cycles and a wave still waits for two fifths of its own.  Heads of
// 256 with FINE keep one workgroup a CU (shared memory).
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
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));

constexpr int ATTN_WAVES = 4;
// Workgroups that share the tokens of all sequences: as many as a chip of 256 CUs holds at
// once.  Three a CU where registers allow it and vector and matrix instructions are much of the time,
// which it overlaps: codes of 64 channels (64 x 4096 tokens, 4 key heads, 8 bits 36.6 -> 33.3 us, 4 bits 31.7 ->
// 29.8, with fp32 40.1 -> 38.1) and 4 bits for up to eight query heads a key head (131072 tokens of 8 x
// 128 46.6 -> 43.6; 64 x 4096 of 4 x 96 with fp32 50.8 -> 48.4).  Two elsewhere: heads of 128 with 8 bits
// 54.9 us, 57.7 with three, bf16 96.7 and 100.0, of 96 with 8 bits 43.4 and 43.3.  One for FINE heads of 256,
// whose shared memory and registers fill a CU (8 x 4096 tokens of 8 bits 33.3 -> 24.6 us, of bf16 35.7 -> 32.0).
constexpr int attn_grid(int D, int kind, bool fine, bool narrow) {
  if (fine && D == 256) return 256;
  if (kind != KV_BF16 && D == 64) return 768;
  return kind == KV_INT4 && narrow && D <= (fine ? 96 : 128) ? 768 : 512;
}
// Whether more than 16 query heads a key head go 32 at a time, so that the cache is read once for
// them: 64 sequences of 4096 tokens, 32 heads of one key head, bf16 55.0 -> 40.0 us, 8 bits 38.4 ->
// 32.3 (at that step).  Not 4 bits, which wait for their vector instructions (35.8 and 35.3), nor FINE or more
// channels, which have no registers or shared memory for it.
constexpr bool attn_two(int D, int kind, bool fine) { return D <= 128 && kind != KV_INT4 && !fine; }
constexpr int ATTN_PAIR = 32;     // tokens of a wave's step: two tiles
// ATTN_TURN (nq_internal.h) is what a unit costs beside its pairs (its queries, places and the waves'
// join), in pairs: 64 sequences of 256 to 4096 tokens of 8 bits 57.0 us counted as 0, 49.8 as 4, 46.9 as
// 8, 47.5 as 12.
// A maximum is raised by more than this (powers of two), and weights are this far below 1 at it, to which a
// power of two keeps them exact.  The subtraction beside the maximum's is 8 of some 330 vector
// instructions a step: 131072 tokens of 8 bits 55.5 us with and without it, of 4 bits 42.4 and 41.9; a
// rise of 2 or 1 without it 42.8 and 43.2 of 4 bits, 64 x 4096 75.6 and 76.3 (74.6 and 73.4).
constexpr float ATTN_RISE = 8.0f;
#define NEG_INF (-__builtin_inff())

__device__ __forceinline__ v4f mfma(u32x4 a, u32x4 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t hi, uint32_t lo) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }
__device__ __forceinline__ float low_f32(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float high_f32(uint32_t pair) { return __uint_as_float(pair & 0xffff0000u); }
// Four signed bytes as bf16.
__device__ __forceinline__ u32x2 bytes_bf16(uint32_t w) {
  uint32_t f[4];
#pragma unroll
  for (int i = 0; i < 4; i++) f[i] = __float_as_uint((float)(int8_t)(w >> (8 * i)));
  return u32x2{high_halves(f[1], f[0]), high_halves(f[3], f[2])};
}
// Nibbles p and p + 4 as bf16 of 16 + nibble, in two instructions, or of 128 + nibble, where
// nibble 0 needs no shift (131072 tokens 44.8 -> 43.4 us, 64 x 4096 73.9 -> 72.2): the masks lie in scalar and 16 and 128 in vector registers,
// which is what the combined and-or takes (left to itself the compiler makes two of it, with
// constants in the instruction).
struct Nibbles {
  uint32_t mask, sixteen, low, high;
  __device__ __forceinline__ Nibbles() {
    asm volatile("s_mov_b32 %0, 0x00780078" : "=s"(mask));
    asm volatile("s_mov_b32 %0, 0x000f000f" : "=s"(low));
    asm volatile("v_mov_b32 %0, 0x41804180" : "=v"(sixteen));
    asm volatile("v_mov_b32 %0, 0x43004300" : "=v"(high));
  }
  __device__ __forceinline__ uint32_t from16(uint32_t w, int p) const { return (w >> (4 * p - 3) & mask) | sixteen; }
  __device__ __forceinline__ uint32_t from128(uint32_t w, int p) const { return (w >> (4 * p) & low) | high; }
};
// What is taken off again of an operand's four words: 128 + 8 and 16 + 8.
__device__ __forceinline__ u32x4 code_bias() { return u32x4{0xc308c308u, 0xc1c0c1c0u, 0xc308c308u, 0xc1c0c1c0u}; }
// Nibbles p and p + 4 as bf16 of (nibble - 8) / 16: the conversion takes four bits as a signed
// number and, where they lie at the bottom of a byte, needs no shift before it (1.75
// instructions a code; with a shift, a mask, a conversion and a subtraction 3.1).
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, int p) {
  const uint32_t s = (p & 1 ? w >> 4 : w) ^ 0x88888888u;
  const float lo = __builtin_amdgcn_cvt_off_f32_i4((int)(s >> (p & 2 ? 8 : 0) & 255u));
  const float hi = __builtin_amdgcn_cvt_off_f32_i4((int)(s >> (p & 2 ? 24 : 16) & 255u));
  return high_halves(__float_as_uint(hi), __float_as_uint(lo));
}

// ------------------------------------------------------------------ which tokens
// Pairs (of tiles, 32 tokens) of a sequence of n tokens that are seen: from first_pair()
// on, the first with tokens from `lo` on.
struct Span {
  int n, lo;
  __device__ __forceinline__ int first_pair() const { return lo / ATTN_PAIR; }
  __device__ __forceinline__ int pairs() const { return n > lo ? (n + ATTN_PAIR - 1) / ATTN_PAIR - first_pair() : 0; }
  __device__ __forceinline__ int cost() const { return n > lo ? pairs() + ATTN_TURN : 0; }
};
__device__ __forceinline__ bool bad_length(const AttnArgs& a, int n) { return n < 0 || n > a.max_length; }
__device__ __forceinline__ Span span_of(const AttnArgs& a, int n) {  // of a length; a bad one has no tokens
  if (bad_length(a, n)) n = 0;
  return Span{n, a.window > 0 && n > a.window ? n - a.window : 0};
}

// The lengths of 64 sequences from `base` on, one a lane, so that going from one
// sequence to the next costs no memory access.
struct Lengths {
  int base, held;
  __device__ __forceinline__ void load(const AttnArgs& a, int from) {
    const int i = from + (threadIdx.x & 63);
    base = from;
    held = i < a.B ? a.lengths[i] : 0;
  }
  __device__ __forceinline__ Span span(const AttnArgs& a, int b) {
    if (b - base >= 64) load(a, b);
    return span_of(a, __builtin_amdgcn_readlane(held, b - base));
  }
};

// Sum over the lanes up to each one, in the vector unit (with shuffles, and divisions of 64 bits in
// place of quotient(), 4096 tokens take 13.3 us, not 13.0).
__device__ __forceinline__ int sum_up(int v) {
#define NQ_DPP_ADD(ctrl, rows) v += __builtin_amdgcn_update_dpp(0, v, ctrl, rows, 0xf, false)
  NQ_DPP_ADD(0x111, 0xf);  // from 1, 2, 4 and 8 lanes before in a row of 16
  NQ_DPP_ADD(0x112, 0xf);
  NQ_DPP_ADD(0x114, 0xf);
  NQ_DPP_ADD(0x118, 0xf);
  NQ_DPP_ADD(0x142, 0xa);  // the row before's last lane
  NQ_DPP_ADD(0x143, 0xc);  // the first half's last lane
#undef NQ_DPP_ADD
  return v;
}

// a / b for 0 <= a and 0 < b; mostly both are small, and then it is a quarter of the instructions.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// What the units of all sequences cost, each its pairs and ATTN_TURN in front of them
// (nothing without pairs), a wave at a time (every wave for itself): lane L has the sum over one unit of
// each of its ceil(B / 64) sequences, and the sum over the lanes in front.
struct Counts {
  int each, mine, before, total;
  __device__ __forceinline__ Counts(const AttnArgs& a, Lengths& n) {
    const int lane = threadIdx.x & 63;
    each = (a.B + 63) / 64;
    n.load(a, 0);
    mine = span_of(a, n.held).cost();
    if (each > 1) {
      mine = 0;
      for (int i = lane * each; i < (lane + 1) * each && i < a.B; i++) mine += span_of(a, a.lengths[i]).cost();
    }
    const int up = sum_up(mine);
    before = up - mine;
    total = __builtin_amdgcn_readlane(up, 63);
  }
};

// A workgroup's share of `total`: at least a pair a wave.
__device__ __forceinline__ long long share_of(long long total, int grid) {  // 256, 512 or 768: no division
  const long long t = total + grid - 1, even = grid == 768 ? t / 768 : grid == 512 ? t / 512 : t / 256;
  return even < ATTN_WAVES ? ATTN_WAVES : even;
}

// The unit, and how far into its cost, that lies `start` into what all units cost: the units of
// sequence b one after the other, b's behind those of all before it.
struct Begin {
  Span sp;
  int b, unit, from;
  // false: nothing there, which is not so while the lengths stay as they were counted
  __device__ __forceinline__ bool find(const AttnArgs& a, const Counts& n, Lengths& lengths, int units, long long start) {
    const bool here = start >= (long long)n.before * units && start < ((long long)n.before + n.mine) * units;
    const int owner = __builtin_ctzll(__ballot(here));
    b = owner * n.each;
    long long rest = start - (long long)__builtin_amdgcn_readlane(n.before, owner) * units;
    if (n.each > 1) lengths.load(a, b);
    sp = lengths.span(a, b);
    while (rest >= (long long)sp.cost() * units) {
      rest -= (long long)sp.cost() * units;
      if (++b >= a.B) return false;
      sp = lengths.span(a, b);
    }
    unit = (int)quotient(rest, sp.cost());
    from = (int)(rest - (long long)unit * sp.cost());
    return true;
  }
};

// Units of a key head's query heads, `cols` (16 or 32) each, and a part of one in the
// workspace: sums [cols][D], maxima [cols], weights' sums [cols].
__host__ __device__ inline int head_tiles(int ratio, int cols) { return (ratio + cols - 1) / cols; }
__host__ __device__ inline size_t slot_floats(int D, int cols) { return (size_t)cols * (D + 2); }

// ------------------------------------------------------------------ a wave's step
// Codes are read once, past the caches: 131072 tokens of 8 bits 61.0 -> 55.5 us, of bf16
// 112 -> 99 us.
template <int LB>
__device__ __forceinline__ void lane_bytes(const uint8_t* tile, int lane, uint32_t (&w)[LB / 4]) {
#pragma unroll
  for (int p = 0; p < LB / 16; p++) {
    const u32x4 u = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(tile + p * 1024 + lane * 16));
#pragma unroll
    for (int i = 0; i < 4; i++) w[4 * p + i] = u[i];
  }
  if constexpr (LB % 16 == 8) {
    const u32x2 u = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(tile + LB / 16 * 1024 + lane * 8));
    w[LB / 4 - 2] = u[0];
    w[LB / 4 - 1] = u[1];
  } else if constexpr (LB % 16 == 12) {
    const u32x3 u = __builtin_nontemporal_load(reinterpret_cast<const u32x3*>(tile + LB / 16 * 1024 + lane * 12));
#pragma unroll
    for (int i = 0; i < 3; i++) w[LB / 4 - 3 + i] = u[i];
  }
}

// Where the two tiles of a pair lie (the same for the wave).
struct Where {
  const uint8_t* tile[2];
  const uint8_t* scales[2];
};

// A pair's keys or values, and the scales of the lane's four slots of either tile,
// NG groups, two words each.
// NARROW (up to eight query heads a key head): columns 8 .. 15 of the MFMA hold no head, and
// the lanes there take over the second tile's scores of head L & 7; a lane then needs the
// scales of one tile.
template <int D, int KIND, bool VALUE, bool NARROW>
struct Half {
  static constexpr int LB = kv_lane_bytes(KIND, D), NG = kv_groups(KIND, D), TILES = NARROW ? 1 : 2;
  uint32_t w[2][LB / 4], s[TILES][NG ? 2 * NG : 1];
  // lane: where no pair is left every lane reads lane 0's part, a line of each piece
  __device__ __forceinline__ void load(const Where& at, int lane) {
#pragma unroll
    for (int i = 0; i < 2; i++) lane_bytes<LB>(at.tile[i] + (VALUE ? kv_half_bytes(KIND, D) : 0), lane, w[i]);
#pragma unroll
    for (int i = 0; i < TILES; i++) {
      const uint8_t* q = (NARROW ? lane & 8 ? at.scales[1] : at.scales[0] : at.scales[i]) + (lane >> 4) * 16 * NG + (VALUE ? 8 * NG : 0);
#pragma unroll
      for (int p = 0; p < NG / 2; p++) {
        const u32x4 u = *reinterpret_cast<const u32x4_at4*>(q + 16 * p);
#pragma unroll
        for (int e = 0; e < 4; e++) s[i][4 * p + e] = u[e];
      }
      if constexpr (NG % 2) {
        const u32x2 u = *reinterpret_cast<const u32x2*>(q + 8 * (NG - 1));
        s[i][2 * NG - 2] = u[0];
        s[i][2 * NG - 1] = u[1];
      }
    }
  }
  __device__ __forceinline__ float scale(int i, int group, int j) const {
    const uint32_t u = s[i][group * 2 + j / 2];
    return j & 1 ? high_f32(u) : low_f32(u);
  }
  // keys: operand of 32 channels of 16 slots
  template <bool FINE>
  __device__ __forceinline__ u32x4 keys(int i, int c, const Nibbles& nb) const {
    if constexpr (KIND == KV_BF16) {
      return u32x4{w[i][4 * c], w[i][4 * c + 1], w[i][4 * c + 2], w[i][4 * c + 3]};
    } else if constexpr (KIND == KV_INT8) {
      const u32x2 a = bytes_bf16(w[i][2 * c]), b = bytes_bf16(w[i][2 * c + 1]);
      return u32x4{a[0], a[1], b[0], b[1]};
    } else {
      const uint32_t u = w[i][c];
      if constexpr (FINE) return u32x4{codes_bf16(u, 0), codes_bf16(u, 1), codes_bf16(u, 2), codes_bf16(u, 3)};
      return u32x4{nb.from128(u, 0), nb.from16(u, 1), nb.from128(u, 2), nb.from16(u, 3)};
    }
  }
  // values: operand of 16 channels of the pair; keep: the bits of bf16 values that are seen
  template <bool FINE>
  __device__ __forceinline__ u32x4 values(int x, const uint32_t (&keep)[4], const Nibbles& nb) const {
    if constexpr (KIND == KV_BF16) {
      return u32x4{w[0][2 * x] & keep[0], w[0][2 * x + 1] & keep[1], w[1][2 * x] & keep[2], w[1][2 * x + 1] & keep[3]};
    } else if constexpr (KIND == KV_INT8) {
      const u32x2 a = bytes_bf16(w[0][x]), b = bytes_bf16(w[1][x]);
      return u32x4{a[0], a[1], b[0], b[1]};
    } else {
      const int h = x & 1;
      const uint32_t a = w[0][x / 2], b = w[1][x / 2];
      if constexpr (FINE) return u32x4{codes_bf16(a, h), codes_bf16(a, 2 + h), codes_bf16(b, h), codes_bf16(b, 2 + h)};
      return u32x4{nb.from128(a, h), nb.from16(a, 2 + h), nb.from128(b, h), nb.from16(b, 2 + h)};
    }
  }
};

// Queries as the operand of the MFMA, in shared memory: [piece][16 heads][32 channels][64 lanes],
// lane L channels 8 (L >> 4) .. + 7 of head L & 15.  FINE: three pieces.
constexpr int query_pieces(bool fine) { return fine ? 3 : 1; }

// A wave's share of them: channels 32 c .. of 16 heads for c = wave, wave + WAVES (and, with HT =
// 2, of the next 16 for c behind D / 32).
template <int D, bool FINE, int WAVES, int HT>
struct Queries {
  static constexpr int CH = D / 32, ALL = HT * CH, EACH = (ALL + WAVES - 1) / WAVES, PIECES = query_pieces(FINE);
  u32x4_at2 raw[EACH][FINE ? 2 : 1];
  // row: the lane's head of the first 16, null for none; next: whether it has one of the next 16
  __device__ __forceinline__ void load(const void* row, bool next, int dtype, int wave, int lane) {
#pragma unroll
    for (int j = 0; j < EACH; j++) {
      const int c = wave + WAVES * j, h = HT == 1 ? 0 : c / CH;
      const int at = 32 * (HT == 1 ? c : c % CH) + 8 * (lane >> 4) + h * 16 * D;
#pragma unroll
      for (int i = 0; i < (FINE ? 2 : 1); i++) raw[j][i] = u32x4_at2{0u, 0u, 0u, 0u};
      if (!row || c >= ALL || (h && !next)) continue;
      if (FINE && dtype == 0) {
#pragma unroll
        for (int i = 0; i < (FINE ? 2 : 1); i++) raw[j][i] = reinterpret_cast<const u32x4_at2*>(static_cast<const float*>(row) + at)[i];
      } else {
        raw[j][0] = *reinterpret_cast<const u32x4_at2*>(static_cast<const uint16_t*>(row) + at);
      }
    }
  }
  __device__ __forceinline__ void put(uint32_t (*to)[64][4], int dtype, int wave, int lane) const {
#pragma unroll
    for (int j = 0; j < EACH; j++) {
      const int c = wave + WAVES * j;
      if (c >= ALL) continue;
      u32x4 out[PIECES];
#pragma unroll
      for (int p = 0; p < PIECES; p++) out[p] = u32x4{0u, 0u, 0u, 0u};
      if (FINE && dtype == 0) {  // pieces cut off, not rounded: none passes the largest value
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float v[2] = {__uint_as_float(raw[j][FINE ? i / 2 : 0][2 * i % 4]), __uint_as_float(raw[j][FINE ? i / 2 : 0][2 * i % 4 + 1])};
          uint32_t part[2];
          const bool finite[2] = {fabsf(v[0]) <= 3.402823466e38f, fabsf(v[1]) <= 3.402823466e38f};
#pragma unroll
          for (int p = 0; p < PIECES; p++) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
              part[h] = __float_as_uint(v[h]) & 0xffff0000u;
              // an infinity or a NaN (a quiet one) is one piece
              if (!finite[h]) part[h] = p ? 0u : v[h] != v[h] ? 0x7fc00000u : part[h];
              v[h] -= __uint_as_float(part[h]);
            }
            out[p][i] = high_halves(part[1], part[0]);
          }
        }
      } else {
        out[0] = raw[j][0];
      }
#pragma unroll
      for (int p = 0; p < PIECES; p++) *reinterpret_cast<u32x4*>(to[p * ALL + c][lane]) = out[p];
    }
  }
};

// The lanes of columns 0 .. 7 of `low`, and in columns 8 .. 15 what `high` has eight lanes before.
__device__ __forceinline__ float two_tiles(float low, float high) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(low), __float_as_int(high), 0x118, 0xf, 0xc, false));
}
// What the lane eight columns on has (zero in columns 8 .. 15).
__device__ __forceinline__ uint32_t eight_on(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x108, 0xf, 0xf, true);
}

template <int D, int KIND, bool FINE, bool NARROW, int HT>
struct Wave {
  static constexpr int CH = D / 32, XT = D / 16, NG = kv_groups(KIND, D), PIECES = query_pieces(FINE), WP = FINE ? 3 : KIND == KV_INT4 ? 1 : 2;
  static constexpr int TILES = NARROW ? 1 : 2, X = 4 * TILES;  // scores of a lane; WP: pieces of a weight
  static constexpr bool BIAS = KIND == KV_INT4 && !FINE;  // codes enter as c + 24 or c + 136
  v4f o[HT][XT];
  float m[HT], safe[HT], l[HT];
  int lane;
  Nibbles nb;

  __device__ __forceinline__ void begin() {
#pragma unroll
    for (int t = 0; t < HT; t++) {
      m[t] = NEG_INF;
      safe[t] = l[t] = 0.0f;
#pragma unroll
      for (int x = 0; x < XT; x++) o[t][x] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
  }

  // the scores (in powers of two) of the lane's 2 x 4 tokens (NARROW: 4) of its head (HT = 2:
  // and of the sixteenth behind it)
  __device__ __forceinline__ void scores(const Half<D, KIND, false, NARROW>& t, const uint32_t (*q)[64][4], float c,
                                         float (&x)[HT][X]) const {
    const u32x4 minus = code_bias();
    v4f s[HT][2];
#pragma unroll
    for (int h = 0; h < HT; h++) s[h][0] = s[h][1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ch = 0; ch < CH; ch++) {
      u32x4 key[2];
#pragma unroll
      for (int h = 0; h < HT; h++) {
        u32x4 query[PIECES];
#pragma unroll
        for (int p = 0; p < PIECES; p++) query[p] = *reinterpret_cast<const u32x4*>(q[(p * HT + h) * CH + ch][lane]);
        v4f less = {0.0f, 0.0f, 0.0f, 0.0f}, d[2];
        if constexpr (BIAS) less = mfma(minus, query[0], less);
#pragma unroll
        for (int i = 0; i < 2; i++) {
          if (h == 0) key[i] = t.template keys<FINE>(i, ch, nb);
          d[i] = KIND == KV_INT4 ? less : s[h][i];
#pragma unroll
          for (int p = PIECES - 1; p >= 0; p--) d[i] = mfma(key[i], query[p], d[i]);
          if constexpr (KIND != KV_INT4) s[h][i] = d[i];
        }
        if constexpr (KIND == KV_INT4) {
#pragma unroll
          for (int i = 0; i < TILES; i++)
#pragma unroll
            for (int j = 0; j < 4; j++)
              s[h][i][j] = fmaf(t.scale(i, ch, j), NARROW ? two_tiles(d[0][j], d[1][j]) : d[i][j], s[h][i][j]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < HT; h++)
#pragma unroll
      for (int j = 0; j < X; j++) {
        x[h][j] = s[h][j / 4][j & 3];
        if constexpr (NARROW && KIND != KV_INT4) x[h][j] = two_tiles(s[h][0][j], s[h][1][j]);
        x[h][j] *= KIND == KV_INT8 ? c * t.scale(j / 4, 0, j & 3) : c;
      }
  }

  // Scores to weights.  32 tokens from `first` on, of which those from lo to n - 1 are seen:
  // the others weigh nothing and `keep` masks their values (bf16) or scales, for what
  // lies there may be anything.
  __device__ __forceinline__ void weigh(float (&x)[HT][X], int first, int lo, int n, uint32_t (&keep)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i++) keep[i] = ~0u;
    if (first < lo || first + ATTN_PAIR > n) {
      asm volatile("");  // a branch: made into selects this costs 45 instructions a step
      const int at = first + 4 * (lane >> 4);
#pragma unroll
      for (int j = 0; j < X; j++) {
        const int token = at + (NARROW ? 2 * (lane & 8) : j / 4 * 16) + (j & 3);
#pragma unroll
        for (int h = 0; h < HT; h++)
          if (token < lo || token >= n) x[h][j] = NEG_INF;
      }
      // bf16 values of both tiles; scales of the lane's own
#pragma unroll
      for (int j = 0; j < (KIND == KV_BF16 ? 8 : X); j++) {
        const int token = at + (NARROW && KIND != KV_BF16 ? 2 * (lane & 8) : j / 4 * 16) + (j & 3);
        if (token < lo || token >= n) keep[j / 2] &= j & 1 ? 0xffffu : 0xffff0000u;
      }
    }
#pragma unroll
    for (int h = 0; h < HT; h++) {
      float top = NEG_INF;
#pragma unroll
      for (int j = 0; j < X; j++) top = fmaxf(top, x[h][j]);
      if (__any(top - m[h] > ATTN_RISE)) raise(h, top);
#pragma unroll
      for (int j = 0; j < X; j++) x[h][j] = __builtin_amdgcn_exp2f((x[h][j] - safe[h]) - ATTN_RISE);
    }
  }

  __device__ __forceinline__ void add(Half<D, KIND, true, NARROW>& t, const float (&p)[HT][X], const uint32_t (&keep)[4], bool edge) {
    if (NG && edge) {
      asm volatile("");
#pragma unroll
      for (int i = 0; i < TILES; i++)
#pragma unroll
        for (int k = 0; k < 2 * NG; k++) t.s[i][k] &= keep[2 * i + (k & 1)];
    }
    constexpr int GROUPS = NG ? NG : 1;
#pragma unroll
    for (int g = 0; g < GROUPS; g++) {
      u32x4 w[HT][WP];
#pragma unroll
      for (int h = 0; h < HT; h++) {
        float ps[X];
#pragma unroll
        for (int j = 0; j < X; j++) ps[j] = NG ? p[h][j] * t.scale(j / 4, NG ? g : 0, j & 3) : p[h][j];
        weights(ps, w[h]);
        if (g == 0) {
#pragma unroll
          for (int j = 0; j < X / 2; j++)
            l[h] += p[h][2 * j] + p[h][2 * j + 1];
        }
      }
#pragma unroll
      for (int x = g * XT / GROUPS; x < (g + 1) * XT / GROUPS; x++) {
        const u32x4 value = t.template values<FINE>(x, keep, nb);
#pragma unroll
        for (int h = 0; h < HT; h++) {
#pragma unroll
          for (int i = WP - 1; i >= 0; i--) o[h][x] = mfma(value, w[h][i], o[h][x]);
          if constexpr (BIAS) {
#pragma unroll
            for (int i = 0; i < WP; i++) o[h][x] = mfma(code_bias(), w[h][i], o[h][x]);
          }
        }
      }
    }
  }

  // weights as bf16, or as pieces that add up to them
  __device__ __forceinline__ static void weights(const float (&p)[X], u32x4 (&w)[WP]) {
#pragma unroll
    for (int j = 0; j < X / 2; j++) {
      float lo = p[2 * j], hi = p[2 * j + 1];
#pragma unroll
      for (int i = 0; i < WP; i++) {
        w[i][j] = pack_bf16(lo, hi);
        lo -= low_f32(w[i][j]);
        hi -= high_f32(w[i][j]);
        if constexpr (NARROW) w[i][2 + j] = eight_on(w[i][j]);  // the second tile's, in the other half of the columns
      }
    }
  }

  __device__ __forceinline__ void raise(int h, float top) {
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if constexpr (NARROW) top = fmaxf(top, __shfl_xor(top, 8));
    const float to = fmaxf(m[h], top);
    const float f = to == m[h] ? 1.0f : __builtin_amdgcn_exp2f(m[h] - to);
    m[h] = to;
    safe[h] = to == NEG_INF ? 0.0f : to;
    l[h] *= f;
#pragma unroll
    for (int x = 0; x < XT; x++) o[h][x] *= f;
  }
};

// ------------------------------------------------------------------ kernel
// What a workgroup does at a time: pairs p0 .. p1 - 1 of one unit (a sequence's key
// head and 16 of its query heads).
struct Segment {
  Span sp;
  int b, unit, p0, p1;
  // from: where the share begins within the unit's cost, left: what it holds from there on
  __device__ __forceinline__ void at(Span span, int seq, int u, int from, long long left) {
    sp = span;
    b = seq;
    unit = u;
    p0 = from > ATTN_TURN ? from - ATTN_TURN : 0;
    p1 = left < sp.cost() - from ? from + (int)left - ATTN_TURN : sp.pairs();
  }
  __device__ __forceinline__ bool empty() const { return p1 <= p0; }
};

// Where the tiles of a wave's pairs lie: lane i looks after the wave's pair k + i, k a
// multiple of 64.  Behind the segment's last pair that one stands again.
template <int WAVES>
struct Places {
  int page[2], tile[2];
  int bad;  // (not a bool, whose padding would take the copies through memory)
  __device__ __forceinline__ void look(const AttnArgs& a, const Segment& g, int wave, int lane, int k, int tpp) {
    int pair = g.p0 + wave + (k + lane) * WAVES;
    pair = g.sp.first_pair() + (pair < g.p1 ? pair : g.p1 - 1);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      int t = pair * 2 + i;
      // a tile without tokens that are seen may have no page: the pair's other one once more
      if (t * KV_TILE >= g.sp.n) t--;
      else if ((t + 1) * KV_TILE <= g.sp.lo) t++;
      const int p = t / tpp;
      tile[i] = t - p * tpp;
      page[i] = a.table[(size_t)g.b * a.table_width + p];
    }
  }
  // pages outside the cache: none is read, and the segment's sums are no numbers
  __device__ __forceinline__ void check(const AttnArgs& a) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const bool out = page[i] < 0 || page[i] >= a.cache.pages;
      bad |= out ? 1 : 0;
      page[i] = out ? 0 : page[i];
    }
  }
};

// SPLIT: the pairs of all units, one after the other, are cut into shares of equal cost, one a
// workgroup, whose waves take a unit's pairs in turn.  A unit that lies within a share is
// finished there; else its parts go to the workgroup's two places (place 1: the part that
// begins a unit, place 0: one that does not) and attn_join_kernel adds them in
// order.  Without SPLIT a workgroup is a unit.
//
// A wave asks for its next pair's keys as soon as it has the scores of this one's, and for
// the values when it has added this one's, across the border of two segments too: the
// next segment's places and queries are looked up while this one is worked on.
template <int D, int KIND, bool FINE, bool NARROW, bool SPLIT, int WAVES, int HT>
__global__ void __launch_bounds__(64 * WAVES, WAVES / 4 > 2 ? WAVES / 4 : 2) attn_kernel(AttnArgs a) {
  constexpr int XT = D / 16, COLS = 16 * HT;
  __shared__ float part_o[WAVES][HT * XT][64][4];
  __shared__ uint32_t queries[query_pieces(FINE) * HT * D / 32][64][4];
  __shared__ float part_m[WAVES][COLS], part_l[WAVES][COLS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15;
  const int heads = a.cache.heads, ratio = a.q_heads / heads, tiles = head_tiles(ratio, COLS), units = heads * tiles;
  const int tpp = a.cache.page / KV_TILE;
  constexpr float CODES = KIND == KV_INT4 && FINE ? 16.0f : 1.0f;  // what codes_bf16() leaves out
  const float c = a.scale * 1.44269504088896341f * CODES;
  Lengths lengths;
  Segment g;
  long long left;  // what this workgroup's share holds behind g
  if constexpr (SPLIT) {
    const Counts n(a, lengths);
    const long long total = (long long)n.total * units, share = share_of(total, (int)gridDim.x), start = share * blockIdx.x;
    if (start >= total) return;
    left = total - start < share ? total - start : share;
    Begin to;
    if (!to.find(a, n, lengths, units, start)) return;
    g.at(to.sp, to.b, to.unit, to.from, left);
    left -= to.sp.cost() - to.from;
    if (g.empty()) return;  // the share ends within what stands in front of its only unit
  } else {
    const int n = a.lengths[blockIdx.x / units];
    left = 0;
    g.at(span_of(a, n), blockIdx.x / units, blockIdx.x % units, 0, (long long)1 << 40);
    if (g.empty()) {
      const int cols = ratio - g.unit % tiles * COLS < COLS ? ratio - g.unit % tiles * COLS : COLS;
      const size_t at = ((size_t)g.b * a.q_heads + g.unit / tiles * ratio + g.unit % tiles * COLS) * D;
      const float y = bad_length(a, n) ? __uint_as_float(0x7fc00000u) : 0.0f;
      for (int i = threadIdx.x; i < cols * D; i += 64 * WAVES) {
        if (a.y_dtype == 0) static_cast<float*>(a.y)[at + i] = y;
        else static_cast<uint16_t*>(a.y)[at + i] = f32_to_bf16(y);
      }
      return;
    }
  }
  Wave<D, KIND, FINE, NARROW, HT> w;
  w.lane = lane;
  Places<WAVES> at, at_ahead;
  auto locate = [&](const Segment& s, const Places<WAVES>& p, int k) {  // the wave's pair k
    const int head = s.unit / tiles;
    Where to;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const uint8_t* page = a.data + (size_t)__builtin_amdgcn_readlane(p.page[i], k & 63) * a.cache.page_bytes;
      const int in = __builtin_amdgcn_readlane(p.tile[i], k & 63);
      to.tile[i] = page + a.cache.tile(head, in);
      to.scales[i] = page + a.cache.scales(head, in);
    }
    return to;
  };
  auto first_head = [&](const Segment& s) { return s.unit / tiles * ratio + s.unit % tiles * COLS; };
  auto columns = [&](const Segment& s) { const int c = ratio - s.unit % tiles * COLS; return c < COLS ? c : COLS; };
  Queries<D, FINE, WAVES, HT> query;
  auto ask = [&](const Segment& s) {
    const size_t row = ((size_t)s.b * a.q_heads + first_head(s) + col) * D;
    query.load(col < columns(s) ? static_cast<const uint8_t*>(a.q) + row * (a.q_dtype == 2 ? 2 : 4) : nullptr,
               16 + col < columns(s), a.q_dtype, wave, lane);
  };
  Half<D, KIND, false, NARROW> keys;
  Half<D, KIND, true, NARROW> values;
  at.bad = 0;
  at.look(a, g, wave, lane, 0, tpp);
  ask(g);
  at.check(a);
  {
    const Where first = locate(g, at, 0);
    keys.load(first, lane);
    values.load(first, lane);
    query.put(queries, a.q_dtype, wave, lane);
  }
  __syncthreads();
  while (true) {
    bool more = SPLIT && left > 0;
    Segment ahead = g;
    if (more) {
      int seq = g.b, unit = g.unit + 1;
      Span sp = g.sp;
      if (unit == units) {
        unit = 0;
        do {
          if (++seq >= a.B) return;  // not reached: what is left of the share lies in units
          sp = lengths.span(a, seq);
        } while (sp.pairs() == 0);
      }
      ahead.at(sp, seq, unit, 0, left);
      left -= sp.cost();
      if (ahead.empty()) {
        ahead = g;
        more = false;
      }
    }
    if (more) {
      at_ahead.bad = 0;
      at_ahead.look(a, ahead, wave, lane, 0, tpp);
      ask(ahead);
    } else {
      at_ahead = at;
    }
    const int cols = columns(g);
    const size_t q_row = ((size_t)g.b * a.q_heads + first_head(g) + col) * D;
    w.begin();
    const int count = g.p1 - g.p0 > wave ? (g.p1 - g.p0 - wave + WAVES - 1) / WAVES : 0;
    for (int k = 0; k < count; k++) {
      const int first = (g.sp.first_pair() + g.p0 + wave + k * WAVES) * ATTN_PAIR;
      float x[HT][NARROW ? 4 : 8];
      w.scores(keys, queries, c, x);
      // the wave's pair k + 1, or the next segment's first, or (no such) a few lines again: a
      // load that may be left out would make the compiler wait for all of them
      Where next;
      if (k + 1 < count) {
        if (((k + 1) & 63) == 0) {
          at.look(a, g, wave, lane, k + 1, tpp);
          at.check(a);
        }
        next = locate(g, at, k + 1);
      } else {
        at_ahead.check(a);
        next = locate(ahead, at_ahead, 0);
      }
      const int reader = more || k + 1 < count ? lane : 0;
      keys.load(next, reader);
      uint32_t keep[4];
      w.weigh(x, first, g.sp.lo, g.sp.n, keep);
      w.add(values, x, keep, first < g.sp.lo || first + ATTN_PAIR > g.sp.n);
      values.load(next, reader);
    }
    if (count == 0 && more) {
      at_ahead.check(a);
      const Where next = locate(ahead, at_ahead, 0);
      keys.load(next, lane);
      values.load(next, lane);
    }
#pragma unroll
    for (int h = 0; h < HT; h++) {
      w.l[h] += __shfl_xor(w.l[h], 16);
      w.l[h] += __shfl_xor(w.l[h], 32);
      if constexpr (NARROW) w.l[h] += __shfl_xor(w.l[h], 8);
      if (__any(at.bad)) w.l[h] = __uint_as_float(0x7fc00000u);
    }
    // the waves' sums: every wave adds a share of the channels, in the order of the waves
    __syncthreads();
#pragma unroll
    for (int h = 0; h < HT; h++) {
      if (lane < 16) {
        part_m[wave][16 * h + lane] = w.m[h];
        part_l[wave][16 * h + lane] = w.l[h];
      }
#pragma unroll
      for (int x = 0; x < XT; x++) *reinterpret_cast<v4f*>(part_o[wave][h * XT + x][lane]) = w.o[h][x];
    }
    if (more) query.put(queries, a.q_dtype, wave, lane);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < HT; h++) {
      const int head = 16 * h + col;
      float m = NEG_INF, f[WAVES], l = 0.0f;
#pragma unroll
      for (int i = 0; i < WAVES; i++) m = fmaxf(m, part_m[i][head]);
#pragma unroll
      for (int i = 0; i < WAVES; i++) {
        f[i] = part_m[i][head] == m ? 1.0f : __builtin_amdgcn_exp2f(part_m[i][head] - m);
        l += f[i] * part_l[i][head];
      }
      const bool whole = g.p0 == 0 && g.p1 == g.sp.pairs();
      const float inv = (whole ? 1.0f / l : 1.0f) * CODES;  // l is 0 where every score is -infinity: a NaN, as the formula's
      float* place = a.part + ((size_t)blockIdx.x * 2 + (g.p0 == 0)) * slot_floats(D, COLS);
      for (int x = wave; x < XT; x += WAVES) {
        v4f s = *reinterpret_cast<const v4f*>(part_o[0][h * XT + x][lane]) * f[0];
#pragma unroll
        for (int i = 1; i < WAVES; i++) s += *reinterpret_cast<const v4f*>(part_o[i][h * XT + x][lane]) * f[i];
        s *= inv;
        if (head < cols) {
          const int ch = 16 * x + 4 * (lane >> 4);
          if (!whole) *reinterpret_cast<v4f*>(place + head * D + ch) = s;
          else if (a.y_dtype == 0) *reinterpret_cast<v4f*>(static_cast<float*>(a.y) + q_row + 16 * h * D + ch) = s;
          else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + q_row + 16 * h * D + ch) = u32x2{pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
        }
      }
      if (!whole && wave == 0 && lane < 16) {
        place[COLS * D + 16 * h + lane] = m;
        place[COLS * (D + 1) + 16 * h + lane] = l;
      }
    }
    if (!more) return;
    g = ahead;
    at = at_ahead;
  }
}

// Joins the parts of units that were cut, `hb` query heads of one unit a workgroup:
// D / 4 threads go through the parts of a head that fall to their group of them, eight
// parts in flight, and the groups' sums are added in order.  Sequences without tokens or
// with a bad length are filled here.
//
// The workgroups are those of every unit, or with BORDERS those of every border of two shares, of
// which the first in a unit joins it, and behind them one for each four sequences, a wave each.
// A workgroup of either kind reads all lengths, so that the former takes time with the square of the
// sequences and is for no more units than there are shares.  B sequences of 1 to 200 tokens and one of
// 4096, 8 key heads of 128, 8 bits, the whole call with a workgroup a unit and with borders: B = 96 30.8
// and 30.2 us, 128 34.0 and 31.6, 256 53.7 and 45.9, 1024 251 and 131, 4096 2244 and 408.
template <int D, bool BORDERS>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnArgs a, int grid, int cols, int hb, int blocks) {
  constexpr int Q = D / 4, SLOTS = 256 / Q, N = 8;
  __shared__ v4f sums[SLOTS][Q];
  __shared__ float slot_m[SLOTS], slot_l[SLOTS];
  const int heads = a.cache.heads, ratio = a.q_heads / heads, tiles = head_tiles(ratio, cols), units = heads * tiles;
  const int tid = threadIdx.x;
  auto put_at = [&](size_t at, v4f y) {
    if (a.y_dtype == 0) *reinterpret_cast<v4f*>(static_cast<float*>(a.y) + at) = y;
    else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + at) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
  };
  auto nothing = [&](int length) { return bad_length(a, length) ? __uint_as_float(0x7fc00000u) : 0.0f; };
  if (BORDERS && (int)blockIdx.x >= (grid - 1) * blocks) {
    const int b = ((int)blockIdx.x - (grid - 1) * blocks) * 4 + (tid >> 6);
    if (b >= a.B) return;
    const int length = a.lengths[b];
    if (span_of(a, length).pairs()) return;
    const float y = nothing(length);
    const int count = a.q_heads * D;
    for (int i = 4 * (tid & 63); i < count; i += 256) put_at((size_t)b * count + i, v4f{y, y, y, y});
    return;
  }
  Lengths lengths;
  const Counts n(a, lengths);
  const long long total = (long long)n.total * units, share = share_of(total, grid);
  int b, unit, pairs, length = 0;
  long long start;  // of the unit's pairs within what all units cost
  if constexpr (BORDERS) {
    const int border = blockIdx.x / blocks + 1;
    Begin to;
    if (share * border >= total || !to.find(a, n, lengths, units, share * border)) return;
    b = to.b;
    unit = to.unit;
    pairs = to.sp.pairs();
    start = share * border - to.from + ATTN_TURN;
    if (quotient(start, share) != border - 1) return;  // cut further in front, or here before its first pair
  } else {
    b = blockIdx.y;
    unit = blockIdx.x / blocks;
    length = n.each > 1 ? a.lengths[b] : __builtin_amdgcn_readlane(lengths.held, b);
    pairs = span_of(a, length).pairs();
    int front = __builtin_amdgcn_readlane(n.before, b / n.each);
    for (int i = b / n.each * n.each; i < b; i++) front += span_of(a, a.lengths[i]).cost();
    start = (long long)front * units + (long long)unit * (pairs + ATTN_TURN) + ATTN_TURN;
  }
  const int slot = tid / Q, d = tid % Q, groups = SLOTS / hb, group = slot / hb, col = blockIdx.x % blocks * hb + slot % hb;
  const bool on = group < groups && col < cols && unit % tiles * cols + col < ratio;
  const size_t at = ((size_t)b * a.q_heads + unit / tiles * ratio + unit % tiles * cols + col) * D + 4 * d;
  auto put = [&](v4f y) { put_at(at, y); };
  if (!BORDERS && !pairs) {
    const float y = nothing(length);
    if (on && group == 0) put(v4f{y, y, y, y});
    return;
  }
  const int w0 = (int)quotient(start, share), w1 = (int)quotient(start + pairs - 1, share), parts = w1 - w0 + 1;
  if (parts == 1 || w1 >= grid) return;  // the latter not while the lengths stay as they were counted
  float m = NEG_INF, l = 0.0f;
  v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i0 = group; on && i0 < parts; i0 += N * groups) {
    float pm[N], pl[N];
    v4f py[N];
#pragma unroll
    for (int k = 0; k < N; k++) {  // behind the last part this group's first stands again, with no weight
      const int i = i0 + k * groups < parts ? i0 + k * groups : i0;
      const float* p = a.part + ((size_t)(w0 + i) * 2 + (i == 0)) * slot_floats(D, cols);
      pm[k] = p[cols * D + col];
      pl[k] = p[cols * (D + 1) + col];
      py[k] = *reinterpret_cast<const v4f*>(p + col * D + 4 * d);
    }
    float to = m;
#pragma unroll
    for (int k = 0; k < N; k++) to = fmaxf(to, pm[k]);
    float f = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
    y *= f;
    l *= f;
    m = to;
#pragma unroll
    for (int k = 0; k < N; k++) {
      f = pm[k] == m ? 1.0f : __builtin_amdgcn_exp2f(pm[k] - m);
      if (i0 + k * groups < parts) {
        l += f * pl[k];
        y += f * py[k];
      }
    }
  }
  if (on) sums[slot][d] = y;
  if (on && d == 0) {
    slot_m[slot] = m;
    slot_l[slot] = l;
  }
  __syncthreads();
  if (!on || group) return;
  const int used = groups < parts ? groups : parts;
  float to = m;
  for (int i = 1; i < used; i++) to = fmaxf(to, slot_m[slot + i * hb]);
  float f = m == to ? 1.0f : __builtin_amdgcn_exp2f(m - to);
  y *= f;
  l *= f;
  for (int i = 1; i < used; i++) {
    const int k = slot + i * hb;
    f = slot_m[k] == to ? 1.0f : __builtin_amdgcn_exp2f(slot_m[k] - to);
    l += f * slot_l[k];
    y += f * sums[k][d];
  }
  put(y * (1.0f / l));
}

// ------------------------------------------------------------------ host
// Units as they are, a workgroup each, or cut into equal shares and joined?  The former is
// one launch (the join is some 6 us with its launch) but takes its longest unit's time; the latter takes 11
// us at least, and more where parts are many.  So the former is for units that take, by
// what the host knows of the longest, no more than 5.5 us beside what any launch takes, and up to 13
// where there are many units.  8 key heads of 128, 8 bits, in us as units and cut: 1 x 512 tokens
// 8.4 and 10.4, 1 x 1024 11.5 and 11.1, 8 x 1024 11.9 and 16.1, 16 x 2048 18.8 and 22.0, 64 of 1
// to 1536 25.8 and 30.9; beyond the limit 8 of 1 to 2048 17.7 and 16.8, 16 of 1 to 3000 23.8 and 20.7.
constexpr float attn_unit_ns(int units) { return units < 120 ? 5500.0f + 62.5f * units : 13000.0f; }
// What a token of a long unit costs, by the chip's times over 1024 to 2048 tokens, heads of 64 to
// 256: bf16 5.0 to 16.6 ns (60 bytes a ns into a CU), codes with four waves 8.2 to 11.8, as long as an
// access takes, with eight 5.0 to 10.1; FINE 8 bits 6.3 to 10.1, 15.4 with four waves, 4
// bits 7.1 to 17.5, four waves 11 to 26.
// Eight waves are for codes and as many units as there are CUs (16 x 1024 tokens of 8 bits 14.3 ->
// 12.3 us, 8 x 1024 of 4 bits 16.8 -> 12.6); for up to 256 tokens (16 x 256: 7.3 -> 7.5 us), bf16 (16 x
// 1024: 15.7 -> 16.3) and more units (64 x 512 of 8 bits 15.8 -> 16.5) four are faster.
constexpr float attn_token_ns(int D, int kind, bool fine, bool wide) {
  if (kind == KV_BF16) return 1.0f + D / 16.5f;
  if (kind == KV_INT8) return wide ? (3.5f + D / 50.0f) * (fine ? 1.25f : 1.0f) : 7.0f + D / (fine ? 30.0f : 60.0f);
  return wide ? fine ? D / 11.0f : 3.5f + D / 40.0f : 7.0f + D / (fine ? 15.0f : 60.0f);
}

template <int D, int KIND, bool FINE, bool NARROW, int HT>
void attn_cut(const AttnArgs& a) {
  const int ratio = a.q_heads / a.cache.heads, units = a.cache.heads * head_tiles(ratio, 16 * HT);
  // The third workgroup a CU is for long work: 32 units of 4096 tokens of 64 channels in 8 bits take
  // 15.1 us with 512 workgroups and 15.6 with 768, of 16384 24.7 and 23.3; 14 of 33028 of 96 in 4 bits a
  // step of 34.3 and 32.5.
  const int longest = a.window > 0 && a.window < a.max_length ? a.window : a.max_length;
  const bool little = (long long)a.B * units * longest < 12288LL * ATTN_PAIR;
  constexpr int full = attn_grid(D, KIND, FINE, NARROW);
  const int grid = full > 512 && little ? 512 : full;
  hipLaunchKernelGGL((attn_kernel<D, KIND, FINE, NARROW, true, ATTN_WAVES, HT>), dim3(grid), dim3(64 * ATTN_WAVES), 0, a.stream, a);
  // Heads of a workgroup of the join: one where there are few, else as many as leave the
  // longest unit (all tokens in one sequence) 64 parts a group at most, and two at least.  With one
  // head each 64 sequences of 64 heads take 11.9 us instead of 5.8, of 32 heads of one key head 10.0
  // instead of 6.4.
  constexpr int SLOTS = 256 / (D / 4);
  const int most = ratio < 16 * HT ? ratio : 16 * HT, groups = (grid / units + 2 + 63) / 64;
  int hb = a.B * a.q_heads <= 512 ? 1 : groups > SLOTS / 2 ? 2 : SLOTS / groups;
  hb = hb < most ? hb : most;
  const int blocks = (most + hb - 1) / hb;
  if ((long long)a.B * units > grid) {
    const dim3 all((unsigned)((grid - 1) * blocks + (a.B + 3) / 4));
    hipLaunchKernelGGL((attn_join_kernel<D, true>), all, dim3(256), 0, a.stream, a, grid, 16 * HT, hb, blocks);
  } else {
    hipLaunchKernelGGL((attn_join_kernel<D, false>), dim3(units * blocks, a.B), dim3(256), 0, a.stream, a, grid, 16 * HT, hb, blocks);
  }
}

template <int D, int KIND, bool FINE, bool NARROW>
void attn_launch(const AttnArgs& a) {
  const int ratio = a.q_heads / a.cache.heads, units = a.cache.heads * head_tiles(ratio, 16);
  const int longest = a.window > 0 && a.window < a.max_length ? a.window : a.max_length;
  constexpr bool can_wide = KIND != KV_BF16 && !(FINE && D == 256);  // (those would spill)
  const bool wide = can_wide && a.B * units <= 256 && longest > 256;
  if (longest * attn_token_ns(D, KIND, FINE, wide) <= attn_unit_ns(a.B * units)) {
    const dim3 blocks((unsigned)(a.B * units));
    if constexpr (can_wide) {
      if (wide) {
        hipLaunchKernelGGL((attn_kernel<D, KIND, FINE, NARROW, false, 8, 1>), blocks, dim3(512), 0, a.stream, a);
        return;
      }
    }
    hipLaunchKernelGGL((attn_kernel<D, KIND, FINE, NARROW, false, ATTN_WAVES, 1>), blocks, dim3(64 * ATTN_WAVES), 0, a.stream, a);
    return;
  }
  if constexpr (attn_two(D, KIND, FINE)) {
    if (ratio > 16) return attn_cut<D, KIND, FINE, NARROW, 2>(a);
  }
  attn_cut<D, KIND, FINE, NARROW, 1>(a);
}

template <int D>
void attn_by_kind(const AttnArgs& a) {
  const bool fine = a.q_dtype == 0 || a.y_dtype == 0;
  if (a.cache.kind == KV_BF16) fine ? attn_launch<D, KV_BF16, true, false>(a) : attn_launch<D, KV_BF16, false, false>(a);
  else if (a.cache.kind == KV_INT8) fine ? attn_launch<D, KV_INT8, true, false>(a) : attn_launch<D, KV_INT8, false, false>(a);
  else if (a.q_heads / a.cache.heads <= 8) fine ? attn_launch<D, KV_INT4, true, true>(a) : attn_launch<D, KV_INT4, false, true>(a);
  else fine ? attn_launch<D, KV_INT4, true, false>(a) : attn_launch<D, KV_INT4, false, false>(a);
}

}  // namespace

size_t attn_workspace(const KvLayout& l) {  // two parts a workgroup, of what takes most
  size_t most = 0;
  for (int form = 0; form < 4; form++) {
    const bool fine = form & 1, narrow = form & 2;
    const size_t floats = attn_grid(l.D, l.kind, fine, narrow) * 2 * slot_floats(l.D, attn_two(l.D, l.kind, fine) ? 32 : 16);
    most = floats > most ? floats : most;
  }
  return align_up(most * 4, 256);
}

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
