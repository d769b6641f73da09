// Layout of the paged cache of keys and values, and the store of one head of one
// token into it (nq_kv.hip writes and reads it, nq_head.hip writes it, nq_attn.hip
// reads it).
//
// A page holds `page` slots (one for each token) of every head, in tiles of 16
// slots that are the register operands of the attention's MFMA 16x16x32 as they
// are, so that a wavefront reads a tile with contiguous 16-byte loads and uses it
// without a shuffle:
//   keys    lane L: slot L & 15, channels 32 i + 8 (L >> 4) + [0, 8), i = 0 .. D/32 - 1;
//   values  lane L: channel 16 x + (L & 15), slots 4 (L >> 4) + [0, 4), x = 0 .. D/16 - 1.
// A lane's bytes, i or x slowest, are cut into pieces of 16 (a last one of 8 or 12
// where D leaves it); a tile is [piece][64 lanes].  Within 8 keys or 4 values:
//   bf16  one after the other;
//   int8  one after the other, signed bytes;
//   int4  code + 8 in a nibble.  Keys: nibble p is channel 2p of the eight, nibble
//         p + 4 channel 2p + 1.  Values: for channels 32 i + c and 32 i + 16 + c (low and high
//         nibble, c = L & 15) a byte a slot, slots in the order 0, 2, 1, 3.
// Both put the two halves of a packed pair 16 bits apart.  No byte holds parts of
// two slots.  Page: [head][tile]{keys, values} | scales [head][tile][4 quads of slots]
// {keys [NG], values [NG]}[4 slots], bf16, NG groups of channels a head, so that what a
// lane needs for its four slots lies together; the page is rounded up to 256 bytes.
#pragma once

#include "nq_common.h"

namespace nq {

enum { KV_BF16 = 0, KV_INT8 = 1, KV_INT4 = 2 };
constexpr int KV_TILE = 16;  // slots

__host__ __device__ constexpr int kv_bits(int kind) { return kind == KV_BF16 ? 16 : kind == KV_INT8 ? 8 : 4; }
__host__ __device__ constexpr int kv_groups(int kind, int D) { return kind == KV_BF16 ? 0 : kind == KV_INT8 ? 1 : D / 32; }
__host__ __device__ constexpr int kv_half_bytes(int kind, int D) { return 2 * D * kv_bits(kind); }  // keys or values of a tile
__host__ __device__ constexpr int kv_lane_bytes(int kind, int D) { return D * kv_bits(kind) / 32; }
__host__ __device__ constexpr int kv_scale_bytes(int kind, int D) { return 2 * 2 * 16 * kv_groups(kind, D); }  // of a tile

// Byte b of a lane within its half of a tile.
__host__ __device__ inline int kv_byte(int lane, int b, int lane_bytes) {
  const int whole = lane_bytes & ~15, rest = lane_bytes & 15;
  return b < whole ? (b >> 4) * 1024 + lane * 16 + (b & 15) : (whole >> 4) * 1024 + lane * rest + (b - whole);
}

// Entry of a tile's scales.
__host__ __device__ inline int kv_scale_at(int row, int value, int group, int groups) {
  return (((row >> 2) * 2 + value) * groups + group) * 4 + (row & 3);
}

struct KvLayout {
  int pages, heads, D, page, kind;
  size_t off_scales, page_bytes;
  __host__ __device__ size_t tile(int head, int t) const {
    return ((size_t)head * (page / KV_TILE) + t) * 2 * kv_half_bytes(kind, D);
  }
  __host__ __device__ size_t scales(int head, int t) const {
    return off_scales + ((size_t)head * (page / KV_TILE) + t) * kv_scale_bytes(kind, D);
  }
};

__host__ __device__ inline KvLayout kv_layout(int pages, int heads, int D, int page, int kind) {
  KvLayout l{pages, heads, D, page, kind, 0, 0};
  const size_t tiles = (size_t)heads * (page / KV_TILE);
  l.off_scales = tiles * 2 * kv_half_bytes(kind, D);
  l.page_bytes = align_up(l.off_scales + tiles * kv_scale_bytes(kind, D), 256);
  return l;
}

#ifdef __HIPCC__
// A slot's place: its page's address, tile and row, or a null page where the slot is
// not one of the cache's.
struct KvPlace {
  uint8_t* page;
  int tile, row;
};
__device__ inline KvPlace kv_place(const KvLayout& l, uint8_t* data, int64_t slot) {
  if (slot < 0 || slot >= (int64_t)l.pages * l.page) return KvPlace{nullptr, 0, 0};
  const uint32_t t = (uint32_t)(slot >> 4), tpp = (uint32_t)l.page >> 4, p = t / tpp;  // below 2^30: a division of 32 bits
  return KvPlace{data + p * l.page_bytes, (int)(t - p * tpp), (int)(slot & 15)};
}

// Two fp32 to bf16, to the nearest, lo in the lower half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const bf2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// The scale of a group: bf16(top / most), top the largest magnitude's bits (as
// whole numbers they are ordered as the values are, infinities and NaN on top).  A
// group with an infinity or a NaN gets a NaN.
__device__ inline float kv_scale(uint32_t top, float most) {
  if (top >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return __uint_as_float((uint32_t)f32_to_bf16(__uint_as_float(top) / most) << 16);
}

// c[e] = v[e] / s to the nearest whole number, ties to even, of the quotient as a
// division rounds it.  The product with 1 / s is off by under 127.5 x 2^-23 < 2^-16 of it: only
// within 2^-15 of a tie, and for scales whose reciprocal is not a normal number, does
// the division itself decide (some 25 instructions; with one for every value 131072
// tokens of 8 heads took 314 us to write).  A scale of zero (a group below 2^-134 x most) or NaN gives zeros.
// Elsewhere |v / s| is below most + 1/2, for s is within 2^-8 of the quotient it stands for.
__device__ __forceinline__ void kv_codes(const float (&v)[8], float s, int most, int (&c)[8]) {
  const bool usual = s >= 0x1p-100f && s <= 0x1p100f, some = s > 0.0f;
  const float r = 1.0f / s;
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const float q = v[e] * r, n = rintf(q);
    c[e] = (int)n;
    const bool unsure = some && !(usual && fabsf(q - n) < 0.5f - 0x1p-15f);
    if (__any(unsure)) {
      const int exact = (int)rintf(v[e] / s);
      if (unsure) c[e] = exact < -most ? -most : exact > most ? most : exact;
    }
    if (!some) c[e] = 0;
  }
}

// Largest over the LG lanes (a power of two) of one head.
template <int LG>
__device__ inline uint32_t kv_top(uint32_t top) {
#pragma unroll
  for (int o = 1; o < LG; o *= 2) {
    const uint32_t other = __shfl_xor(top, o);
    top = other > top ? other : top;
  }
  return top;
}

// Stores channels 8 m .. 8 m + 7 (v, m = lane of its head's LG lanes, `on` where
// 8 m < D) of one head of one token as its key and / or value.  All lanes of the
// wavefront take part in the exchanges; those without a place store nothing.
template <int KIND, int LG, bool VALUE>
__device__ inline void kv_store(const KvLayout& l, const KvPlace& at, int head, int m, bool on, const float (&v)[8]) {
  constexpr int kind = KIND;
  const int D = l.D, lb = kv_lane_bytes(kind, D);
  const bool write = on && at.page != nullptr;
  uint8_t* half = at.page + l.tile(head, at.tile) + (VALUE ? kv_half_bytes(kind, D) : 0);
  const int klane = at.row + 16 * (m & 3);      // keys: the lane of these channels
  const int x = m >> 1, c0 = 8 * (m & 1);       // values: channel tile, first channel in it
  const int vg = at.row >> 2, vj = at.row & 3;  // values: lane group and place of the slot
  if (kind == KV_BF16) {
    if (!write) return;
    if (!VALUE) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; i++) u[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<uint4*>(half + kv_byte(klane, 16 * (m >> 2), lb)) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint32_t two = pack_bf16(v[e], v[e + 1]);
        *reinterpret_cast<uint16_t*>(half + kv_byte(c0 + e + 16 * vg, 8 * x + 2 * vj, lb)) = (uint16_t)two;
        *reinterpret_cast<uint16_t*>(half + kv_byte(c0 + e + 1 + 16 * vg, 8 * x + 2 * vj, lb)) = (uint16_t)(two >> 16);
      }
    }
    return;
  }
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const uint32_t bits = on ? __float_as_uint(v[e]) & 0x7fffffffu : 0u;
    top = bits > top ? bits : top;
  }
  constexpr bool wide = kind == KV_INT8;
  top = wide ? kv_top<LG>(top) : kv_top<4>(top);
  const int most = wide ? 127 : 7;
  const float s = kv_scale(top, (float)most);
  int q[8];
  kv_codes(v, s, most, q);
  uint16_t* scales = reinterpret_cast<uint16_t*>(at.page + l.scales(head, at.tile));
  if (write && (wide ? m == 0 : (m & 3) == 0))
    scales[kv_scale_at(at.row, VALUE, wide ? 0 : m >> 2, kv_groups(kind, D))] = (uint16_t)(__float_as_uint(s) >> 16);
  if (wide) {
    if (!write) return;
    if (!VALUE) {
      uint32_t u[2];
#pragma unroll
      for (int i = 0; i < 2; i++)
        u[i] = (q[4 * i] & 255) | (q[4 * i + 1] & 255) << 8 | (q[4 * i + 2] & 255) << 16 | (uint32_t)q[4 * i + 3] << 24;
      *reinterpret_cast<uint2*>(half + kv_byte(klane, 8 * (m >> 2), lb)) = make_uint2(u[0], u[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) half[kv_byte(c0 + e + 16 * vg, 4 * x + vj, lb)] = (uint8_t)q[e];
    }
    return;
  }
  if (!VALUE) {
    uint32_t u = 0;
#pragma unroll
    for (int p = 0; p < 4; p++) u |= (uint32_t)(q[2 * p] + 8) << (4 * p) | (uint32_t)(q[2 * p + 1] + 8) << (4 * p + 16);
    if (write) *reinterpret_cast<uint32_t*>(half + kv_byte(klane, 4 * (m >> 2), lb)) = u;
  } else {  // the lane of the lower sixteen channels of a group stores both
    const int place = vj == 1 ? 2 : vj == 2 ? 1 : vj;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const int high = __shfl_xor(q[e], 2);
      if (write && !(m & 2)) half[kv_byte(c0 + e + 16 * vg, 4 * (m >> 2) + place, lb)] = (uint8_t)(q[e] + 8 | (high + 8) << 4);
    }
  }
}

// Channels 8 m .. 8 m + 7 of one head's key or value as they are held.
template <int KIND, bool VALUE>
__device__ inline void kv_load(const KvLayout& l, const KvPlace& at, int head, int m, float (&v)[8]) {
  constexpr int kind = KIND;
  const int D = l.D, lb = kv_lane_bytes(kind, D);
  const uint8_t* half = at.page + l.tile(head, at.tile) + (VALUE ? kv_half_bytes(kind, D) : 0);
  const int klane = at.row + 16 * (m & 3), x = m >> 1, c0 = 8 * (m & 1), vg = at.row >> 2, vj = at.row & 3;
  if (kind == KV_BF16) {
    if (!VALUE) {
      const uint4 u = *reinterpret_cast<const uint4*>(half + kv_byte(klane, 16 * (m >> 2), lb));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++)
        v[e] = to_f32<uint16_t>(*reinterpret_cast<const uint16_t*>(half + kv_byte(c0 + e + 16 * vg, 8 * x + 2 * vj, lb)));
    }
    return;
  }
  const uint16_t* scales = reinterpret_cast<const uint16_t*>(at.page + l.scales(head, at.tile));
  const float s = to_f32<uint16_t>(scales[kv_scale_at(at.row, VALUE, kind == KV_INT8 ? 0 : m >> 2, kv_groups(kind, D))]);
  if (kind == KV_INT8) {
    if (!VALUE) {
      const uint2 u = *reinterpret_cast<const uint2*>(half + kv_byte(klane, 8 * (m >> 2), lb));
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] = s * (float)(int8_t)((e < 4 ? u.x : u.y) >> (8 * (e & 3)));
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] = s * (float)(int8_t)half[kv_byte(c0 + e + 16 * vg, 4 * x + vj, lb)];
    }
    return;
  }
  if (!VALUE) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(half + kv_byte(klane, 4 * (m >> 2), lb));
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = s * (float)((int)(u >> (4 * (e >> 1) + 16 * (e & 1)) & 15) - 8);
  } else {
    const int place = vj == 1 ? 2 : vj == 2 ? 1 : vj;
#pragma unroll
    for (int e = 0; e < 8; e++)
      v[e] = s * (float)((int)(half[kv_byte(c0 + e + 16 * vg, 4 * (m >> 2) + place, lb)] >> (m & 2 ? 4 : 0) & 15) - 8);
  }
}
#endif

}  // namespace nq
