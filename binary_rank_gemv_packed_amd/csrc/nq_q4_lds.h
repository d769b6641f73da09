// Shared memory of a workgroup of the 4-bit decode kernel (nq_q4.hip), from
// offset 0: the fp16 image of x, P pieces of [tiles][B][128]; a power of two for
// each (tile, row of x); the sums kept of shared row tiles, [keep][W][B][16] floats.
// The sums are written four floats at a time, so they begin at a multiple of 16
// bytes, which tiles x B floats need not be.  No HIP header: also read by a host
// program.
#pragma once

#include <stddef.h>

namespace nq {

struct Q4DecLds {
  size_t fac, red, total;  // bytes
};

constexpr int q4_dec_fac_floats(int B, int tiles) { return (tiles * B + 3) / 4 * 4; }

constexpr Q4DecLds q4_dec_lds(int P, int B, int tiles, int W, int keep) {
  const size_t fac = (size_t)P * tiles * B * 256, red = fac + (size_t)q4_dec_fac_floats(B, tiles) * 4;
  return {fac, red, red + (size_t)keep * W * B * 64};
}

}  // namespace nq
