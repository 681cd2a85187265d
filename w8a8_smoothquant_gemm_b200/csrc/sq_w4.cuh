// sq_w4.cuh -- the 4-bit weight format and the products on it, shared by the few-token GEMM and
// the mixture-of-experts layer.
//
// Format ("量化：只压权重，与训练后量化（PTQ）": group-wise INT4 weights, group 128, activations left in
// 16 bits).  A row of K codes is cut into blocks of 128, 64 bytes each (the last one padded with
// zero nibbles).  Inside a block, k = 32 w + 8 t + i (w, t < 4, i < 8) sits in the 32-bit word at
// byte 16 t + 4 w, nibble i / 2 + 4 (i % 2).  So
//   - lane t of a quad reads the 16 bytes of "its" k with one load and holds, for each w, the 8
//     consecutive codes 8 t .. 8 t + 7 of the 32-code group w: every mma step stays inside one
//     group of 32, and any group size that is a multiple of 32 needs no exchange of codes;
//   - (word >> 4 p) & 0x000f000f is the pair (code 2 p, code 2 p + 1), two consecutive k, as the
//     mma's packed operands want them: one shift and one three-input logic operation a pair.
#pragma once

#include "sq_ptx.cuh"

namespace sqk {

constexpr int W4_BLOCK = 128;       // codes per block
constexpr int W4_BLOCK_BYTES = 64;  // bytes per block

__host__ __device__ __forceinline__ int64_t w4_blocks(int64_t K) { return (K + W4_BLOCK - 1) / W4_BLOCK; }

// Bits of the bf16 number 128 + v for an integer 0 <= v < 128 (exact: 128 .. 255 have spacing 1).
__device__ __forceinline__ uint32_t bf16_128_plus(uint32_t v) { return 0x4300u + v; }

// Pair p of a word as two bf16 numbers (code - zero), exact; `z` holds 128 + zero twice.
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int p, uint32_t z) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(word >> (4 * p)), "n"(0x000f000f), "n"(0x43004300));
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(z));
  return d;
}

// D += A B, 16 x 8 x 16, bf16 operands, binary32 sums.  Lane (g, t) = (lane / 4, lane % 4) holds
// a0, a2 of row g and a1, a3 of row g + 8 for the k pairs (2t, 2t + 1) and (2t + 8, 2t + 9), b0 and
// b1 of column g for the same k, d0, d1 of row g, columns 2t, 2t + 1, and d2, d3 of row g + 8.
// Which k the sixteen slots stand for is free as long as A and B agree.
__device__ __forceinline__ void mma_bf16(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x as a sum of bf16 numbers.  Parts are cut off, not rounded, so a finite x is exactly the sum of
// three (8 + 8 + 8 significand bits; the last ones of numbers near the subnormal range may be
// lost) and two keep 16 bits.  Infinities and NaN stand in the first part, the others are then 0.
template <int S>
__device__ __forceinline__ void split_bf16(float x, uint32_t part[S]) {
  uint32_t b = __float_as_uint(x);
  if ((b & 0x7f800000u) == 0x7f800000u) {
    part[0] = (b >> 16) | ((b & 0x007fffffu) ? 0x40u : 0u);
#pragma unroll
    for (int s = 1; s < S; ++s) part[s] = 0u;
    return;
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    part[s] = b >> 16;
    b = __float_as_uint(__fsub_rn(__uint_as_float(b), __uint_as_float(b & 0xffff0000u)));
  }
}

// The same for values whose parts are stored for a later product: two parts are rounded, not cut
// (error at most 2^-16 of the value).  A finite value whose first part would round to infinity is cut.
template <int S>
__device__ __forceinline__ void split_bf16_stored(float x, uint32_t part[S]) {
  if (S == 2) {
    const uint32_t hi = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    if ((hi & 0x7f80u) != 0x7f80u) {
      part[0] = hi;
      part[1] = __bfloat16_as_ushort(__float2bfloat16_rn(__fsub_rn(x, __uint_as_float(hi << 16))));
      return;
    }
  }
  split_bf16<S>(x, part);
}

// One lane's share of 16 rows x 128 codes: 16 bytes of row g and of row g + 8, and for each the
// scale and zero point of one group of the block (lane t those of the group that holds 32 t).
struct W4Block {
  uint4 lo, hi;
  uint32_t s;  // scales (bf16 bits): row g in the low half, row g + 8 in the high half
  uint32_t z;  // zero points: row g in bits 0-7, row g + 8 in bits 8-15
};

// The rows a lane reads: codes of rows g and g + 8 at this lane's 16 bytes of block 0, scales and
// zero points of group 0, and the distance (in elements) between groups.
struct W4Rows {
  const char *lo, *hi;
  const uint16_t *slo, *shi;
  const uint8_t *zlo, *zhi;
  int64_t pitch;
  int last;  // last group
};

template <int GW, bool ASYM>
__device__ __forceinline__ void w4_load(W4Block& w, const W4Rows& r, int64_t b, int t) {
  w.lo = ldg_stream16(r.lo + b * W4_BLOCK_BYTES);
  w.hi = ldg_stream16(r.hi + b * W4_BLOCK_BYTES);
  // the padding of the last block has no group of its own: any finite scale will do there
  const int64_t g = min((int)(b * (4 / GW)) + t / GW, r.last) * r.pitch;
  w.s = (uint32_t)__ldg(r.slo + g) | ((uint32_t)__ldg(r.shi + g) << 16);
  if (ASYM) w.z = (uint32_t)__ldg(r.zlo + g) | ((uint32_t)__ldg(r.zhi + g) << 8);
}

// acc += scale * ((codes - zero) . x) for one block: NT column tiles of 8, S bf16 parts of x, GW
// 32-code words per scale.  xload(nt, s, w) gives the 8 values of x at 32 w + 8 t of column
// 8 nt + g, part s.  The integer part is summed by the tensor cores in binary32 over one group
// (codes - zero and x are exact bf16, their products exact), then scaled and added in binary32.
template <int NT, int S, int GW, bool ASYM, typename XLoad>
__device__ __forceinline__ void w4_mac(float (&acc)[NT][4], const W4Block& w, int lane, XLoad xload) {
  const uint32_t* lo = &w.lo.x;
  const uint32_t* hi = &w.hi.x;
  float tmp[NT][4];
  uint32_t zlo = bf16_128_plus(8) * 0x10001u, zhi = zlo;
  float slo, shi;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i % GW == 0) {
      uint32_t s = w.s, z = w.z;
      if (GW < 4) {  // the lane of this quad that loaded the group of word i
        s = __shfl_sync(0xffffffffu, w.s, (lane & ~3) | i);
        if (ASYM) z = __shfl_sync(0xffffffffu, w.z, (lane & ~3) | i);
      }
      slo = bf16lo(s);
      shi = bf16hi(s);
      if (ASYM) {
        zlo = bf16_128_plus(z & 0xffu) * 0x10001u;
        zhi = bf16_128_plus((z >> 8) & 0xffu) * 0x10001u;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) tmp[n][0] = tmp[n][1] = tmp[n][2] = tmp[n][3] = 0.0f;
    }
    uint32_t a[4], c[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      a[p] = w4_pair(lo[i], p, zlo);
      c[p] = w4_pair(hi[i], p, zhi);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const uint4 x = xload(n, s, i);
        mma_bf16(tmp[n], a[0], c[0], a[1], c[1], x.x, x.y);
        mma_bf16(tmp[n], a[2], c[2], a[3], c[3], x.z, x.w);
      }
    }
    if (i % GW == GW - 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[n][0] = __fmaf_rn(slo, tmp[n][0], acc[n][0]);
        acc[n][1] = __fmaf_rn(slo, tmp[n][1], acc[n][1]);
        acc[n][2] = __fmaf_rn(shi, tmp[n][2], acc[n][2]);
        acc[n][3] = __fmaf_rn(shi, tmp[n][3], acc[n][3]);
      }
    }
  }
}

// Lets the previous kernel of a programmatic launch finish before anything it wrote is read.  What
// that kernel may have written (activations, workspaces) is then read with plain loads: the
// non-coherent ones are for data that nothing writes while this kernel is resident.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void store_out(void* y, int64_t at, float v, bool bf16) {
  if (bf16) reinterpret_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else reinterpret_cast<float*>(y)[at] = v;
}

}  // namespace sqk
