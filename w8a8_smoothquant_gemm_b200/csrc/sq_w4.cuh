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

// Codes as mma operands.  OR-ing a code into the low significand bits of 128.0 (bf16, where the
// spacing is 1) makes 128 + code, and subtracting 128 + zero leaves code - zero, all exact: a
// shift, a logic operation and a packed subtraction for two codes.
__device__ __forceinline__ uint32_t w4_zero(uint32_t zero) { return zero * 0x10001u + 0x43004300u; }

// The eight codes of a word as four operand pairs (code 2p - zero, code 2p + 1 - zero).
__device__ __forceinline__ void w4_unpack(uint32_t (&a)[4], uint32_t word, uint32_t zero) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(word >> (4 * p)), "n"(0x000f000f), "n"(0x43004300));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(a[p]) : "r"(v), "r"(zero));
  }
}

// D += A B, 16 x 8 x 16, binary32 sums.  Lane (g, t) = (lane / 4, lane % 4) holds a0, a2 of row g
// and a1, a3 of row g + 8 for the k pairs (2t, 2t + 1) and (2t + 8, 2t + 9), b0 and b1 of column g
// for the same k, d0, d1 of row g, columns 2t, 2t + 1, and d2, d3 of row g + 8.  Which k the
// sixteen slots stand for is free as long as A and B agree.
// FIRST: D = A B.
template <bool FIRST>
__device__ __forceinline__ void w4_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if (FIRST)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// acc += scale * v for rows g (slo) and g + 8 (shi), two columns each.
__device__ __forceinline__ void w4_scale_add(float (&acc)[4], float slo, float shi, const float (&v)[4]) {
  const float2 a = __ffma2_rn(make_float2(slo, slo), make_float2(v[0], v[1]), make_float2(acc[0], acc[1]));
  const float2 b = __ffma2_rn(make_float2(shi, shi), make_float2(v[2], v[3]), make_float2(acc[2], acc[3]));
  acc[0] = a.x;
  acc[1] = a.y;
  acc[2] = b.x;
  acc[3] = b.y;
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

// ---------------------------------------------------------------------------- the weight stream
// A warp's share of the weights is a list of units: 16 rows x 256 codes (two blocks, 2 KB) with the
// scales and zero points of their groups.  They travel from memory to shared memory with
// asynchronous copies, DEPTH - 1 units ahead, in a ring that belongs to the warp alone: a lane reads
// back only codes that it copied itself, so no barrier is needed, only the copies' own group count
// (and a __syncwarp for the scales, which also says that the last unit's slot has been read and can
// be filled again).  Registers hold one block, whatever the depth.
//   What sets the depth is latency: at 6.5 TB/s and about 1 us under load an SM needs some 45 KB in
// flight; 16 warps with a unit each on its way and one at work have 32 to 64 KB, and asking the L2 for
// 256 bytes where the copies take 128 of a row fetches what the warp wants next (231 MB of weights: 47.8
// us with the hint, 55.7 without; DEPTH 3 is 3 % faster there and 10 % slower at 30 MB).  Once the bytes are
// there a block takes 58 to 61 clocks of an SM, against 46 in which HBM delivers it, with no unit at its limit:
// the unpacking (56 shifts and logic operations a block on the half-rate integer pipe) fills 28 of them, its 143
// instructions 36, the tensor pipe about 16; a scheduler's four warps lose the rest to a full math pipe, to each other
// and to loads.  So everything else in the loop is kept few: two blocks to a unit halve the control and address arithmetic.
constexpr int W4_UNIT = 2 * W4_BLOCK;

__host__ __device__ __forceinline__ int w4_units(int64_t K) { return (int)((K + W4_UNIT - 1) / W4_UNIT); }

struct W4Base {  // bases that a whole CTA shares, so that offsets are 32-bit
  const char* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  uint32_t row_bytes;  // of a row of codes
  uint32_t pitch;      // scales of a group
  int groups;          // groups of a row
};

template <int GW, bool ASYM>
struct W4Slot {  // of the ring: per block, codes of rows g and of rows g + 8; then scales, zero points
  static constexpr int GPB = 4 / GW, GPU = 2 * GPB;  // groups per block, per unit
  static constexpr int SCALES = 2048, ZEROS = SCALES + GPU * 32, BYTES = ZEROS + (ASYM ? GPU * 16 : 0);
};

// 16 bytes, or zeros where `bytes` is 0.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes = 16) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16_if(bool on, uint32_t dst, const void* src) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst),
               "l"(src), "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ void cp_async8_if(bool on, uint32_t dst, const void* src) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p cp.async.ca.shared.global [%0], [%1], 8;\n\t}" ::"r"(dst),
               "l"(src), "r"((uint32_t)on)
               : "memory");
}
// Loads from shared memory by address.  Volatile: they keep their place between the waits.
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t at, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(v) : "memory");
}
__device__ __forceinline__ void sts8(uint32_t at, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// What a lane copies of the next unit.
struct W4Cursor {
  const char *lo, *hi;  // its 16 bytes of rows g and g + 8
  uint32_t sc;          // element offset of the scales it copies
  uint32_t sc_end;      // and of those of the last group: the padding of a row's last block has no
                        // group of its own, and any finite scale will do there
};

// At unit u of the tile whose rows are row0 .. row0 + 7 and row8 .. row8 + 7 (relative to the base);
// rows past last_row repeat it.  ALIGNED: 8 rows' scales (zero points) are one 16-byte (8-byte) piece.
template <int GW, bool ASYM, bool ALIGNED>
__device__ __forceinline__ W4Cursor w4_place(const W4Base& base, uint32_t row0, uint32_t row8, uint32_t last_row, int u,
                                             int lane) {
  const uint32_t col = (uint32_t)u * (2 * W4_BLOCK_BYTES) + (lane % 4) * 16;
  W4Cursor c;
  c.lo = base.codes + (min(row0 + lane / 4, last_row) * base.row_bytes + col);
  c.hi = base.codes + (min(row8 + lane / 4, last_row) * base.row_bytes + col);
  // lane 2 q + h copies half h of group q (the last 8 rows stand in for a half that is past the
  // end); where that is no aligned piece, lane r < 16 fetches row r of every group
  uint32_t row, group = (uint32_t)u * W4Slot<GW, ASYM>::GPU;
  if (ALIGNED) {
    row = min(lane % 2 ? row8 : row0, last_row - 7);
    group += lane / 2;
  } else {
    row = min(lane < 8 ? row0 + lane : row8 + lane % 8, last_row);
  }
  c.sc = group * base.pitch + row;
  c.sc_end = (uint32_t)(base.groups - 1) * base.pitch + row;
  return c;
}

// Starts the copies of the cursor's unit, of which only the first block exists where `half`.
template <int GW, bool ASYM, bool ALIGNED>
__device__ __forceinline__ void w4_issue(uint32_t slot, const W4Base& base, W4Cursor& c, bool half, int lane) {
  using L = W4Slot<GW, ASYM>;
  const uint32_t second = half ? 0u : 16u;
  cp_async16(slot + lane * 16, c.lo);
  cp_async16(slot + 512 + lane * 16, c.hi);
  cp_async16(slot + 1024 + lane * 16, c.lo + W4_BLOCK_BYTES, second);
  cp_async16(slot + 1536 + lane * 16, c.hi + W4_BLOCK_BYTES, second);
  if (ALIGNED) {
    const uint32_t at = min(c.sc, c.sc_end);
    cp_async16_if(lane < 2 * L::GPU, slot + L::SCALES + lane * 16, base.scales + at);
    if (ASYM) cp_async8_if(lane < 2 * L::GPU, slot + L::ZEROS + lane * 8, base.zeros + at);
  } else if (lane < 16) {
#pragma unroll
    for (int q = 0; q < L::GPU; ++q) {
      const uint32_t at = min(c.sc + q * base.pitch, c.sc_end);
      sts16(slot + L::SCALES + q * 32 + lane * 2, __ldg(base.scales + at));
      if (ASYM) sts8(slot + L::ZEROS + q * 16 + lane, __ldg(base.zeros + at));
    }
  }
  c.lo += 2 * W4_BLOCK_BYTES;
  c.hi += 2 * W4_BLOCK_BYTES;
  c.sc += L::GPU * base.pitch;
}

// acc += scale * ((codes - zero) . x) for the unit in `slot`: NT column tiles of 8, S parts of x.
// xload(nt, s, w) gives the 8 values of x at 32 w + 8 t (w < 8) of column 8 nt + g, part s.  The
// integer part is summed by the tensor cores in binary32 over one group (codes - zero and x are
// exact operands, their products exact), then scaled and added in binary32.
template <int NT, int S, int GW, bool ASYM, int NTA, typename XLoad>
__device__ __forceinline__ void w4_mac(float (&acc)[NTA][4], uint32_t slot, int lane, XLoad xload) {
  static_assert(NT <= NTA, "column tiles beyond the sums");
  using L = W4Slot<GW, ASYM>;
  const uint32_t row = lane / 4;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint4 wl = lds128(slot + b * 1024 + lane * 16), wh = lds128(slot + b * 1024 + 512 + lane * 16);
    const uint32_t lo[4] = {wl.x, wl.y, wl.z, wl.w}, hi[4] = {wh.x, wh.y, wh.z, wh.w};
    float tmp[NT][4];
    uint32_t zlo = w4_zero(8), zhi = zlo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = b * L::GPB + i / GW;  // group within the unit
      if (i % GW == 0) {
        if (ASYM) {
          zlo = w4_zero(lds8(slot + L::ZEROS + q * 16 + row));
          zhi = w4_zero(lds8(slot + L::ZEROS + q * 16 + 8 + row));
        }
      }
      uint32_t a[4], c[4];
      w4_unpack(a, lo[i], zlo);
      w4_unpack(c, hi[i], zhi);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const uint4 x = xload(n, s, 4 * b + i);
          if (i % GW == 0 && s == 0) w4_mma<true>(tmp[n], a[0], c[0], a[1], c[1], x.x, x.y);
          else w4_mma<false>(tmp[n], a[0], c[0], a[1], c[1], x.x, x.y);
          w4_mma<false>(tmp[n], a[2], c[2], a[3], c[3], x.z, x.w);
        }
      }
      if (i % GW == GW - 1) {
        const float slo = bf16lo(lds16(slot + L::SCALES + q * 32 + row * 2));
        const float shi = bf16lo(lds16(slot + L::SCALES + q * 32 + 16 + row * 2));
#pragma unroll
        for (int n = 0; n < NT; ++n) w4_scale_add(acc[n], slo, shi, tmp[n]);
      }
    }
  }
}

// Few columns whose x has S parts need not take S products: the parts can be columns of one product
// beside each other.  Column g of 8 is then part g / C of column g % C (C = 4 for two parts, 2 for
// three), and the sums of a column's parts are added at the end.
__host__ __device__ constexpr int w4_fold_columns(int S) { return S == 2 ? 4 : S == 3 ? 2 : 0; }
template <int S>
__device__ __forceinline__ int2 w4_part_column(int g) {
  constexpr int C = S == 2 ? 4 : 2;
  return make_int2(g % C, min(g / C, S - 1));
}
// Adds the parts; the lanes of columns below C have the sums.
template <int S>
__device__ __forceinline__ void w4_fold(float (&acc)[4], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (S == 2) {
      acc[i] = __fadd_rn(acc[i], __shfl_xor_sync(0xffffffffu, acc[i], 2));
    } else {
      const float b = __shfl_sync(0xffffffffu, acc[i], (lane & ~3) | 1), c = __shfl_sync(0xffffffffu, acc[i], (lane & ~3) | 2);
      acc[i] = __fadd_rn(acc[i], __fadd_rn(b, c));
    }
  }
}

// ---------------------------------------------------------------------------- runs and cells
// A CTA's line of units (tile after tile) is cut into equal runs, one a warp.  A warp's sum over its
// part of a tile goes to a cell of its own; the cells of a tile are then added in the order of the
// warps.  Cells lie in the order of the line, so there is at most one more per run than tiles.
//   A cell of NT column tiles is 16 rows x 8 NT columns; a lane's pairs of columns leave in one store
// each, and half a warp's cover the banks once.
__host__ __device__ constexpr int w4_cell_floats(int NT) { return 128 * NT; }

template <int NT, int NTA>
__device__ __forceinline__ void w4_put_cell(float* cell, const float (&acc)[NTA][4], int lane) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float* q = cell + (lane / 4) * (8 * NTA) + 8 * n + 2 * (lane % 4);
    *reinterpret_cast<float2*>(q) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(q + 8 * (8 * NTA)) = make_float2(acc[n][2], acc[n][3]);
  }
}

template <int WARPS>
struct W4Runs {  // in shared memory
  int first_cell[WARPS], first_tile[WARPS], cells;
};

// n / d for n >= 0 and a quotient below 2^22, with inv = 1 / d: (float)n, inv and the product are each off by at
// most 2^-24 of themselves, so the product by less than one, and its integer part by one at most.  (Quotients
// here are tokens, rows, tiles or runs: thousands.)
__device__ __forceinline__ int w4_div(int n, int d, float inv) {
  const int q = (int)__fmul_rn((float)n, inv), r = n - q * d;
  return q + (r >= d) - (r < 0);
}

// Where run w of a line begins.
template <int WARPS>
__device__ __forceinline__ int w4_cut(int line, int w) {
  return (int)((uint32_t)(line * w) / (uint32_t)WARPS);
}

struct W4Run {  // this warp's
  int units;    // of the line
  int tile, b;  // where it begins
  int cell;     // its first cell
};

// Fills `runs` (warp 0; a __syncthreads must follow before it is read) and returns this warp's run.
template <int WARPS>
__device__ __forceinline__ W4Run w4_runs(W4Runs<WARPS>& runs, int line, int per_tile, int warp, int lane) {
  static_assert(WARPS <= 32, "a lane per run");
  const float inv = __frcp_rn((float)per_tile);
  const int a0 = w4_cut<WARPS>(line, lane), a1 = lane < WARPS ? w4_cut<WARPS>(line, lane + 1) : a0;
  const int at = w4_div(a0, per_tile, inv), n = a1 > a0 ? w4_div(a1 - 1, per_tile, inv) - at + 1 : 0;
  int sum = n;
#pragma unroll
  for (int o = 1; o < WARPS; o *= 2) {
    const int other = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += other;
  }
  if (warp == 0 && lane < WARPS) {
    runs.first_cell[lane] = sum - n;
    runs.first_tile[lane] = at;
    if (lane == WARPS - 1) runs.cells = sum;
  }
  W4Run r;
  r.units = __shfl_sync(0xffffffffu, a1 - a0, warp);
  r.tile = __shfl_sync(0xffffffffu, at, warp);
  r.b = __shfl_sync(0xffffffffu, a0 - at * per_tile, warp);
  r.cell = __shfl_sync(0xffffffffu, sum - n, warp);
  return r;
}

// The first cell of tile `ti` (of n_tiles; n_tiles itself: the number of cells); inv = 1 / line.
template <int WARPS>
__device__ __forceinline__ int w4_first_cell(const W4Runs<WARPS>& runs, int ti, int n_tiles, int line, float inv,
                                             int per_tile) {
  if (ti >= n_tiles) return runs.cells;
  // the run that holds the tile's first unit: w4_cut(w) <= l < w4_cut(w + 1)
  const int w = w4_div(WARPS * (ti * per_tile + 1) - 1, line, inv);
  return runs.first_cell[w] + ti - runs.first_tile[w];
}

// part i of n equal parts of a count whose quotient and remainder by n are q and r: where it begins
__device__ __forceinline__ int64_t w4_part(int64_t i, int64_t q, int r) { return i * q + min(i, (int64_t)r); }

// Lets the previous kernel of a programmatic launch finish before anything it wrote is read.  What
// that kernel may have written (activations, workspaces) is then read with plain loads: the
// non-coherent ones are for data that nothing writes while this kernel is resident.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void store_out(void* y, int64_t at, float v, bool bf16) {
  if (bf16) reinterpret_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else reinterpret_cast<float*>(y)[at] = v;
}

}  // namespace sqk

namespace sqh {
// Lets a kernel of the current device take `bytes` of dynamic shared memory (set once per kernel and device:
// the call would cost a launch's host time a fair part).
cudaError_t allow_shared_memory(const void* kern, int64_t bytes);
}  // namespace sqh
