// sq_w4_fold.cu -- the offline side of the 4-bit weight format: smoothing folded in, group scales,
// codes; and the values that codes stand for.
//
// Quantiser ("量化：只压权重，与训练后量化（PTQ）": group-wise round to nearest; "SmoothQuant大模型
// 平滑量化技术", Python demo: max / largest code, round, clip), every operation one binary32 rounding:
//   W' = s_j W[j, n]
//   symmetric:        scale = bf16(max|W'| * RN(1/7)),         code = 8 + clamp(rne(W' / scale), -7, 7)
//   with zero points: lo = min(0, min W'), hi = max(0, max W'),
//                     scale = bf16((hi - lo) * RN(1/15)), zero = clamp(rne(-lo / scale), 0, 15),
//                     code = clamp(rne(W' / scale) + zero, 0, 15)
// A zero scale gives codes equal to the zero point.  The scale is rounded to bf16 before the codes
// are taken, so the rounding costs no accuracy beyond the grid's own: codes are nearest on the grid
// that is stored.  The product with the rounded reciprocal, one multiplication, is within 2^-23 of the quotient by 7
// or 15; for 70 (symmetric) and 104 of 2^23 significands it lies on the other side of the middle of two bf16
// numbers and so rounds to the other one, which is as near to the quotient, to 2^-23 of it.
//
// Bound: one read of W and one write of the codes.  A block takes 256 input channels (two blocks of
// the format) of 64 output channels; each thread two output channels and one 32-code word column,
// so a group's extremes are in registers (group 32) or meet through shared memory once, and the two
// channels' quotients run on packed binary32 pairs (one reciprocal a group, Markstein's correction).
// Measured (4096 x 28672 bf16, group 64, zero points): 85 us, 3.5 TB/s.  No unit is at its limit (DRAM 39 %, integer
// pipe 54 %, 2.5 of 4 instructions a clock): a block's loads, arithmetic and stores follow each other, and three
// blocks an SM cover each other's only in part.  The values: 52 us, 5.7 TB/s of codes read and values written.
#include <algorithm>

#include "sq_w4.cuh"

namespace sqk {

constexpr int W4F_COLS = 64;        // output channels per block
constexpr int W4F_THREADS = 256;    // 32 column pairs x 2 format blocks x 4 word columns
constexpr int W4F_PITCH = 128 + 16; // bytes per staged code row (16-byte aligned, spreads the banks)

template <bool BF16, bool ASYM>
__global__ void __launch_bounds__(W4F_THREADS, BF16 ? 3 : 2)
w4_fold_kernel(const char* __restrict__ W, int64_t K, int64_t N, int64_t ld_bytes, const float* __restrict__ s,
               const float* __restrict__ gamma, const float* __restrict__ beta, int gw, int groups, int64_t row_bytes,
               char* __restrict__ wq, uint16_t* __restrict__ sg, uint8_t* __restrict__ zp, float* __restrict__ gamma_f,
               float* __restrict__ beta_f) {
  wait_for_previous_kernel();
  __shared__ float2 ext[2][8][W4F_COLS / 2];  // extremes of each 32-code column, by column pair
  __shared__ __align__(16) float factor[W4_UNIT];
  __shared__ __align__(16) char codes[W4F_COLS * W4F_PITCH];
  const int tid = threadIdx.x, pair = tid % 32, col = tid / 32, w = col % 4;
  const int64_t u0 = (int64_t)blockIdx.y * W4_UNIT, n0 = (int64_t)blockIdx.x * W4F_COLS, n = n0 + 2 * pair;
  const int64_t k0 = u0 + 32 * col;
  const int rows = n < N ? (int)max((int64_t)0, min((int64_t)32, K - k0)) : 0;  // rows are whole 16-byte
  const char* src = W + k0 * ld_bytes + n * (BF16 ? 2 : 4);                     // vectors: N is even
  uint32_t raw[BF16 ? 32 : 64];
  auto read = [&](int i, const char* at) {
    if (BF16) {
      raw[i] = __ldg(reinterpret_cast<const uint32_t*>(at));
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
      raw[BF16 ? 0 : 2 * i] = v.x;
      raw[BF16 ? 0 : 2 * i + 1] = v.y;
    }
  };
  if (rows == 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i, src += ld_bytes) read(i, src);
  } else {
#pragma unroll
    for (int i = 0; i < (BF16 ? 32 : 64); ++i) raw[i] = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i, src += ld_bytes)
      if (i < rows) read(i, src);
  }
  {
    const int64_t k = u0 + tid;
    const float sj = s && k < K ? s[k] : 1.0f;
    factor[tid] = sj;
    if (blockIdx.x == 0 && k < K) {  // LayerNorm folding, one channel per thread
      if (gamma && gamma_f) gamma_f[k] = __fdiv_rn(gamma[k], sj);
      if (beta && beta_f) beta_f[k] = __fdiv_rn(beta[k], sj);
    }
  }
  __syncthreads();
  // W' of row i (bf16: from the bits each time, which keeps the registers at half; the product is one
  // operation for two channels)
  auto value = [&](int i, float f) {
    const float2 a = BF16 ? make_float2(bf16lo(raw[i]), bf16hi(raw[i]))
                          : make_float2(__uint_as_float(raw[BF16 ? 0 : 2 * i]), __uint_as_float(raw[BF16 ? 0 : 2 * i + 1]));
    return __fmul2_rn(make_float2(f, f), a);
  };
  float2 top = make_float2(0.0f, 0.0f), bot = top;  // for symmetric scales, top is the largest magnitude
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(factor + 32 * col + i);
    const float2 v[4] = {value(i, f.x), value(i + 1, f.y), value(i + 2, f.z), value(i + 3, f.w)};
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const float2 p = v[j], q = v[j + 1];
      if (ASYM) {
        top = make_float2(fmax3(top.x, p.x, q.x), fmax3(top.y, p.y, q.y));
        bot = make_float2(-fmax3(-bot.x, -p.x, -q.x), -fmax3(-bot.y, -p.y, -q.y));
      } else {
        top = make_float2(fmax3(top.x, fabsf(p.x), fabsf(q.x)), fmax3(top.y, fabsf(p.y), fabsf(q.y)));
      }
    }
  }
  if (gw > 1) {
    ext[0][col][pair] = top;
    if (ASYM) ext[1][col][pair] = bot;
    __syncthreads();
    const int g0 = col / gw * gw;  // first word column of this thread's group
    for (int q = g0; q < g0 + gw; ++q) {
      const float2 e = ext[0][q][pair];
      top = make_float2(fmaxf(top.x, e.x), fmaxf(top.y, e.y));
      if (ASYM) {
        const float2 d = ext[1][q][pair];
        bot = make_float2(fminf(bot.x, d.x), fminf(bot.y, d.y));
      }
    }
  }
  const float per = ASYM ? 1.0f / 15.0f : 1.0f / 7.0f;
  const float2 range = ASYM ? make_float2(__fmul_rn(__fsub_rn(top.x, bot.x), per), __fmul_rn(__fsub_rn(top.y, bot.y), per))
                            : make_float2(__fmul_rn(top.x, per), __fmul_rn(top.y, per));
  const __nv_bfloat16 sb[2] = {__float2bfloat16_rn(range.x), __float2bfloat16_rn(range.y)};
  const float2 scale = make_float2(__bfloat162float(sb[0]), __bfloat162float(sb[1]));
  float2 zero = make_float2(8.0f, 8.0f);
  if (ASYM) {
    zero.x = scale.x == 0.0f ? 0.0f : fminf(rintf(__fdiv_rn(-bot.x, scale.x)), 15.0f);
    zero.y = scale.y == 0.0f ? 0.0f : fminf(rintf(__fdiv_rn(-bot.y, scale.y)), 15.0f);
  }
  const SharedDivisor dx(scale.x), dy(scale.y);
  uint32_t wx[4], wy[4];
  if (dx.fast && dy.fast) {
    // Adding 1.5 * 2^23 rounds the quotient q to an integer, ties to even, and leaves it in the low bits
    // of the sum (0x4b400000 + q).  Shifted sums of eight are a word of codes after one correction: their
    // exponents and leading bits (the larger shifts push them out), and the zero point in every nibble.
    // q lies within 1 + 2^-8 (the scale's rounding to bf16) of the codes' range: below 7.03 of a symmetric
    // grid's 7.5, and never below rne(lo / scale) = -zero; only the upper end of a grid with a zero point
    // can need the clip.
    constexpr uint32_t excess = 0x4b400000u + (0x4b400000u << 4) + (0x4b400000u << 8);
    const uint32_t fixx = (uint32_t)(int)zero.x * 0x11111111u - excess, fixy = (uint32_t)(int)zero.y * 0x11111111u - excess;
    const float2 rc = make_float2(dx.y, dy.y), nb = make_float2(-dx.b, -dy.b), magic = make_float2(12582912.0f, 12582912.0f);
    const float2 most = make_float2(12582927.0f - zero.x, 12582927.0f - zero.y);
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      uint32_t ax = 0u, ay = 0u;
      const float4 fa = *reinterpret_cast<const float4*>(factor + 32 * col + i);
      const float4 fb = *reinterpret_cast<const float4*>(factor + 32 * col + i + 4);
      const float f[8] = {fa.x, fa.y, fa.z, fa.w, fb.x, fb.y, fb.z, fb.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float2 t = __fadd2_rn(markstein2(value(i + j, f[j]), rc, nb), magic);
        if (ASYM) t = make_float2(fminf(t.x, most.x), fminf(t.y, most.y));
        const int sh = 4 * (j / 2) + 16 * (j % 2);
        ax += __float_as_uint(t.x) << sh;
        ay += __float_as_uint(t.y) << sh;
      }
      wx[i / 8] = ax + fixx;
      wy[i / 8] = ay + fixy;
    }
  } else {  // rare: a scale outside the fast range (its rounding to bf16 may then be coarse)
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      uint32_t ax = 0u, ay = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int sh = 4 * (j / 2) + 16 * (j % 2);
        const float2 v = value(i + j, factor[32 * col + i + j]);
        const float qx = rintf(dx.div(v.x)), qy = rintf(dy.div(v.y));
        const float cx = ASYM ? fminf(fmaxf(__fadd_rn(qx, zero.x), 0.0f), 15.0f) : fminf(fmaxf(qx, -7.0f), 7.0f) + 8.0f;
        const float cy = ASYM ? fminf(fmaxf(__fadd_rn(qy, zero.y), 0.0f), 15.0f) : fminf(fmaxf(qy, -7.0f), 7.0f) + 8.0f;
        ax |= (uint32_t)(int)cx << sh;
        ay |= (uint32_t)(int)cy << sh;
      }
      wx[i / 8] = ax;
      wy[i / 8] = ay;
    }
  }
  const int64_t gidx = (blockIdx.y * 8 + col) / gw;
  if (col % gw == 0 && gidx < groups && rows > 0) {
    reinterpret_cast<uint16_t*>(sg)[gidx * N + n] = __bfloat16_as_ushort(sb[0]);
    reinterpret_cast<uint16_t*>(sg)[gidx * N + n + 1] = __bfloat16_as_ushort(sb[1]);
    if (ASYM) {
      zp[gidx * N + n] = (uint8_t)(int)zero.x;
      zp[gidx * N + n + 1] = (uint8_t)(int)zero.y;
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const bool there = 8 * t < rows;  // channels come in sixteens; the padding of the last block is 0
    char* at = codes + 2 * pair * W4F_PITCH + (col / 4) * W4_BLOCK_BYTES + 16 * t + 4 * w;
    *reinterpret_cast<uint32_t*>(at) = there ? wx[t] : 0u;
    *reinterpret_cast<uint32_t*>(at + W4F_PITCH) = there ? wy[t] : 0u;
  }
  __syncthreads();
  const int64_t b0 = (int64_t)blockIdx.y * (2 * W4_BLOCK_BYTES);
#pragma unroll
  for (int i = tid; i < W4F_COLS * 8; i += W4F_THREADS) {
    const int row = i / 8, t = i % 8;
    if (n0 + row < N && b0 + 16 * t < row_bytes)
      *reinterpret_cast<uint4*>(wq + (n0 + row) * row_bytes + b0 + 16 * t) =
          *reinterpret_cast<const uint4*>(codes + row * W4F_PITCH + 16 * t);
  }
}

constexpr int W4D_THREADS = 128, W4D_ROWS = W4D_THREADS / 32 * 4;

// Values: (code - zero) * scale, at most 12 significant bits (exact in binary32), rounded once for
// bf16.  A thread takes 16 bytes of codes (four runs of 8 consecutive k) of four rows, so that four
// loads are on their way and the rows' scales come together; a warp takes 32 pieces of each row, so both
// sides are whole lines.  Bound by the values' bytes.
template <bool BF16>
__global__ void __launch_bounds__(W4D_THREADS, 6)
w4_dequant_kernel(const char* __restrict__ wq, const uint16_t* __restrict__ sg, const uint8_t* __restrict__ zp, int K,
                  int64_t N, int gw, int row_bytes, char* __restrict__ y, int64_t ld_bytes, bool together) {
  wait_for_previous_kernel();
  const int piece = blockIdx.x * 32 + threadIdx.x % 32, b = piece / 4, t = piece % 4;
  if (piece * 16 >= row_bytes) return;
  for (int64_t n0 = (int64_t)blockIdx.y * W4D_ROWS + threadIdx.x / 32 * 4; n0 < N; n0 += (int64_t)gridDim.y * W4D_ROWS) {
    uint4 c[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
      c[r] = n0 + r < N ? ldg_stream16(wq + (n0 + r) * row_bytes + piece * 16) : make_uint4(0u, 0u, 0u, 0u);
    uint2 s = make_uint2(0u, 0u);
    uint32_t z = 0x08080808u;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int k = b * W4_BLOCK + 32 * w + 8 * t;
      if (k >= K) continue;
      if (w % gw == 0) {  // the four rows' scales and zero points of this group
        const int64_t g = (int64_t)(b * (4 / gw) + w / gw) * N + n0;
        if (together) {
          s = __ldg(reinterpret_cast<const uint2*>(sg + g));
          if (zp) z = __ldg(reinterpret_cast<const uint32_t*>(zp + g));
        } else {
          uint32_t v[4] = {0u, 0u, 0u, 0u}, q[4] = {8u, 8u, 8u, 8u};
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n0 + r < N) {
              v[r] = __ldg(sg + g + r);
              if (zp) q[r] = __ldg(zp + g + r);
            }
          s = make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
          z = q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (n0 + r >= N) continue;
        const uint32_t word = w == 0 ? c[r].x : w == 1 ? c[r].y : w == 2 ? c[r].z : c[r].w;
        const float scale = r % 2 ? bf16hi(r < 2 ? s.x : s.y) : bf16lo(r < 2 ? s.x : s.y);
        const float zero = __uint_as_float(0x4b000000u | ((z >> (8 * r)) & 0xffu));  // 2^23 + zero
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t code = (word >> (4 * (e / 2) + 16 * (e % 2))) & 15u;
          f[e] = __fmul_rn(__fsub_rn(__uint_as_float(0x4b000000u | code), zero), scale);
        }
        char* out = y + (n0 + r) * ld_bytes + (int64_t)k * (BF16 ? 2 : 4);
        if (BF16) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
            o[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          __stcs(reinterpret_cast<uint4*>(out), make_uint4(o[0], o[1], o[2], o[3]));
        } else {
          __stcs(reinterpret_cast<float4*>(out), make_float4(f[0], f[1], f[2], f[3]));
          __stcs(reinterpret_cast<float4*>(out + 16), make_float4(f[4], f[5], f[6], f[7]));
        }
      }
    }
  }
}

}  // namespace sqk

namespace sqh {
namespace {

// A launch that may begin before the previous kernel on the stream is done (the kernels wait for it), which
// also costs the host less than one without the attribute.
struct Dependent {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  Dependent(dim3 grid, unsigned threads, cudaStream_t st) {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
};

}  // namespace

cudaError_t launch_w4_fold(const void* W, bool bf16, int64_t K, int64_t N, int64_t ldw, const float* s,
                           const float* gamma, const float* beta, int group, uint8_t* wq, uint16_t* sg, uint8_t* zp,
                           float* gamma_f, float* beta_f, cudaStream_t st) {
  const int64_t row_bytes = sqk::w4_blocks(K) * sqk::W4_BLOCK_BYTES, ldb = ldw * (bf16 ? 2 : 4);
  const int gw = group / 32, groups = (int)((K + group - 1) / group);
  const dim3 grid((unsigned)((N + sqk::W4F_COLS - 1) / sqk::W4F_COLS), (unsigned)sqk::w4_units(K));
  Dependent launch(grid, sqk::W4F_THREADS, st);
  auto go = [&](auto kern) {
    return cudaLaunchKernelEx(&launch.cfg, kern, (const char*)W, K, N, ldb, s, gamma, beta, gw, groups, row_bytes,
                              (char*)wq, sg, zp, gamma_f, beta_f);
  };
  if (bf16) return zp ? go(sqk::w4_fold_kernel<true, true>) : go(sqk::w4_fold_kernel<true, false>);
  return zp ? go(sqk::w4_fold_kernel<false, true>) : go(sqk::w4_fold_kernel<false, false>);
}

cudaError_t launch_w4_dequant(const uint8_t* wq, const uint16_t* sg, const uint8_t* zp, int64_t K, int64_t N, int group,
                              void* y, bool y_bf16, int64_t ldy, cudaStream_t st) {
  const int row_bytes = (int)(sqk::w4_blocks(K) * sqk::W4_BLOCK_BYTES);
  const dim3 grid((unsigned)((row_bytes / 16 + 31) / 32), (unsigned)std::min<int64_t>((N + sqk::W4D_ROWS - 1) / sqk::W4D_ROWS, 65535));
  const bool together = N % 4 == 0 && (uintptr_t)sg % 8 == 0 && (uintptr_t)zp % 4 == 0;
  Dependent launch(grid, sqk::W4D_THREADS, st);
  auto go = [&](auto kern) {
    return cudaLaunchKernelEx(&launch.cfg, kern, (const char*)wq, sg, zp, (int)K, N, group / 32, row_bytes, (char*)y,
                              ldy * (y_bf16 ? 2 : 4), together);
  };
  return y_bf16 ? go(sqk::w4_dequant_kernel<true>) : go(sqk::w4_dequant_kernel<false>);
}

}  // namespace sqh
