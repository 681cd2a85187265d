// sq_w4_fold.cu -- the offline side of the 4-bit weight format: smoothing folded in, group scales,
// codes; and the values that codes stand for.
//
// Quantiser ("量化：只压权重，与训练后量化（PTQ）": group-wise round to nearest; "SmoothQuant大模型
// 平滑量化技术", Python demo: max / largest code, round, clip), every operation one binary32 rounding:
//   W' = s_j W[j, n]
//   symmetric:        scale = bf16(max|W'| / 7),               code = 8 + clamp(rne(W' / scale), -7, 7)
//   with zero points: lo = min(0, min W'), hi = max(0, max W'),
//                     scale = bf16((hi - lo) / 15), zero = clamp(rne(-lo / scale), 0, 15),
//                     code = clamp(rne(W' / scale) + zero, 0, 15)
// A zero scale gives codes equal to the zero point.  The scale is rounded to bf16 before the codes
// are taken, so the rounding costs no accuracy beyond the grid's own: codes are nearest on the grid
// that is stored.
//
// Bound: one read of W and one write of the codes.  A block takes 128 input channels (one block of
// the format) of 64 output channels; each thread two output channels and one 32-code word column,
// so a group's extremes are in registers (group 32) or meet through shared memory once.
#include <algorithm>

#include "sq_w4.cuh"

namespace sqk {

constexpr int W4F_COLS = 64;       // output channels per block
constexpr int W4F_THREADS = 128;   // 32 column pairs x 4 word columns
constexpr int W4F_PITCH = 64 + 16; // bytes per staged code row (16-byte aligned, spreads the banks)

template <bool BF16, bool ASYM>
__global__ void __launch_bounds__(W4F_THREADS)
w4_fold_kernel(const char* __restrict__ W, int64_t K, int64_t N, int64_t ld_bytes, const float* __restrict__ s,
               const float* __restrict__ gamma, const float* __restrict__ beta, int gw, int groups, int64_t row_bytes,
               char* __restrict__ wq, uint16_t* __restrict__ sg, uint8_t* __restrict__ zp, float* __restrict__ gamma_f,
               float* __restrict__ beta_f) {
  __shared__ float ext[2][4][W4F_COLS];  // extremes of each 32-code column
  __shared__ __align__(16) char codes[W4F_COLS * W4F_PITCH];
  const int tid = threadIdx.x, pair = tid % 32, w = tid / 32;
  const int64_t b = blockIdx.y, n0 = (int64_t)blockIdx.x * W4F_COLS, n = n0 + 2 * pair;
  const int64_t k0 = b * W4_BLOCK + 32 * w;
  if (blockIdx.x == 0) {  // LayerNorm folding, one channel per thread
    const int64_t k = b * W4_BLOCK + tid;
    if (k < K) {
      const float sj = s ? s[k] : 1.0f;
      if (gamma && gamma_f) gamma_f[k] = __fdiv_rn(gamma[k], sj);
      if (beta && beta_f) beta_f[k] = __fdiv_rn(beta[k], sj);
    }
  }
  float v[2][32];
  float top[2] = {0.0f, 0.0f}, bot[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[0][i] = v[1][i] = 0.0f;
    if (k0 + i < K && n < N) {  // rows are whole 16-byte vectors, so a pair never straddles the end
      const float sj = s ? __ldg(s + k0 + i) : 1.0f;
      if (BF16) {
        const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(W + (k0 + i) * ld_bytes + n * 2));
        v[0][i] = __fmul_rn(sj, bf16lo(u));
        v[1][i] = __fmul_rn(sj, bf16hi(u));
      } else {
        const float2 u = __ldg(reinterpret_cast<const float2*>(W + (k0 + i) * ld_bytes + n * 4));
        v[0][i] = __fmul_rn(sj, u.x);
        v[1][i] = __fmul_rn(sj, u.y);
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      top[c] = fmaxf(top[c], v[c][i]);
      bot[c] = fminf(bot[c], v[c][i]);
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    ext[0][w][2 * pair + c] = top[c];
    ext[1][w][2 * pair + c] = bot[c];
  }
  __syncthreads();
  const int g0 = w / gw * gw;  // first word column of this thread's group
  const int64_t gidx = b * (4 / gw) + w / gw;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    for (int q = g0; q < g0 + gw; ++q) {
      top[c] = fmaxf(top[c], ext[0][q][2 * pair + c]);
      bot[c] = fminf(bot[c], ext[1][q][2 * pair + c]);
    }
    float scale = ASYM ? __fdiv_rn(__fsub_rn(top[c], bot[c]), 15.0f) : __fdiv_rn(fmaxf(top[c], -bot[c]), 7.0f);
    const __nv_bfloat16 sb = __float2bfloat16_rn(scale);
    scale = __bfloat162float(sb);
    float zero = 8.0f;
    if (ASYM) zero = scale == 0.0f ? 0.0f : fminf(fmaxf(rintf(__fdiv_rn(-bot[c], scale)), 0.0f), 15.0f);
    const SharedDivisor d(scale);
    uint32_t word[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float q = rintf(d.div(v[c][i]));
      const float code = ASYM ? fminf(fmaxf(__fadd_rn(q, zero), 0.0f), 15.0f) : __fadd_rn(fminf(fmaxf(q, -7.0f), 7.0f), 8.0f);
      const uint32_t u = k0 + i < K ? (uint32_t)(int)code : 0u;  // padding of the last block
      word[i / 8] |= u << (4 * ((i % 8) / 2) + 16 * (i % 2));
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
      *reinterpret_cast<uint32_t*>(codes + (2 * pair + c) * W4F_PITCH + 16 * t + 4 * w) = word[t];
    if (w == g0 && gidx < groups && n + c < N) {
      sg[gidx * N + n + c] = __bfloat16_as_ushort(sb);
      if (ASYM) zp[gidx * N + n + c] = (uint8_t)(int)zero;
    }
  }
  __syncthreads();
  for (int i = tid; i < W4F_COLS * 4; i += W4F_THREADS) {
    const int row = i / 4, t = i % 4;
    if (n0 + row < N)
      *reinterpret_cast<uint4*>(wq + (n0 + row) * row_bytes + b * W4_BLOCK_BYTES + 16 * t) =
          *reinterpret_cast<const uint4*>(codes + row * W4F_PITCH + 16 * t);
  }
}

// Values: (code - zero) * scale, at most 12 significant bits (exact in binary32), rounded once for
// bf16.  One thread per 16 bytes of codes: four runs of 8 consecutive k.
template <bool BF16>
__global__ void __launch_bounds__(256)
w4_dequant_kernel(const char* __restrict__ wq, const uint16_t* __restrict__ sg, const uint8_t* __restrict__ zp,
                  int64_t K, int64_t N, int gw, int groups, int64_t row_bytes, char* __restrict__ y, int64_t ld_bytes) {
  const int64_t pieces = row_bytes / 16;
  const int64_t total = pieces * N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t n = i / pieces, piece = i % pieces, b = piece / 4;
    const int t = (int)(piece % 4);
    const uint4 c = ldg_stream16(wq + n * row_bytes + piece * 16);
    const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int64_t k = b * W4_BLOCK + 32 * w + 8 * t;
      if (k >= K) continue;
      const int64_t g = (b * (4 / gw) + w / gw) * N + n;
      const float scale = __uint_as_float((uint32_t)__ldg(sg + g) << 16);
      const int zero = zp ? (int)__ldg(zp + g) : 8;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int code = (int)((word[w] >> (4 * (e / 2) + 16 * (e % 2))) & 15u);
        f[e] = __fmul_rn((float)(code - zero), scale);
      }
      char* out = y + n * ld_bytes + k * (BF16 ? 2 : 4);
      if (BF16) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
          o[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        *reinterpret_cast<float4*>(out) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(out + 16) = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
  }
}

}  // namespace sqk

namespace sqh {

cudaError_t launch_w4_fold(const void* W, bool bf16, int64_t K, int64_t N, int64_t ldw, const float* s,
                           const float* gamma, const float* beta, int group, uint8_t* wq, uint16_t* sg, uint8_t* zp,
                           float* gamma_f, float* beta_f, cudaStream_t st) {
  const int64_t nb = sqk::w4_blocks(K), row_bytes = nb * sqk::W4_BLOCK_BYTES, ldb = ldw * (bf16 ? 2 : 4);
  const int gw = group / 32, groups = (int)((K + group - 1) / group);
  const dim3 grid((unsigned)((N + sqk::W4F_COLS - 1) / sqk::W4F_COLS), (unsigned)nb);
  auto go = [&](auto kern) {
    kern<<<grid, sqk::W4F_THREADS, 0, st>>>((const char*)W, K, N, ldb, s, gamma, beta, gw, groups, row_bytes,
                                            (char*)wq, sg, zp, gamma_f, beta_f);
  };
  if (bf16) zp ? go(sqk::w4_fold_kernel<true, true>) : go(sqk::w4_fold_kernel<true, false>);
  else zp ? go(sqk::w4_fold_kernel<false, true>) : go(sqk::w4_fold_kernel<false, false>);
  return cudaGetLastError();
}

cudaError_t launch_w4_dequant(const uint8_t* wq, const uint16_t* sg, const uint8_t* zp, int64_t K, int64_t N, int group,
                              void* y, bool y_bf16, int64_t ldy, cudaStream_t st) {
  const int64_t row_bytes = sqk::w4_blocks(K) * sqk::W4_BLOCK_BYTES, total = row_bytes / 16 * N;
  const int groups = (int)((K + group - 1) / group);
  const unsigned grid = (unsigned)std::min<int64_t>((total + 255) / 256, (int64_t)num_sms() * 64);
  if (y_bf16)
    sqk::w4_dequant_kernel<true><<<grid, 256, 0, st>>>((const char*)wq, sg, zp, K, N, group / 32, groups, row_bytes,
                                                       (char*)y, ldy * 2);
  else
    sqk::w4_dequant_kernel<false><<<grid, 256, 0, st>>>((const char*)wq, sg, zp, K, N, group / 32, groups, row_bytes,
                                                        (char*)y, ldy * 4);
  return cudaGetLastError();
}

}  // namespace sqh
