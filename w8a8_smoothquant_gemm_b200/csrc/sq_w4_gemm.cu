// sq_w4_gemm.cu -- x [M, K] times 4-bit weights [N, K] with group scales, for a few tokens.
//
// y[m, n] = sum_g scale[g, n] * sum_{k in g} (code[n, k] - zero[g, n]) * x[m, k]
//
// Bound: the weight codes' K N / 2 bytes from HBM; at a few tokens every other term is small.  So
// the codes go from memory to registers once, with 16-byte loads kept several blocks ahead, and
// are turned into bf16 operands there (exact small integers).  The products run on mma.sync: its
// operands are registers, which is where the codes are unpacked, and at M <= 8 one 16 x 8 x 16
// step consumes 256 weights, so the tensor pipe is far from its limit (tcgen05 would want the
// unpacked operand written to shared memory first, four times the bytes of the codes).
//
// A CTA owns 16 WR rows of weights over its K range; its 8 warps are WR row tiles x 8 / WR K
// slices (interleaved blocks, so a CTA reads whole lines).  x is staged in shared memory once as
// bf16 parts (one for bf16, three for binary32, which together are x exactly).  Partial sums meet
// in shared memory and, when K is cut over a cluster because there are few row tiles, in
// distributed shared memory, always in the same order: no atomics, no workspace.
#include <algorithm>

#include "sq_w4.cuh"

namespace sqk {

constexpr int W4G_THREADS = 256;
constexpr int W4G_DEPTH = 4;  // blocks a warp keeps in flight

struct W4GemmParams {
  const char* x;
  int64_t ldx_bytes;
  int M, K;
  const char* wq;
  const uint16_t* sg;
  const uint8_t* zp;
  int64_t N, row_bytes;
  int groups;
  void* y;
  int64_t ldy;
  int y_bf16;
  int C;      // CTAs of the cluster, over K
  int chunk;  // blocks of x staged at a time
};

template <int NT, int S, int GW, bool ASYM, int WR>
__global__ void __launch_bounds__(W4G_THREADS) w4_gemm_kernel(const W4GemmParams p) {
  constexpr int WK = 8 / WR, ROWS = 16 * WR, RP = ROWS + 4;  // RP: padded row count, conflict-free partial sums
  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int wr = warp % WR, wk = warp / WR;
  const int rank = blockIdx.x % p.C;
  const int64_t row0 = (int64_t)(blockIdx.x / p.C) * ROWS;
  const int m0 = blockIdx.y * 8 * NT, Mr = min(8 * NT, p.M - m0);
  const int nb = (int)w4_blocks(p.K);
  const int b0 = (int)((int64_t)nb * rank / p.C), b1 = (int)((int64_t)nb * (rank + 1) / p.C);

  wait_for_previous_kernel();
  allow_dependent_launch();

  W4Rows r;
  {
    const int64_t last = p.N - 1;  // rows past the end repeat the last one and are not stored
    const int64_t lo = min(row0 + wr * 16 + g, last), hi = min(row0 + wr * 16 + g + 8, last);
    r.lo = p.wq + lo * p.row_bytes + t * 16;
    r.hi = p.wq + hi * p.row_bytes + t * 16;
    r.slo = p.sg + lo;
    r.shi = p.sg + hi;
    r.zlo = p.zp + (ASYM ? lo : 0);
    r.zhi = p.zp + (ASYM ? hi : 0);
    r.pitch = p.N;
    r.last = p.groups - 1;
  }

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;

  const int pitch = p.chunk * 256 + 64;  // bytes per staged token: rows 64 bytes apart modulo 128
  const char* xs[NT];                    // this lane's columns; absent tokens read the last one
#pragma unroll
  for (int n = 0; n < NT; ++n) xs[n] = smem + (int64_t)min(8 * n + g, Mr - 1) * pitch + t * 16;
  const int64_t plane = (int64_t)Mr * pitch;

  for (int c0 = b0; c0 < b1; c0 += p.chunk) {
    const int c1 = min(c0 + p.chunk, b1);
    W4Block w[W4G_DEPTH];
#pragma unroll
    for (int u = 0; u < W4G_DEPTH; ++u) {
      const int b = c0 + wk + u * WK;
      if (b < c1) w4_load<GW, ASYM>(w[u], r, b, t);
    }
    if (c0 != b0) __syncthreads();  // the last chunk has been read
    const int vecs = (c1 - c0) * 16;  // 8-value pieces per token
    for (int i = tid; i < vecs * Mr; i += W4G_THREADS) {
      const int m = i / vecs, v = i % vecs;
      const int64_t k = (int64_t)c0 * W4_BLOCK + v * 8;
      char* dst = smem + (int64_t)m * pitch + v * 16;
      const char* src = p.x + (m0 + m) * p.ldx_bytes;
      if (S == 1) {
        uint4 a = make_uint4(0, 0, 0, 0);
        if (k < p.K) a = *reinterpret_cast<const uint4*>(src + k * 2);
        *reinterpret_cast<uint4*>(dst) = a;
      } else {
        float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (k < p.K) {
          *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(src + k * 4);
          *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(src + k * 4 + 16);
        }
        uint32_t part[8][S];
#pragma unroll
        for (int e = 0; e < 8; ++e) split_bf16<S>(f[e], part[e]);
#pragma unroll
        for (int s = 0; s < S; ++s)
          *reinterpret_cast<uint4*>(dst + s * plane) =
              make_uint4(part[0][s] | (part[1][s] << 16), part[2][s] | (part[3][s] << 16),
                         part[4][s] | (part[5][s] << 16), part[6][s] | (part[7][s] << 16));
      }
    }
    __syncthreads();
    for (int bb = c0 + wk; bb < c1; bb += WK * W4G_DEPTH) {
#pragma unroll
      for (int u = 0; u < W4G_DEPTH; ++u) {
        const int b = bb + u * WK;
        if (b < c1) {
          w4_mac<NT, S, GW, ASYM>(acc, w[u], lane, [&](int n, int s, int i) {
            return *reinterpret_cast<const uint4*>(xs[n] + s * plane + (b - c0) * 256 + i * 64);
          });
          const int next = b + WK * W4G_DEPTH;
          if (next < c1) w4_load<GW, ASYM>(w[u], r, next, t);
        }
      }
    }
  }

  // partial sums: red[wk][token][row]
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float* q = red + (wk * 8 * NT + 8 * n + 2 * t) * RP + wr * 16 + g;
    q[0] = acc[n][0];
    q[RP] = acc[n][1];
    q[8] = acc[n][2];
    q[RP + 8] = acc[n][3];
  }
  __syncthreads();
  const int outs = Mr * ROWS;
  if (p.C == 1) {
    for (int o = tid; o < outs; o += W4G_THREADS) {
      const int m = o / ROWS, row = o % ROWS;
      float v = red[m * RP + row];
#pragma unroll
      for (int k = 1; k < WK; ++k) v = __fadd_rn(v, red[(k * 8 * NT + m) * RP + row]);
      if (row0 + row < p.N) store_out(p.y, (m0 + m) * p.ldy + row0 + row, v, p.y_bf16);
    }
    return;
  }
  for (int o = tid; o < outs; o += W4G_THREADS) {  // each thread sums its own cells, in place
    const int m = o / ROWS, row = o % ROWS;
    float v = red[m * RP + row];
#pragma unroll
    for (int k = 1; k < WK; ++k) v = __fadd_rn(v, red[(k * 8 * NT + m) * RP + row]);
    red[m * RP + row] = v;
  }
  cluster_sync();
  for (int o = rank * W4G_THREADS + tid; o < outs; o += p.C * W4G_THREADS) {
    const int m = o / ROWS, row = o % ROWS;
    float v = ld_dsmem_f32(red + m * RP + row, 0);
    for (int c = 1; c < p.C; ++c) v = __fadd_rn(v, ld_dsmem_f32(red + m * RP + row, c));
    if (row0 + row < p.N) store_out(p.y, (m0 + m) * p.ldy + row0 + row, v, p.y_bf16);
  }
  cluster_sync();  // no CTA leaves while its sums are read
}

}  // namespace sqk

namespace sqh {
namespace {

constexpr int kSmemBudget = 200 * 1024;

template <int NT, int S, int GW, bool ASYM, int WR>
cudaError_t launch_w4_gemm_t(sqk::W4GemmParams p, cudaStream_t st) {
  const int rows = 16 * WR, wk = 8 / WR;
  const int64_t tiles = (p.N + rows - 1) / rows, mt = (p.M + 8 * NT - 1) / (8 * NT);
  const int nb = (int)sqk::w4_blocks(p.K);
  int C = 1;
  while (C < 8 && tiles * mt * C < 2 * num_sms() && nb / (2 * C) >= wk) C *= 2;
  const int mr = std::min(p.M, 8 * NT);
  const int64_t per_block = (int64_t)S * mr * 256, fixed = (int64_t)S * mr * 64;
  p.C = C;
  p.chunk = (int)std::max<int64_t>(1, std::min<int64_t>((nb + C - 1) / C, (kSmemBudget - fixed) / per_block));
  const int64_t red = (int64_t)wk * 8 * NT * (rows + 4) * 4;
  const size_t smem = (size_t)std::max(fixed + p.chunk * per_block, red);
  auto kern = sqk::w4_gemm_kernel<NT, S, GW, ASYM, WR>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * C), (unsigned)mt);
  cfg.blockDim = dim3(sqk::W4G_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int NT, int S, int WR>
cudaError_t launch_w4_gemm_g(const sqk::W4GemmParams& p, int group, cudaStream_t st) {
  if (p.zp) {
    if (group == 32) return launch_w4_gemm_t<NT, S, 1, true, WR>(p, st);
    if (group == 64) return launch_w4_gemm_t<NT, S, 2, true, WR>(p, st);
    return launch_w4_gemm_t<NT, S, 4, true, WR>(p, st);
  }
  if (group == 32) return launch_w4_gemm_t<NT, S, 1, false, WR>(p, st);
  if (group == 64) return launch_w4_gemm_t<NT, S, 2, false, WR>(p, st);
  return launch_w4_gemm_t<NT, S, 4, false, WR>(p, st);
}

template <int S>
cudaError_t launch_w4_gemm_m(const sqk::W4GemmParams& p, int group, cudaStream_t st) {
  if (p.M <= 8) return launch_w4_gemm_g<1, S, 1>(p, group, st);
  if (p.M <= 16) return launch_w4_gemm_g<2, S, 2>(p, group, st);
  return launch_w4_gemm_g<4, S, 4>(p, group, st);
}

}  // namespace

cudaError_t launch_w4_gemm(const void* x, bool bf16, int64_t M, int64_t K, int64_t ldx, const uint8_t* wq,
                           const uint16_t* sg, const uint8_t* zp, int64_t N, int group, void* y, bool y_bf16,
                           int64_t ldy, cudaStream_t st) {
  sqk::W4GemmParams p{};
  p.x = (const char*)x;
  p.ldx_bytes = ldx * (bf16 ? 2 : 4);
  p.M = (int)M;
  p.K = (int)K;
  p.wq = (const char*)wq;
  p.sg = sg;
  p.zp = zp;
  p.N = N;
  p.row_bytes = sqk::w4_blocks(K) * sqk::W4_BLOCK_BYTES;
  p.groups = (int)((K + group - 1) / group);
  p.y = y;
  p.ldy = ldy;
  p.y_bf16 = y_bf16;
  return bf16 ? launch_w4_gemm_m<1>(p, group, st) : launch_w4_gemm_m<3>(p, group, st);
}

}  // namespace sqh
