// sq_moe.cu -- a whole mixture-of-experts layer for a few tokens, experts' weights in 4 bits.
//
//   logits[t, e] = sum_d x[t, d] Wr[e, d]     p = softmax(logits)     the k largest of each token
//   h[t, e, f]   = silu(W1_e[f] . x_t) * (W3_e[f] . x_t)
//   y[t]         = sum over the chosen e of weight[t, e] * (W2_e h[t, e])
//
// Bound: the chosen experts' codes, each read once from HBM.  Three kernels, chained as
// programmatic dependents: the router (its last block builds the lists), gate/up, down.  The work
// is cut by (expert, rows), never by token: an expert's weights are read once for all of its
// tokens, which are the columns of the mma (sq_w4.cuh).
//   Router sums are binary64, so that which experts are chosen does not hang on rounding.  h is
// kept as two bf16 parts (16 significant bits; three for a binary32 layer), so the only bf16
// rounding of the layer is the final store.  Every sum has a fixed order; the only atomics are the
// lists' bit masks (order-free) and the router's arrival count.
#include <algorithm>

#include "sq_w4.cuh"

namespace sqk {

constexpr int MOE_MAX_T = 64;    // tokens: one bit each of an expert's token mask
constexpr int MOE_MAX_E = 1024;  // experts
constexpr int MOE_MAX_K = 32;    // choices per token
constexpr int MOE_THREADS = 256;

struct MoeLists {  // in the workspace, written by the router (or from given choices)
  unsigned int arrived;  // router blocks that are done; wraps to 0 by itself
  int active;            // experts with tokens
};

struct MoeParams {
  const char* x;
  int64_t ldx_bytes;
  const char* wr;
  int x_bf16, wr_bf16;
  int T, D, F, E, top_k, renorm;
  int* ids;
  float* wts;
  const int* ids_in;
  const float* wts_in;
  const char *w13, *w2;
  const uint16_t *s13, *s2;
  const uint8_t *z13, *z2;
  int64_t rb13, rb2;  // bytes per packed row
  int g13, g2;        // groups per row
  void* y;
  int64_t ldy;
  int y_bf16;
  // workspace
  MoeLists* lists;
  double* logits;       // [T, E]
  int* expert;          // [active] expert of an entry
  int* start;           // [active + 1] its first slot
  int* slot_token;      // [T k]
  float* slot_weight;   // [T k]
  uint16_t* xparts;     // [3, T, D] (binary32 x)
  uint16_t* h;          // [parts, T k, F]
  int C;                // CTAs of the down kernel's cluster
};

// ---------------------------------------------------------------------------- lists
struct MoeShared {
  unsigned long long mask[MOE_MAX_E];
  int offset[MOE_MAX_E];
  int scan[MOE_THREADS];
};

// Builds the expert lists from the choices in `ids`, `wts` [T, k] (one block).  A choice outside
// [0, E) is left out; one that a token names twice counts once, with the weights' sum.
__device__ void moe_build_lists(const MoeParams& p, MoeShared& sh, const int* ids, const float* wts) {
  const int tid = threadIdx.x;
  for (int e = tid; e < p.E; e += MOE_THREADS) sh.mask[e] = 0ull;
  __syncthreads();
  const int pairs = p.T * p.top_k;
  for (int i = tid; i < pairs; i += MOE_THREADS) {
    const int e = ids[i];
    if (e >= 0 && e < p.E) atomicOr(&sh.mask[e], 1ull << (i / p.top_k));
  }
  __syncthreads();
  // exclusive sums of tokens and of active experts: a run of experts per thread, then a scan
  const int per = (p.E + MOE_THREADS - 1) / MOE_THREADS;
  int tokens = 0, active = 0;
  for (int e = tid * per; e < min(p.E, (tid + 1) * per); ++e) {
    const int c = __popcll(sh.mask[e]);
    tokens += c;
    active += c > 0;
  }
  int packed = tokens | (active << 16);  // at most 2048 slots and 1024 experts
  sh.scan[tid] = packed;
  __syncthreads();
  for (int o = 1; o < MOE_THREADS; o *= 2) {
    const int v = tid >= o ? sh.scan[tid - o] : 0;
    __syncthreads();
    sh.scan[tid] += v;
    __syncthreads();
  }
  const int before = sh.scan[tid] - packed;
  tokens = before & 0xffff;
  active = before >> 16;
  for (int e = tid * per; e < min(p.E, (tid + 1) * per); ++e) {
    const int c = __popcll(sh.mask[e]);
    sh.offset[e] = tokens;
    if (c > 0) {
      p.expert[active] = e;
      p.start[active] = tokens;
      ++active;
      tokens += c;
    }
  }
  if (tid == MOE_THREADS - 1) {
    const int total = sh.scan[tid];
    p.lists->active = total >> 16;
    p.start[total >> 16] = total & 0xffff;
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += MOE_THREADS) {
    const int e = ids[i], t = i / p.top_k, first = t * p.top_k;
    if (e < 0 || e >= p.E) continue;
    float w = 0.0f;
    bool earlier = false;
    for (int j = first; j < first + p.top_k; ++j) {
      if (ids[j] != e) continue;
      earlier |= j < i;
      w = __fadd_rn(w, wts[j]);
    }
    if (earlier) continue;
    const int slot = sh.offset[e] + __popcll(sh.mask[e] & ((1ull << t) - 1ull));
    p.slot_token[slot] = t;
    p.slot_weight[slot] = w;
  }
}

// ---------------------------------------------------------------------------- router
template <bool BF16>
__device__ __forceinline__ void load8(const char* p, float f[8]) {
  if (BF16) {
    unpack8_bf16(*reinterpret_cast<const uint4*>(p), f);
  } else {
    *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(p);
    *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(p + 16);
  }
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The k largest logits of one token, by one warp: ties to the lowest index, NaN counts as -inf.
__device__ void moe_choose(const MoeParams& p, int t, int lane) {
  constexpr int PER = MOE_MAX_E / 32;
  const double* row = p.logits + (int64_t)t * p.E;
  const double none = -__longlong_as_double(0x7ff0000000000000ll);
  unsigned int taken = 0u;  // one bit per value of this lane
  double top = none;
  bool nan = false;
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    if (e >= p.E) break;
    const double v = row[e];
    nan |= v != v;
    top = v > top ? v : top;
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    const double v = __shfl_xor_sync(0xffffffffu, top, o);
    top = v > top ? v : top;
  }
  nan = __any_sync(0xffffffffu, nan);
  double sum = 0.0;
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    if (e >= p.E) break;
    sum += (double)expf((float)(row[e] - top));
  }
  sum = warp_sum(sum);
  double chosen_sum = 0.0, mine = 0.0;
  int my_id = 0;
  for (int j = 0; j < p.top_k; ++j) {
    double best = none;
    int at = INT32_MAX;
    for (int i = 0; i < PER; ++i) {
      const int e = i * 32 + lane;
      if (e >= p.E) break;
      if (taken >> i & 1u) continue;
      const double v = row[e];
      if (at == INT32_MAX || v > best) {
        best = v == v ? v : none;
        at = e;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
      const double v = __shfl_xor_sync(0xffffffffu, best, o);
      const int a = __shfl_xor_sync(0xffffffffu, at, o);
      if (a != INT32_MAX && (at == INT32_MAX || v > best || (v == best && a < at))) {
        best = v;
        at = a;
      }
    }
    if (at % 32 == lane) taken |= 1u << (at / 32);
    const double w = nan ? __longlong_as_double(0x7ff8000000000000ll) : (double)expf((float)(best - top)) / sum;
    chosen_sum += w;
    if (j == lane) {
      mine = w;
      my_id = at;
    }
  }
  if (lane < p.top_k) {
    p.ids[t * p.top_k + lane] = my_id;
    p.wts[t * p.top_k + lane] = (float)(p.renorm ? mine / chosen_sum : mine);
  }
}

// Block (e, token block): logits of one expert, tokens in turn; the 8 warps split D.
template <bool XB, bool RB>
__global__ void __launch_bounds__(MOE_THREADS) moe_router_kernel(const MoeParams p) {
  __shared__ MoeShared sh;
  __shared__ double part[8];
  __shared__ bool last;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  wait_for_previous_kernel();
  allow_dependent_launch();
  const int e = blockIdx.x;
  const char* wrow = p.wr + (int64_t)e * p.D * (RB ? 2 : 4);
  for (int t = blockIdx.y; t < p.T; t += gridDim.y) {
    double sum = 0.0;
    for (int d = tid * 8; d < p.D; d += MOE_THREADS * 8) {
      float a[8], w[8];
      load8<XB>(p.x + t * p.ldx_bytes + (int64_t)d * (XB ? 2 : 4), a);
      load8<RB>(wrow + (int64_t)d * (RB ? 2 : 4), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fma((double)a[i], (double)w[i], sum);
    }
    sum = warp_sum(sum);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      double v = 0.0;
      for (int i = 0; i < 8; ++i) v += part[i];
      p.logits[(int64_t)t * p.E + e] = v;
    }
    __syncthreads();
  }
  // the last block to arrive chooses and builds the lists
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicInc(&p.lists->arrived, gridDim.x * gridDim.y - 1) == gridDim.x * gridDim.y - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int t = warp; t < p.T; t += 8) moe_choose(p, t, lane);
  __syncthreads();
  moe_build_lists(p, sh, p.ids, p.wts);
}

__global__ void __launch_bounds__(MOE_THREADS) moe_lists_kernel(const MoeParams p) {
  __shared__ MoeShared sh;
  wait_for_previous_kernel();
  allow_dependent_launch();
  moe_build_lists(p, sh, p.ids_in, p.wts_in);
}

// binary32 x as three bf16 planes.
__global__ void __launch_bounds__(256) moe_split_kernel(const MoeParams p) {
  wait_for_previous_kernel();
  allow_dependent_launch();
  const int64_t plane = (int64_t)p.T * p.D;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < plane; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / p.D, d = i % p.D;
    uint32_t part[3];
    split_bf16<3>(reinterpret_cast<const float*>(p.x + t * p.ldx_bytes)[d], part);
#pragma unroll
    for (int s = 0; s < 3; ++s) p.xparts[s * plane + i] = (uint16_t)part[s];
  }
}

// ---------------------------------------------------------------------------- gate and up
__device__ __forceinline__ uint4 ld_parts(const char* row, int64_t k, int64_t K) {
  return k < K ? *reinterpret_cast<const uint4*>(row + k * 2) : make_uint4(0, 0, 0, 0);
}

constexpr int MOE_DEPTH = 4;

// Blocks [b0, b1) in steps of `step`, `depth` of them in flight.
template <int NT, int S, int GW, bool ASYM>
__device__ __forceinline__ void moe_run(float (&acc)[NT][4], const W4Rows& r, const char* const (&rows)[NT],
                                        int64_t plane_bytes, int b0, int b1, int step, int64_t K, int lane) {
  const int t = lane % 4;
  W4Block w[MOE_DEPTH];
#pragma unroll
  for (int u = 0; u < MOE_DEPTH; ++u)
    if (b0 + u * step < b1) w4_load<GW, ASYM>(w[u], r, b0 + u * step, t);
  for (int bb = b0; bb < b1; bb += step * MOE_DEPTH) {
#pragma unroll
    for (int u = 0; u < MOE_DEPTH; ++u) {
      const int b = bb + u * step;
      if (b < b1) {
        w4_mac<NT, S, GW, ASYM>(acc, w[u], lane, [&](int n, int s, int i) {
          return ld_parts(rows[n] + s * plane_bytes, (int64_t)b * W4_BLOCK + 32 * i + 8 * t, K);
        });
        if (b + step * MOE_DEPTH < b1) w4_load<GW, ASYM>(w[u], r, b + step * MOE_DEPTH, t);
      }
    }
  }
}

// Item: 8 rows f of one expert's gate and the same 8 of its up projection, as the two halves of a
// 16-row tile, so one thread ends up with both sums of an h.  The block's 8 warps split D.
template <int NT, int S, int SH, int GW, bool ASYM>
__device__ __forceinline__ void moe_up_tile(const MoeParams& p, float* red, int e, int f0, int slot0, int count) {
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int nb = (int)w4_blocks(p.D);
  W4Rows r;
  const int f = min(f0 + g, p.F - 1);
  const int64_t row = (int64_t)e * 2 * p.F + f;
  r.lo = p.w13 + row * p.rb13 + t * 16;
  r.hi = p.w13 + (row + p.F) * p.rb13 + t * 16;
  const int64_t sbase = (int64_t)e * p.g13 * 2 * p.F + f;
  r.slo = p.s13 + sbase;
  r.shi = p.s13 + sbase + p.F;
  r.zlo = p.z13 + (ASYM ? sbase : 0);
  r.zhi = p.z13 + (ASYM ? sbase + p.F : 0);
  r.pitch = 2 * (int64_t)p.F;
  r.last = p.g13 - 1;
  const char* rows[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int tok = p.slot_token[slot0 + min(8 * n + g, count - 1)];
    rows[n] = S == 1 ? p.x + tok * p.ldx_bytes : reinterpret_cast<const char*>(p.xparts) + (int64_t)tok * p.D * 2;
  }
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
  moe_run<NT, S, GW, ASYM>(acc, r, rows, (int64_t)p.T * p.D * 2, warp, nb, 8, p.D, lane);
  __syncthreads();  // the last tile's sums have been read
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[((n * 4 + i) * 8 + warp) * 32 + lane] = acc[n][i];
  __syncthreads();
  for (int o = tid; o < NT * 64; o += MOE_THREADS) {  // (column 8 n + 2 q + c, row gg) of lane gg * 4 + q
    const int n = o / 64, c = o / 32 % 2, l = o % 32, col = 8 * n + 2 * (l % 4) + c, ff = f0 + l / 4;
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      gate = __fadd_rn(gate, red[((n * 4 + c) * 8 + k) * 32 + l]);
      up = __fadd_rn(up, red[((n * 4 + 2 + c) * 8 + k) * 32 + l]);
    }
    if (col < count && ff < p.F) {
      // silu(v) = v / (1 + exp(-v)); exp overflows to inf for very negative v, and v / inf is -0
      const float h = __fmul_rn(__fdiv_rn(gate, __fadd_rn(1.0f, expf(-gate))), up);
      uint32_t part[SH];
      split_bf16_stored<SH>(h, part);
#pragma unroll
      for (int s = 0; s < SH; ++s)
        p.h[((int64_t)s * p.T * p.top_k + slot0 + col) * p.F + ff] = (uint16_t)part[s];
    }
  }
}

template <int S, int SH, int GW, bool ASYM>
__global__ void __launch_bounds__(MOE_THREADS) moe_up_kernel(const MoeParams p) {
  __shared__ float red[2 * 4 * 8 * 32];
  wait_for_previous_kernel();
  allow_dependent_launch();
  const int tiles = (p.F + 7) / 8;
  const int items = p.lists->active * tiles;
  for (int i = blockIdx.x; i < items; i += gridDim.x) {
    const int a = i / tiles, e = p.expert[a], f0 = (i % tiles) * 8;
    const int s1 = p.start[a + 1];
    for (int s0 = p.start[a]; s0 < s1; s0 += 16) {
      if (s1 - s0 <= 8) moe_up_tile<1, S, SH, GW, ASYM>(p, red, e, f0, s0, s1 - s0);
      else moe_up_tile<2, S, SH, GW, ASYM>(p, red, e, f0, s0, min(16, s1 - s0));
    }
  }
}

// ---------------------------------------------------------------------------- down
template <int NT, int SH, int GW, bool ASYM>
__device__ __forceinline__ void moe_down_part(const MoeParams& p, float* mine, int e, int d0, int slot0, int count,
                                              int b0, int b1) {
  const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  W4Rows r;
  const int lo = min(d0 + g, p.D - 1), hi = min(d0 + g + 8, p.D - 1);
  r.lo = p.w2 + ((int64_t)e * p.D + lo) * p.rb2 + t * 16;
  r.hi = p.w2 + ((int64_t)e * p.D + hi) * p.rb2 + t * 16;
  const int64_t sbase = (int64_t)e * p.g2 * p.D;
  r.slo = p.s2 + sbase + lo;
  r.shi = p.s2 + sbase + hi;
  r.zlo = p.z2 + (ASYM ? sbase + lo : 0);
  r.zhi = p.z2 + (ASYM ? sbase + hi : 0);
  r.pitch = p.D;
  r.last = p.g2 - 1;
  const char* rows[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    rows[n] = reinterpret_cast<const char*>(p.h + (int64_t)(slot0 + min(8 * n + g, count - 1)) * p.F);
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
  moe_run<NT, SH, GW, ASYM>(acc, r, rows, (int64_t)p.T * p.top_k * p.F * 2, b0, b1, 1, p.F, lane);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = 8 * n + 2 * t + c;
      if (col < count) {  // an expert's tokens differ, so no two lanes meet in a cell
        const float w = p.slot_weight[slot0 + col];
        float* cell = mine + p.slot_token[slot0 + col] * 16 + g;
        cell[0] = __fmaf_rn(w, acc[n][c], cell[0]);
        cell[8] = __fmaf_rn(w, acc[n][2 + c], cell[8]);
      }
    }
  }
  __syncwarp();
}

// A cluster owns 16 rows d for every token; its warps cut the (expert, block) line into equal runs.
template <int SH, int GW, bool ASYM>
__global__ void __launch_bounds__(MOE_THREADS) moe_down_kernel(const MoeParams p) {
  extern __shared__ __align__(16) float sums[];  // [8 warps][T][16]
  const int tid = threadIdx.x, warp = tid / 32;
  const int rank = blockIdx.x % p.C, d0 = blockIdx.x / p.C * 16;
  const int cells = p.T * 16;
  for (int i = tid; i < 8 * cells; i += MOE_THREADS) sums[i] = 0.0f;
  wait_for_previous_kernel();
  allow_dependent_launch();
  __syncthreads();
  const int nb = (int)w4_blocks(p.F);
  const int64_t line = (int64_t)p.lists->active * nb;
  const int runs = 8 * p.C, run = rank * 8 + warp;
  const int64_t l1 = line * (run + 1) / runs;
  for (int64_t l = line * run / runs; l < l1;) {
    const int a = (int)(l / nb), b0 = (int)(l % nb), b1 = (int)min((int64_t)nb, b0 + (l1 - l));
    const int e = p.expert[a], s1 = p.start[a + 1];
    for (int s0 = p.start[a]; s0 < s1; s0 += 16) {
      if (s1 - s0 <= 8) moe_down_part<1, SH, GW, ASYM>(p, sums + warp * cells, e, d0, s0, s1 - s0, b0, b1);
      else moe_down_part<2, SH, GW, ASYM>(p, sums + warp * cells, e, d0, s0, min(16, s1 - s0), b0, b1);
    }
    l += b1 - b0;
  }
  __syncthreads();
  for (int o = tid; o < cells; o += MOE_THREADS) {
    float v = sums[o];
#pragma unroll
    for (int k = 1; k < 8; ++k) v = __fadd_rn(v, sums[k * cells + o]);
    sums[o] = v;
  }
  if (p.C > 1) cluster_sync();
  else __syncthreads();
  for (int o = rank * MOE_THREADS + tid; o < cells; o += p.C * MOE_THREADS) {
    const int t = o / 16, d = d0 + o % 16;
    float v = sums[o];
    if (p.C > 1) {
      v = ld_dsmem_f32(sums + o, 0);
      for (int c = 1; c < p.C; ++c) v = __fadd_rn(v, ld_dsmem_f32(sums + o, c));
    }
    if (d < p.D) store_out(p.y, t * p.ldy + d, v, p.y_bf16);
  }
  if (p.C > 1) cluster_sync();
}

}  // namespace sqk

namespace sqh {
namespace {

cudaError_t launch_dependent(const void* kern, unsigned gx, unsigned gy, size_t smem, int cluster,
                             const sqk::MoeParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(gx, gy);
  cfg.blockDim = dim3(sqk::MOE_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  void* args[] = {const_cast<sqk::MoeParams*>(&p)};
  return cudaLaunchKernelExC(&cfg, kern, args);
}

template <int S, int SH, int GW, bool ASYM>
cudaError_t launch_experts(sqk::MoeParams p, cudaStream_t st) {
  const int sms = num_sms();
  cudaError_t e = launch_dependent((const void*)sqk::moe_up_kernel<S, SH, GW, ASYM>, (unsigned)(4 * sms), 1, 0, 1, p, st);
  if (e != cudaSuccess) return e;
  const int tiles = (p.D + 15) / 16;
  p.C = 1;
  while (p.C < 8 && tiles * p.C < 3 * sms) p.C *= 2;
  const size_t smem = (size_t)8 * p.T * 16 * 4;
  return launch_dependent((const void*)sqk::moe_down_kernel<SH, GW, ASYM>, (unsigned)(tiles * p.C), 1, smem, p.C, p, st);
}

template <int S, int SH>
cudaError_t launch_experts_g(const sqk::MoeParams& p, int group, cudaStream_t st) {
  if (p.z13) {
    if (group == 32) return launch_experts<S, SH, 1, true>(p, st);
    if (group == 64) return launch_experts<S, SH, 2, true>(p, st);
    return launch_experts<S, SH, 4, true>(p, st);
  }
  if (group == 32) return launch_experts<S, SH, 1, false>(p, st);
  if (group == 64) return launch_experts<S, SH, 2, false>(p, st);
  return launch_experts<S, SH, 4, false>(p, st);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

// Slices of the workspace; returns its size.
static size_t moe_layout(sqk::MoeParams* p, char* base, int64_t T, int64_t D, int64_t F, int64_t E, int64_t k) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* r = base ? base + at : nullptr;
    at += up256(bytes);
    return r;
  };
  sqk::MoeParams q{};
  q.lists = (sqk::MoeLists*)take(sizeof(sqk::MoeLists));
  q.logits = (double*)take((size_t)(T * E) * 8);
  q.expert = (int*)take((size_t)E * 4);
  q.start = (int*)take((size_t)(E + 1) * 4);
  q.slot_token = (int*)take((size_t)(T * k) * 4);
  q.slot_weight = (float*)take((size_t)(T * k) * 4);
  q.xparts = (uint16_t*)take((size_t)(3 * T * D) * 2);
  q.h = (uint16_t*)take((size_t)(3 * T * k * F) * 2);
  if (p) {
    p->lists = q.lists;
    p->logits = q.logits;
    p->expert = q.expert;
    p->start = q.start;
    p->slot_token = q.slot_token;
    p->slot_weight = q.slot_weight;
    p->xparts = q.xparts;
    p->h = q.h;
  }
  return at;
}

size_t moe_workspace_size(int64_t T, int64_t D, int64_t F, int64_t E, int64_t top_k) {
  return moe_layout(nullptr, nullptr, T, D, F, E, top_k);
}

// wr != NULL: the router chooses, writing ids and wts; else ids_in and wts_in are the choices.
cudaError_t launch_moe_w4(const void* x, bool bf16, int64_t T, int64_t D, int64_t ldx, const void* wr, bool wr_bf16,
                          int64_t E, int64_t top_k, bool renorm, int* ids, float* wts, const int* ids_in,
                          const float* wts_in, const uint8_t* w13, const uint16_t* s13, const uint8_t* z13,
                          const uint8_t* w2, const uint16_t* s2, const uint8_t* z2, int64_t F, int group, void* y,
                          bool y_bf16, int64_t ldy, void* workspace, cudaStream_t st) {
  sqk::MoeParams p{};
  moe_layout(&p, (char*)workspace, T, D, F, E, top_k);
  p.x = (const char*)x;
  p.ldx_bytes = ldx * (bf16 ? 2 : 4);
  p.wr = (const char*)wr;
  p.x_bf16 = bf16;
  p.wr_bf16 = wr_bf16;
  p.T = (int)T;
  p.D = (int)D;
  p.F = (int)F;
  p.E = (int)E;
  p.top_k = (int)top_k;
  p.renorm = renorm;
  p.ids = ids;
  p.wts = wts;
  p.ids_in = ids_in;
  p.wts_in = wts_in;
  p.w13 = (const char*)w13;
  p.s13 = s13;
  p.z13 = z13;
  p.w2 = (const char*)w2;
  p.s2 = s2;
  p.z2 = z2;
  p.rb13 = sqk::w4_blocks(D) * sqk::W4_BLOCK_BYTES;
  p.rb2 = sqk::w4_blocks(F) * sqk::W4_BLOCK_BYTES;
  p.g13 = (int)((D + group - 1) / group);
  p.g2 = (int)((F + group - 1) / group);
  p.y = y;
  p.ldy = ldy;
  p.y_bf16 = y_bf16;
  p.C = 1;
  cudaError_t e;
  if (!bf16) {
    e = launch_dependent((const void*)sqk::moe_split_kernel, (unsigned)num_sms(), 1, 0, 1, p, st);
    if (e != cudaSuccess) return e;
  }
  if (wr) {
    const void* k = bf16 ? (wr_bf16 ? (const void*)sqk::moe_router_kernel<true, true> : (const void*)sqk::moe_router_kernel<true, false>)
                         : (wr_bf16 ? (const void*)sqk::moe_router_kernel<false, true> : (const void*)sqk::moe_router_kernel<false, false>);
    e = launch_dependent(k, (unsigned)E, (unsigned)std::min<int64_t>(T, 8), 0, 1, p, st);
  } else {
    e = launch_dependent((const void*)sqk::moe_lists_kernel, 1, 1, 0, 1, p, st);
  }
  if (e != cudaSuccess) return e;
  return bf16 ? launch_experts_g<1, 2>(p, group, st) : launch_experts_g<3, 3>(p, group, st);
}

}  // namespace sqh
