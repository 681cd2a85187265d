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
// lists' bit masks (order-free) and the router's arrival count.  The expert kernels are one CTA per
// SM with the weight stream of sq_w4.cuh.
#include <algorithm>

#include "sq_w4.cuh"

namespace sqk {

constexpr int MOE_MAX_T = 64;    // tokens: one bit each of an expert's token mask
constexpr int MOE_MAX_E = 1024;  // experts
constexpr int MOE_MAX_K = 32;    // choices per token
constexpr int MOE_THREADS = 256;
constexpr int MOE_ENTRY = 32;    // tokens of an entry: four column tiles of the mma

struct MoeLists {  // in the workspace, written by the router (or from given choices)
  unsigned int arrived;  // router blocks that are done; wraps to 0 by itself
  int active;            // entries: experts with tokens, MOE_ENTRY of them at a time
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
  int* start;           // [active + 1] its first slot; the slots of an expert's entries follow one another
  int* slot_token;      // [T k]
  float* slot_weight;   // [T k]
  uint16_t* xparts;     // [3, T, D] (binary32 x)
  uint16_t* h;          // [parts, T k, F]
  // the expert kernels' shared memory
  bool x_staged;        // x in shared memory
  int up_cells_at, up_ring_at, up_pass;  // tiles whose cells fit
  int down_ring_at, down_pass;
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
  // exclusive sums of tokens and of entries: a run of experts per thread, then a scan
  const int per = (p.E + MOE_THREADS - 1) / MOE_THREADS;
  int tokens = 0, active = 0;
  for (int e = tid * per; e < min(p.E, (tid + 1) * per); ++e) {
    const int c = __popcll(sh.mask[e]);
    tokens += c;
    active += (c + MOE_ENTRY - 1) / MOE_ENTRY;
  }
  int packed = tokens | (active << 16);  // at most 2048 slots and as many entries
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
    for (int first = 0; first < c; first += MOE_ENTRY) {
      p.expert[active] = e;
      p.start[active] = tokens + first;
      ++active;
    }
    tokens += c;
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

// ---------------------------------------------------------------------------- experts
constexpr int MOE_DEPTH = 3;   // slots of a warp's ring
constexpr int MOE_WARPS = 16;  // of an expert kernel's CTA
constexpr int MOE_EXPERT_THREADS = 32 * MOE_WARPS;
constexpr int MOE_NT = MOE_ENTRY / 8;

// The 8 values at k of a row of x or h (shared or global memory); zeros past its end.
__device__ __forceinline__ uint4 moe_row8(const char* row, int k, int K) {
  return k < K ? *reinterpret_cast<const uint4*>(row + k * 2) : make_uint4(0, 0, 0, 0);
}

// One unit for an entry of `count` tokens: as many column tiles as they need.
template <int S, int GW, bool ASYM>
__device__ __forceinline__ void moe_mac(float (&acc)[MOE_NT][4], uint32_t slot, int lane, int count,
                                        const char* const (&rows)[MOE_NT], int64_t plane, int b, int K) {
  const int k0 = b * W4_UNIT + (lane % 4) * 8;
  auto x = [&](int n, int s, int i) { return moe_row8(rows[n] + s * plane, k0 + 32 * i, K); };
  if (count <= 8) w4_mac<1, S, GW, ASYM>(acc, slot, lane, x);
  else if (count <= 16) w4_mac<2, S, GW, ASYM>(acc, slot, lane, x);
  else w4_mac<4, S, GW, ASYM>(acc, slot, lane, x);
}

// Gate and up: a tile is 8 rows f of an entry's gate and the same 8 of its up projection, as the two
// halves of a 16-row tile, so one thread finds both sums of an h.  The tiles of all entries are one
// line, cut over the CTAs and there over the warps (sq_w4.cuh).
template <int S, int SH, int GW, bool ASYM>
__global__ void __launch_bounds__(MOE_EXPERT_THREADS, 1) moe_up_kernel(const MoeParams p) {
  constexpr int SLOT = W4Slot<GW, ASYM>::BYTES, RP = W4_RP;
  extern __shared__ __align__(16) char smem[];
  __shared__ W4Runs<MOE_WARPS> runs;
  const int tid = threadIdx.x, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);
  const int cell_floats = min(p.T, MOE_ENTRY) * RP;
  float* cells = reinterpret_cast<float*>(smem + p.up_cells_at);
  const uint32_t ring = smem_u32(smem + p.up_ring_at) + warp * MOE_DEPTH * SLOT;
  const int nb = w4_units(p.D), per_expert = p.F / 8;
  wait_for_previous_kernel();
  allow_dependent_launch();
  const int64_t tiles = (int64_t)p.lists->active * per_expert;
  const int64_t t0 = tiles * blockIdx.x / gridDim.x;
  const int my_tiles = (int)(tiles * (blockIdx.x + 1) / gridDim.x - t0);
  const char* xbase = S == 1 ? p.x : reinterpret_cast<const char*>(p.xparts);
  const int64_t xpitch = S == 1 ? p.ldx_bytes : (int64_t)p.D * 2;
  const int64_t xplane = S == 1 ? 0 : (int64_t)p.T * p.D * 2;
  const int spitch = (int)w4_blocks(p.D) * 256 + 64;  // rows 64 bytes apart modulo 128

  for (int p0 = 0; p0 < my_tiles; p0 += p.up_pass) {
    const int n_tiles = min(p.up_pass, my_tiles - p0), line = n_tiles * nb;
    if (p0 != 0) __syncthreads();  // the last pass's cells have been read
    else if (p.x_staged) {
      for (int m = 0; m < S * p.T; ++m) {
        const char* src = xbase + (m % p.T) * xpitch + m / p.T * xplane;
        for (int v = tid; v < p.D / 8; v += MOE_EXPERT_THREADS) cp_async16(smem_u32(smem + m * spitch + v * 16), src + v * 16);
      }
    }
    cp_commit();
    const W4Run run = w4_runs<MOE_WARPS>(runs, line, nb, warp, lane);
    int tile = run.tile, b = run.b;
    float* cell = cells + run.cell * cell_floats + g;

    W4Base base{};
    base.row_bytes = (uint32_t)p.rb13;
    base.pitch = 2 * p.F;
    base.groups = p.g13;
    auto place = [&](int ti, int at_b) {
      const int64_t at = t0 + p0 + ti;
      const int a = (int)(at / per_expert), f0 = (int)(at - (int64_t)a * per_expert) * 8;
      const int64_t e = p.expert[a];
      base.codes = p.w13 + e * 2 * p.F * p.rb13;
      base.scales = p.s13 + e * p.g13 * 2 * p.F;
      if (ASYM) base.zeros = p.z13 + e * p.g13 * 2 * p.F;
      return w4_place<GW, ASYM, true>(base, f0, p.F + f0, 2 * p.F - 1, at_b, lane);
    };
    int to_load = run.units, load_tile = tile, load_b = b;
    W4Cursor cur{};
    if (to_load > 0) cur = place(tile, b);
    const bool odd = w4_blocks(p.D) % 2 != 0;  // the last unit of a row is half a one
    auto issue = [&](uint32_t into) {
      if (to_load > 0) {
        w4_issue<GW, ASYM, true>(into, base, cur, odd && load_b == nb - 1, lane);
        --to_load;
        if (++load_b == nb) {
          load_b = 0;
          ++load_tile;
          if (to_load > 0) cur = place(load_tile, 0);
        }
      }
      cp_commit();
    };
#pragma unroll 1
    for (int u = 0; u < MOE_DEPTH - 1; ++u) issue(ring + u * SLOT);
    cp_wait<MOE_DEPTH - 1>();  // x; the ring's blocks are younger
    __syncthreads();

    float acc[MOE_NT][4] = {};
    const char* rows[MOE_NT];
    int count = 0;
    bool begin = true;
    uint32_t slot = ring, spent = ring + (MOE_DEPTH - 1) * SLOT;
    for (int left = run.units; left > 0; --left) {
      if (begin) {
        const int a = (int)((t0 + p0 + tile) / per_expert), s0 = p.start[a];
        count = p.start[a + 1] - s0;
#pragma unroll
        for (int n = 0; n < MOE_NT; ++n) {
          const int tok = p.slot_token[s0 + min(8 * n + g, count - 1)];
          rows[n] = p.x_staged ? smem + tok * spitch : xbase + tok * xpitch;
        }
        begin = false;
      }
      cp_wait<MOE_DEPTH - 2>();
      __syncwarp();
      issue(spent);
      moe_mac<S, GW, ASYM>(acc, slot, lane, count, rows, p.x_staged ? (int64_t)p.T * spitch : xplane, b, p.D);
      spent = slot;
      slot = slot == ring + (MOE_DEPTH - 1) * SLOT ? ring : slot + SLOT;
      if (++b == nb || left == 1) {
#pragma unroll
        for (int n = 0; n < MOE_NT; ++n) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int m = 8 * n + 2 * t + c;
            if (m < count) {
              cell[m * RP] = acc[n][c];
              cell[m * RP + 8] = acc[n][2 + c];
            }
            acc[n][c] = acc[n][2 + c] = 0.0f;
          }
        }
        cell += cell_floats;
        b = 0;
        ++tile;
        begin = true;
      }
    }
    __syncthreads();
    const int cols = min(p.T, MOE_ENTRY);
    const float inv_line = __frcp_rn((float)line);
    for (int o = tid; o < n_tiles * cols * 8; o += MOE_EXPERT_THREADS) {
      const int f = o % 8, mt = o / 8, ti = mt / cols, m = mt - ti * cols;
      const int64_t at = t0 + p0 + ti;
      const int a = (int)(at / per_expert), s0 = p.start[a];
      if (m >= p.start[a + 1] - s0) continue;
      const float* q = cells + m * RP + f;
      float gate = 0.0f, up = 0.0f;
      const int from = w4_first_cell<MOE_WARPS>(runs, ti, n_tiles, line, inv_line, nb);
      const int to = w4_first_cell<MOE_WARPS>(runs, ti + 1, n_tiles, line, inv_line, nb);
      for (int c = from; c < to; ++c) {
        gate = __fadd_rn(gate, q[c * cell_floats]);
        up = __fadd_rn(up, q[c * cell_floats + 8]);
      }
      // silu(v) = v / (1 + exp(-v)); exp overflows to inf for very negative v, and v / inf is -0
      const float h = __fmul_rn(__fdiv_rn(gate, __fadd_rn(1.0f, expf(-gate))), up);
      uint32_t part[SH];
      split_bf16_stored<SH>(h, part);
      const int64_t ff = (at - (int64_t)a * per_expert) * 8 + f;
#pragma unroll
      for (int s = 0; s < SH; ++s) p.h[((int64_t)s * p.T * p.top_k + s0 + m) * p.F + ff] = (uint16_t)part[s];
    }
  }
}

// Down: a tile is 16 rows d; its blocks are those of every entry in turn (a rank of a cluster takes
// a share of that line, where there are few tiles).  A cell holds sums for every token, to which an
// entry's are added with the tokens' weights when the warp leaves the entry.
template <int SH, int GW, bool ASYM>
__global__ void __launch_bounds__(MOE_EXPERT_THREADS, 1) moe_down_kernel(const MoeParams p) {
  constexpr int SLOT = W4Slot<GW, ASYM>::BYTES, RP = W4_RP;
  extern __shared__ __align__(16) char smem[];
  __shared__ W4Runs<MOE_WARPS> runs;
  const int tid = threadIdx.x, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);
  const int cell_floats = p.T * RP;
  float* cells = reinterpret_cast<float*>(smem);
  const uint32_t ring = smem_u32(smem + p.down_ring_at) + warp * MOE_DEPTH * SLOT;
  float* out = reinterpret_cast<float*>(smem + p.down_ring_at);  // [tile][token][row] over the ranks, after the rings
  const int nb = w4_units(p.F);
  const int rank = blockIdx.x % p.C, cluster = blockIdx.x / p.C, clusters = gridDim.x / p.C;
  const int tiles = (p.D + 15) / 16, t0 = (int)((int64_t)tiles * cluster / clusters);
  const int my_tiles = (int)((int64_t)tiles * (cluster + 1) / clusters) - t0;
  wait_for_previous_kernel();
  allow_dependent_launch();
  const int all = p.lists->active * nb, first = (int)((int64_t)all * rank / p.C);
  const int per_tile = (int)((int64_t)all * (rank + 1) / p.C) - first;
  const int64_t plane = (int64_t)p.T * p.top_k * p.F * 2;

  for (int p0 = 0; p0 < my_tiles; p0 += p.down_pass) {
    const int n_tiles = min(p.down_pass, my_tiles - p0), line = n_tiles * per_tile;
    if (p0 != 0) __syncthreads();
    if (line > 0) {
      const W4Run run = w4_runs<MOE_WARPS>(runs, line, per_tile, warp, lane);
        int tile = run.tile, at = run.b;  // block of the tile's line
      int a = (first + at) / nb, b = first + at - a * nb;
      float* cell = cells + run.cell * cell_floats;

      W4Base base{};
      base.row_bytes = (uint32_t)p.rb2;
      base.pitch = p.D;
      base.groups = p.g2;
        auto place = [&](int ti, int entry, int at_b) {
        const int64_t e = p.expert[entry];
        base.codes = p.w2 + e * p.D * p.rb2;
        base.scales = p.s2 + e * p.g2 * p.D;
        if (ASYM) base.zeros = p.z2 + e * p.g2 * p.D;
        const int row = (t0 + p0 + ti) * 16;
        return w4_place<GW, ASYM, true>(base, row, row + 8, p.D - 1, at_b, lane);
      };
      int to_load = run.units, load_tile = tile, load_at = at, load_a = a, load_b = b;
      W4Cursor cur{};
      if (to_load > 0) cur = place(tile, a, b);
      const bool odd = w4_blocks(p.F) % 2 != 0;  // the last unit of a row is half a one
      auto issue = [&](uint32_t into) {
        if (to_load > 0) {
          w4_issue<GW, ASYM, true>(into, base, cur, odd && load_b == nb - 1, lane);
          --to_load;
          ++load_at;
          if (++load_b == nb || load_at == per_tile) {
            load_b = 0;
            ++load_a;
            if (load_at == per_tile) {
              load_at = 0;
              ++load_tile;
              load_a = first / nb;
              load_b = first - load_a * nb;
            }
            if (to_load > 0) cur = place(load_tile, load_a, load_b);
          }
        }
        cp_commit();
      };
#pragma unroll 1
      for (int u = 0; u < MOE_DEPTH - 1; ++u) issue(ring + u * SLOT);

      float acc[MOE_NT][4] = {};
      const char* rows[MOE_NT];
      int s0 = 0, count = 0;
      bool begin = true, fresh = true;
      uint32_t slot = ring, spent = ring + (MOE_DEPTH - 1) * SLOT;
      for (int left = run.units; left > 0; --left) {
        if (fresh) {
          for (int i = lane; i < cell_floats; i += 32) cell[i] = 0.0f;
          __syncwarp();
          fresh = false;
        }
        if (begin) {
          s0 = p.start[a];
          count = p.start[a + 1] - s0;
#pragma unroll
          for (int n = 0; n < MOE_NT; ++n)
            rows[n] = reinterpret_cast<const char*>(p.h + (int64_t)(s0 + min(8 * n + g, count - 1)) * p.F);
          begin = false;
        }
        cp_wait<MOE_DEPTH - 2>();
        __syncwarp();
        issue(spent);
        moe_mac<SH, GW, ASYM>(acc, slot, lane, count, rows, plane, b, p.F);
        spent = slot;
        slot = slot == ring + (MOE_DEPTH - 1) * SLOT ? ring : slot + SLOT;
        ++at;
        if (++b == nb || at == per_tile || left == 1) {
#pragma unroll
          for (int n = 0; n < MOE_NT; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int m = 8 * n + 2 * t + c;
              if (m < count) {  // an entry's tokens differ, so no two lanes meet in a place
                const float w = p.slot_weight[s0 + m];
                float* q = cell + p.slot_token[s0 + m] * RP + g;
                q[0] = __fmaf_rn(w, acc[n][c], q[0]);
                q[8] = __fmaf_rn(w, acc[n][2 + c], q[8]);
              }
              acc[n][c] = acc[n][2 + c] = 0.0f;
            }
          }
          __syncwarp();
          b = 0;
          ++a;
          begin = true;
          if (at == per_tile) {
            at = 0;
            ++tile;
            a = first / nb;
            b = first - a * nb;
            cell += cell_floats;
            fresh = true;
          }
        }
      }
    }
    __syncthreads();
    const int outs = n_tiles * p.T * 16;
    const float inv_line = __frcp_rn((float)max(line, 1));
    for (int o = tid; o < outs; o += MOE_EXPERT_THREADS) {
      const int row = o % 16, mt = o / 16, ti = mt / p.T, m = mt - ti * p.T;
      float v = 0.0f;
      if (line > 0) {
        const int from = w4_first_cell<MOE_WARPS>(runs, ti, n_tiles, line, inv_line, per_tile);
        const int to = w4_first_cell<MOE_WARPS>(runs, ti + 1, n_tiles, line, inv_line, per_tile);
        for (int c = from; c < to; ++c) v = __fadd_rn(v, cells[c * cell_floats + m * RP + row]);
      }
      const int d = (t0 + p0 + ti) * 16 + row;
      if (p.C > 1) out[o] = v;
      else if (d < p.D) store_out(p.y, m * p.ldy + d, v, p.y_bf16);
    }
    if (p.C > 1) {
      cluster_sync();
      for (int o = rank * MOE_EXPERT_THREADS + tid; o < outs; o += p.C * MOE_EXPERT_THREADS) {
        const int row = o % 16, mt = o / 16, ti = mt / p.T, m = mt - ti * p.T;
        float v = ld_dsmem_f32(out + o, 0);
        for (int c = 1; c < p.C; ++c) v = __fadd_rn(v, ld_dsmem_f32(out + o, c));
        const int d = (t0 + p0 + ti) * 16 + row;
        if (d < p.D) store_out(p.y, m * p.ldy + d, v, p.y_bf16);
      }
      cluster_sync();  // no CTA leaves, or reuses its sums, while they are read
    }
  }
}

}  // namespace sqk

namespace sqh {
namespace {

cudaError_t launch_dependent(const void* kern, unsigned gx, unsigned gy, unsigned threads, size_t smem, int cluster,
                             const sqk::MoeParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(gx, gy);
  cfg.blockDim = dim3(threads);
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

constexpr int64_t kSmemBudget = 226 * 1024;  // of 227 KB; the rest covers the static arrays

template <int S, int SH, int GW, bool ASYM>
cudaError_t launch_experts(sqk::MoeParams p, cudaStream_t st) {
  const void* up = (const void*)sqk::moe_up_kernel<S, SH, GW, ASYM>;
  const void* down = (const void*)sqk::moe_down_kernel<SH, GW, ASYM>;
  for (const void* k : {up, down}) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBudget);
    if (e != cudaSuccess) return e;
  }
  const int64_t ring = (int64_t)sqk::MOE_WARPS * sqk::MOE_DEPTH * sqk::W4Slot<GW, ASYM>::BYTES;
  const int64_t sms = num_sms();
  // gate and up: as many tiles a pass as a CTA can have, as far as their cells fit beside x, and x in
  // shared memory if half the tiles (at least eight) still have cells
  const int64_t per = ((int64_t)std::min(p.E, p.T * p.top_k) * (p.F / 8) + sms - 1) / sms;
  const int64_t cell = (int64_t)std::min(p.T, sqk::MOE_ENTRY) * sqk::W4_RP * 4;
  const int64_t x = (int64_t)S * p.T * (sqk::w4_blocks(p.D) * 256 + 64);
  auto passes = [&](int64_t room, int64_t c, int64_t n) { return std::min(n, room / c - (sqk::MOE_WARPS - 1)); };
  p.x_staged = passes(kSmemBudget - ring - x, cell, per) >= std::min<int64_t>(per, std::max<int64_t>(8, per / 2));
  p.up_cells_at = p.x_staged ? (int)x : 0;
  p.up_pass = (int)passes(kSmemBudget - ring - p.up_cells_at, cell, per);
  p.up_ring_at = (int)(p.up_cells_at + (p.up_pass + sqk::MOE_WARPS - 1) * cell);
  cudaError_t e = launch_dependent(up, (unsigned)sms, 1, sqk::MOE_EXPERT_THREADS, (size_t)(p.up_ring_at + ring), 1, p, st);
  if (e != cudaSuccess) return e;

  const int64_t tiles = (p.D + 15) / 16, cell2 = (int64_t)p.T * sqk::W4_RP * 4;
  p.C = 1;
  while (p.C < 8 && tiles * p.C * 2 <= sms) p.C *= 2;
  int64_t clusters = std::min<int64_t>(tiles, sms / p.C);
  if (p.C > 1) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)p.C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(clusters * p.C));
    cfg.blockDim = dim3(sqk::MOE_EXPERT_THREADS);
    cfg.dynamicSmemBytes = (size_t)kSmemBudget;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int active = 0;
    e = max_active_clusters(down, &cfg, &active);
    if (e != cudaSuccess) return e;
    clusters = std::min<int64_t>(clusters, std::max(active, 1));
  }
  const int64_t per2 = (tiles + clusters - 1) / clusters;
  // the sums over the ranks take the rings' place
  p.down_pass = (int)std::min(passes(kSmemBudget - ring, cell2, per2), std::max<int64_t>(1, ring / ((int64_t)p.T * 64)));
  p.down_ring_at = (int)((p.down_pass + sqk::MOE_WARPS - 1) * cell2);
  return launch_dependent(down, (unsigned)(clusters * p.C), 1, sqk::MOE_EXPERT_THREADS, (size_t)(p.down_ring_at + ring), p.C, p,
                          st);
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
  const int64_t entries = std::min(T * k, E + T * k / sqk::MOE_ENTRY);  // every expert's last one may be short
  q.expert = (int*)take((size_t)entries * 4);
  q.start = (int*)take((size_t)(entries + 1) * 4);
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
    e = launch_dependent((const void*)sqk::moe_split_kernel, (unsigned)num_sms(), 1, 256, 0, 1, p, st);
    if (e != cudaSuccess) return e;
  }
  if (wr) {
    const void* k = bf16 ? (wr_bf16 ? (const void*)sqk::moe_router_kernel<true, true> : (const void*)sqk::moe_router_kernel<true, false>)
                         : (wr_bf16 ? (const void*)sqk::moe_router_kernel<false, true> : (const void*)sqk::moe_router_kernel<false, false>);
    e = launch_dependent(k, (unsigned)E, (unsigned)std::min<int64_t>(T, 8), sqk::MOE_THREADS, 0, 1, p, st);
  } else {
    e = launch_dependent((const void*)sqk::moe_lists_kernel, 1, 1, sqk::MOE_THREADS, 0, 1, p, st);
  }
  if (e != cudaSuccess) return e;
  return bf16 ? launch_experts_g<1, 2>(p, group, st) : launch_experts_g<3, 3>(p, group, st);
}

}  // namespace sqh
