// sq_moe.cu -- a whole mixture-of-experts layer for a few tokens, experts' weights in 4 bits.
//
//   logits[t, e] = sum_d x[t, d] Wr[e, d]     p = softmax(logits)     the k largest of each token
//   h[t, e, f]   = silu(W1_e[f] . x_t) * (W3_e[f] . x_t)
//   y[t]         = sum over the chosen e of weight[t, e] * (W2_e h[t, e])
//
// Bound: the chosen experts' codes, each read once from HBM.  Three kernels, chained as
// programmatic dependents: router and choice; gate and up; down.  The work is cut by (expert,
// rows), never by token: an expert's weights are read once for all of its tokens, which are the
// columns of the mma (sq_w4.cuh).
//   Router sums are binary64, so that which experts are chosen does not hang on rounding.  The last
// of the blocks that work on a token makes its choice; the lists are short enough that every CTA of the
// gate/up kernel builds them for itself.  h is kept as two bf16 parts (16 significant bits; three for a
// binary32 layer), so the only bf16 rounding of the layer is the final store.  Every sum has a fixed
// order; the only atomics are the lists' bit masks (order-free) and the router's arrival counts.  The
// expert kernels are one CTA per SM with the weight stream of sq_w4.cuh.
//
// Measured: 1 token, 8 of 128 experts, 2048 x 768 19 us (the three kernels' latencies: 5, 7 and 7); 1 token, 2 of 8
// experts, 4096 x 14336 57 us = 3.3 TB/s (gate/up 33, down 24); 32 tokens, 8 of 128 experts, 2048 x 768, group 64
// 106 us (gate/up 55, down 44).
#include <algorithm>

#include "sq_w4.cuh"

namespace sqk {

constexpr int MOE_MAX_T = 64;    // tokens: one bit each of an expert's token mask
constexpr int MOE_MAX_E = 1024;  // experts
constexpr int MOE_MAX_K = 32;    // choices per token

struct MoeParams {
  const char* x;
  int64_t ldx_bytes;
  const char* wr;
  int T, D, F, E, top_k, renorm;
  int* ids;
  float* wts;
  const int* ids_in;    // what the experts go by: ids and wts, or choices made elsewhere
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
  unsigned int* arrived;  // [8] router blocks that are done with 8 tokens; wrap to 0 by themselves
  double* logits;         // [T, E]
  int* lists;             // see MoeLists
  uint16_t* xparts;       // [3, T, D] (binary32 x)
  uint16_t* h;            // [parts, T k, F]
  // the expert kernels' shared memory
  int entries;          // most entries of the lists
  int entry;            // most tokens of one: 8 a column tile of the mma
  int up_x_at, up_cells_at, up_ring_at, up_pass;  // the lists come first; pass: tiles whose cells fit
  int down_h_at, down_cells_at, down_ring_at, down_pass;
  int C;                // CTAs of the down kernel's cluster
};

constexpr int MOE_DEPTH = 2;   // slots of a warp's ring
constexpr int MOE_WARPS = 16;  // of an expert kernel's CTA
constexpr int MOE_EXPERT_THREADS = 32 * MOE_WARPS;
constexpr int MOE_LOGIT_WARPS = 8;
constexpr int MOE_RP = 20;  // floats between the down kernel's tokens of a cell: 16 rows, padded to spread the banks

// ---------------------------------------------------------------------------- lists
// Entries (an expert and up to p.entry of its tokens), and slots (a token of an expert), which lie
// in the order of the experts and, for one expert, of the tokens.  All in one array of ints, so that
// the down kernel can copy it as it is.
struct MoeLists {
  int* active;  // number of entries
  int* expert;  // [entries]
  int* start;   // [entries + 1] first slot
  int* token;   // [T k] of a slot
  float* weight;
  __host__ __device__ MoeLists(int* at, int entries, int slots)
      : active(at), expert(at + 1), start(expert + entries), token(start + entries + 1),
        weight(reinterpret_cast<float*>(token + slots)) {}
  __host__ __device__ static int64_t ints(int64_t entries, int64_t slots) { return 2 + 2 * entries + 2 * slots; }
};

// What building them needs for a while.
struct MoeScratch {
  unsigned long long* mask;  // [E] tokens of an expert
  int* offset;               // [E] its first slot
  int* ids;                  // [T k]
  float* wts;                // [T k]
  __device__ MoeScratch(char* at, int E, int slots)
      : mask(reinterpret_cast<unsigned long long*>(at)), offset(reinterpret_cast<int*>(mask + E)), ids(offset + E),
        wts(reinterpret_cast<float*>(ids + slots)) {}
  __host__ __device__ static int64_t bytes(int64_t E, int64_t slots) { return 12 * E + 8 * slots; }
};

// Builds the lists from the choices in `sc` (a block of MOE_EXPERT_THREADS).  A choice outside
// [0, E) is left out; one that a token names twice counts once, with the weights' sum.
__device__ void moe_build_lists(const MoeParams& p, const MoeLists& l, const MoeScratch& sc, int* warp_sums) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  for (int e = tid; e < p.E; e += MOE_EXPERT_THREADS) sc.mask[e] = 0ull;
  __syncthreads();
  const int pairs = p.T * p.top_k;
  for (int i = tid; i < pairs; i += MOE_EXPERT_THREADS) {
    const int e = sc.ids[i];
    if (e >= 0 && e < p.E) atomicOr(&sc.mask[e], 1ull << (i / p.top_k));
  }
  __syncthreads();
  // exclusive sums of tokens (low half) and of entries (high half) over the experts, a run of them per
  // thread: at most 2048 of either
  const int per = (p.E + MOE_EXPERT_THREADS - 1) / MOE_EXPERT_THREADS;
  int mine = 0;
  for (int e = tid * per; e < min(p.E, (tid + 1) * per); ++e) {
    const int c = __popcll(sc.mask[e]);
    mine += c + ((c + p.entry - 1) / p.entry << 16);
  }
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  int before = sum - mine, total = 0;
  for (int w = 0; w < MOE_WARPS; ++w) {
    const int v = warp_sums[w];
    before += w < warp ? v : 0;
    total += v;
  }
  int tokens = before & 0xffff, active = before >> 16;
  for (int e = tid * per; e < min(p.E, (tid + 1) * per); ++e) {
    const int c = __popcll(sc.mask[e]);
    sc.offset[e] = tokens;
    for (int first = 0; first < c; first += p.entry) {
      l.expert[active] = e;
      l.start[active] = tokens + first;
      ++active;
    }
    tokens += c;
  }
  if (tid == 0) {
    *l.active = total >> 16;
    l.start[total >> 16] = total & 0xffff;
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += MOE_EXPERT_THREADS) {
    const int e = sc.ids[i], t = i / p.top_k, first = t * p.top_k;
    if (e < 0 || e >= p.E) continue;
    float w = 0.0f;
    bool earlier = false;
    for (int j = first; j < first + p.top_k; ++j) {
      if (sc.ids[j] != e) continue;
      earlier |= j < i;
      w = __fadd_rn(w, sc.wts[j]);
    }
    if (earlier) continue;
    const int slot = sc.offset[e] + __popcll(sc.mask[e] & ((1ull << t) - 1ull));
    l.token[slot] = t;
    l.weight[slot] = w;
  }
  __syncthreads();
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

// The k largest logits of one token, by one warp, PER of them a lane: ties to the lowest index, NaN
// ranks last.  Compared as integers of the same order (0: none, 1: NaN).
template <int PER>
__device__ void moe_choose(const MoeParams& p, int t, int lane) {
  const double* row = p.logits + (int64_t)t * p.E;
  double v[PER];
  unsigned long long key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = i * 32 + lane < p.E ? __ldcg(row + i * 32 + lane) : 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const unsigned long long b = (unsigned long long)__double_as_longlong(v[i]);
    key[i] = i * 32 + lane >= p.E ? 0ull : v[i] != v[i] ? 1ull : b >> 63 ? ~b : b | 1ull << 63;
  }
  double top = 0.0, best = 0.0, mine = 0.0;
  int my_id = 0;
  for (int j = 0; j < p.top_k; ++j) {
    unsigned long long k = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < PER; ++i) {
      at = key[i] > k ? i : at;
      k = key[i] > k ? key[i] : k;
    }
    const uint32_t hi = (uint32_t)(k >> 32), hi_max = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lo = hi == hi_max ? (uint32_t)k : 0u, lo_max = __reduce_max_sync(0xffffffffu, lo);
    const bool tied = hi == hi_max && (uint32_t)k == lo_max;
    const int id = (int)__reduce_min_sync(0xffffffffu, tied ? (uint32_t)(at * 32 + lane) : 0xffffffffu);
    const unsigned long long w = (unsigned long long)hi_max << 32 | lo_max;
    best = w == 1ull ? __longlong_as_double(0x7ff8000000000000ll)
                     : __longlong_as_double((long long)(w >> 63 ? w & ~(1ull << 63) : ~w));
    if (j == 0) top = best;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * 32 + lane == id) key[i] = 0ull;
    if (j == lane) {
      mine = best;
      my_id = id;
    }
  }
  double sum = 0.0;  // a NaN logit makes it, and so every weight, NaN
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i * 32 + lane < p.E) sum += (double)expf((float)(v[i] - top));
  sum = warp_sum(sum);
  const double w = lane < p.top_k ? (double)expf((float)(mine - top)) / sum : 0.0;
  const double chosen = p.renorm ? warp_sum(w) : 1.0;
  if (lane < p.top_k) {
    p.ids[t * p.top_k + lane] = my_id;
    p.wts[t * p.top_k + lane] = (float)(w / chosen);
  }
}

// Logits of EB experts and TB tokens by one block, its 8 warps and their lanes along D.  Bound by the
// conversions to binary64 (EB + TB of them for EB TB multiply-adds).  The last block to arrive for its
// tokens makes their choices, a warp each.
template <bool XB, bool RB, int EB, int TB>
__global__ void __launch_bounds__(32 * MOE_LOGIT_WARPS) moe_logits_kernel(const MoeParams p) {
  __shared__ double part[MOE_LOGIT_WARPS][EB * TB];
  __shared__ bool last;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int e0 = blockIdx.x * EB, t0 = blockIdx.y * TB;
  wait_for_previous_kernel();
  allow_dependent_launch();
  double sum[EB][TB] = {};
  for (int d = tid * 8; d < p.D; d += MOE_LOGIT_WARPS * 256) {
    float w[EB][8];
#pragma unroll
    for (int e = 0; e < EB; ++e)  // experts and tokens past the end repeat the last one, not stored
      load8<RB>(p.wr + ((int64_t)min(e0 + e, p.E - 1) * p.D + d) * (RB ? 2 : 4), w[e]);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      float x[8];
      load8<XB>(p.x + min(t0 + t, p.T - 1) * p.ldx_bytes + (int64_t)d * (XB ? 2 : 4), x);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < EB; ++e) sum[e][t] = fma((double)x[i], (double)w[e][i], sum[e][t]);
    }
  }
#pragma unroll
  for (int e = 0; e < EB; ++e)
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const double v = warp_sum(sum[e][t]);
      if (lane == 0) part[warp][e * TB + t] = v;
    }
  __syncthreads();
  if (tid < EB * TB) {
    double v = part[0][tid];
#pragma unroll
    for (int i = 1; i < MOE_LOGIT_WARPS; ++i) v += part[i][tid];
    const int e = e0 + tid / TB, t = t0 + tid % TB;
    if (e < p.E && t < p.T) p.logits[(int64_t)t * p.E + e] = v;
    __threadfence();
  }
  __syncthreads();
  if (tid == 0) last = atomicInc(p.arrived + blockIdx.y, gridDim.x - 1) == gridDim.x - 1;
  __syncthreads();
  if (!last || warp >= TB || t0 + warp >= p.T) return;
  __threadfence();
  if (p.E <= 32) moe_choose<1>(p, t0 + warp, lane);
  else if (p.E <= 128) moe_choose<4>(p, t0 + warp, lane);
  else if (p.E <= 256) moe_choose<8>(p, t0 + warp, lane);
  else moe_choose<MOE_MAX_E / 32>(p, t0 + warp, lane);
}

// The lists, by one CTA, from the choices in global memory.
__device__ __forceinline__ void moe_route(const MoeParams& p, const MoeLists& l, char* scratch, int* warp_sums) {
  const int pairs = p.T * p.top_k;
  if (p.T == 1) {  // every choice is an entry of its own, in the order of the choices; one warp sees them all
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x, e = lane < pairs ? p.ids_in[lane] : -1;
      const float mine = lane < pairs ? p.wts_in[lane] : 0.0f;
      const bool valid = e >= 0 && e < p.E;
      bool first = valid;
      float w = 0.0f;
      for (int j = 0; j < pairs; ++j) {
        const bool same = __shfl_sync(0xffffffffu, e, j) == e;
        const float v = __shfl_sync(0xffffffffu, mine, j);
        if (same) w = __fadd_rn(w, v);
        if (same && j < lane) first = false;
      }
      const uint32_t entries = __ballot_sync(0xffffffffu, first);
      const int at = __popc(entries & ((1u << lane) - 1u)), n = __popc(entries);
      if (first) {
        l.expert[at] = e;
        l.token[at] = 0;
        l.weight[at] = w;
      }
      if (lane <= n) l.start[lane] = lane;
      if (lane == 0) {
        *l.active = n;
        l.start[n] = n;
      }
    }
    __syncthreads();
    return;
  }
  const MoeScratch sc(scratch, p.E, pairs);
  for (int i = threadIdx.x; i < pairs; i += MOE_EXPERT_THREADS) {
    sc.ids[i] = p.ids_in[i];
    sc.wts[i] = p.wts_in[i];
  }
  moe_build_lists(p, l, sc, warp_sums);
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
// One unit for an entry of `count` <= 8 NTM tokens: as many column tiles as they need, or a single one
// that holds the parts of x beside each other where they fit (w4_part_column).  STAGED: rows are
// addresses in shared memory, padded with zeros to whole units; else they are read from global memory,
// `K` values of them.
template <bool STAGED, int S, int GW, bool ASYM, int NTM, typename Row>
__device__ __forceinline__ void moe_mac(float (&acc)[NTM][4], uint32_t slot, int lane, int count,
                                        const Row (&rows)[NTM], int64_t plane, int u, int K) {
  auto x = [&](int n, int s, int i) {
    if constexpr (STAGED) {
      return lds128(rows[n] + s * (uint32_t)plane + u * (2 * W4_UNIT) + i * 64);
    } else {
      const int k = u * W4_UNIT + (lane % 4) * 8 + 32 * i;
      return k < K ? *reinterpret_cast<const uint4*>(rows[n] + s * plane + k * 2) : make_uint4(0, 0, 0, 0);
    }
  };
  if (S > 1 && count <= w4_fold_columns(S)) w4_mac<1, 1, GW, ASYM>(acc, slot, lane, x);
  else if (NTM == 1 || count <= 8) w4_mac<1, S, GW, ASYM>(acc, slot, lane, x);
  else w4_mac<NTM, S, GW, ASYM>(acc, slot, lane, x);
}

// The row (token of the entry) and part that this lane's column n reads.
template <int S>
__device__ __forceinline__ int2 moe_column(int n, int g, int count) {
  if (S > 1 && count <= w4_fold_columns(S)) return make_int2(min(w4_part_column<S>(g).x, count - 1), w4_part_column<S>(g).y);
  return make_int2(min(8 * n + g, count - 1), 0);
}

template <bool STAGED>
struct MoeRow {
  using type = const char*;
  static __device__ __forceinline__ type of(uint32_t, const char* global, int) { return global; }
};
template <>
struct MoeRow<true> {
  using type = uint32_t;
  static __device__ __forceinline__ type of(uint32_t shared, const char*, int lane) { return shared + (lane % 4) * 16; }
};

// Bytes between staged rows of K bf16 numbers: whole units, rows 64 bytes apart modulo 128.
__host__ __device__ __forceinline__ int moe_row_pitch(int K) { return w4_units(K) * (2 * W4_UNIT) + 64; }

// Starts the copies of `rows` rows of K bf16 numbers (row r at src(r)) to shared memory, with zeros up to
// whole units.
template <typename Src>
__device__ __forceinline__ void moe_stage_rows(char* dst, int rows, int K, Src src) {
  const int pieces = w4_units(K) * (W4_UNIT / 8), pitch = moe_row_pitch(K);
  const float inv = __frcp_rn((float)pieces);
  for (int i = threadIdx.x; i < rows * pieces; i += MOE_EXPERT_THREADS) {
    const int r = w4_div(i, pieces, inv), v = i - r * pieces;
    if (v * 8 < K) cp_async16(smem_u32(dst + r * pitch + v * 16), src(r) + v * 16);
    else *reinterpret_cast<uint4*>(dst + r * pitch + v * 16) = make_uint4(0, 0, 0, 0);
  }
}

// Gate and up: a tile is 8 rows f of an entry's gate and the same 8 of its up projection, as the two
// halves of a 16-row tile, so one thread finds both sums of an h.  The tiles of all entries are one
// line, cut over the CTAs and there over the warps (sq_w4.cuh).
template <bool STAGED, int NTM, int S, int SH, int GW, bool ASYM>
__global__ void __launch_bounds__(MOE_EXPERT_THREADS, 1) moe_up_kernel(const MoeParams p) {
  constexpr int SLOT = W4Slot<GW, ASYM>::BYTES, CELL = w4_cell_floats(NTM);
  extern __shared__ __align__(16) char smem[];
  __shared__ W4Runs<MOE_WARPS> runs;
  __shared__ int warp_sums[MOE_WARPS];
  const int tid = threadIdx.x, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);
  float* cells = reinterpret_cast<float*>(smem + p.up_cells_at);
  const uint32_t ring = smem_u32(smem + p.up_ring_at) + warp * MOE_DEPTH * SLOT;
  const int nb = w4_units(p.D), per_expert = p.F / 8;
  const int spitch = moe_row_pitch(p.D);
  char* xs = smem + p.up_x_at;
  const int slots = p.T * p.top_k;
  const MoeLists l(reinterpret_cast<int*>(smem), p.entries, slots);
  wait_for_previous_kernel();
  allow_dependent_launch();
  if (STAGED && S == 1) moe_stage_rows(xs, p.T, p.D, [&](int r) { return p.x + r * p.ldx_bytes; });
  cp_commit();
  moe_route(p, l, smem + p.up_ring_at, warp_sums);
  if (blockIdx.x == 0)  // for the down kernel
    for (int i = tid; i < MoeLists::ints(p.entries, slots); i += MOE_EXPERT_THREADS)
      p.lists[i] = reinterpret_cast<const int*>(smem)[i];
  const uint32_t tiles = (uint32_t)*l.active * per_expert;
  const int64_t t0 = w4_part(blockIdx.x, tiles / gridDim.x, tiles % gridDim.x);
  const int my_tiles = tiles / gridDim.x + (blockIdx.x < tiles % gridDim.x);
  const char* xbase = S == 1 ? p.x : reinterpret_cast<const char*>(p.xparts);
  const int64_t xpitch = S == 1 ? p.ldx_bytes : (int64_t)p.D * 2;
  const int64_t xplane = S == 1 ? 0 : (int64_t)p.T * p.D * 2;
  for (int p0 = 0; p0 < my_tiles; p0 += p.up_pass) {
    const int n_tiles = min(p.up_pass, my_tiles - p0), line = n_tiles * nb;
    __syncthreads();  // the last pass's cells have been read, and the route's scratch, where the rings are
    const W4Run run = w4_runs<MOE_WARPS>(runs, line, nb, warp, lane);
    int tile = run.tile, b = run.b;
    float* cell = cells + run.cell * CELL;

    W4Base base{};
    base.row_bytes = (uint32_t)p.rb13;
    base.pitch = 2 * p.F;
    base.groups = p.g13;
    auto place = [&](int ti, int at_b) {
      const uint32_t at = (uint32_t)t0 + p0 + ti;  // of the tiles of all entries, below 2^32
      const int a = (int)(at / (uint32_t)per_expert), f0 = (int)(at - a * per_expert) * 8;
      const int64_t e = l.expert[a];
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
    if (STAGED && S > 1 && p0 == 0) {
      const int pieces = nb * (W4_UNIT / 8);
      const float inv = __frcp_rn((float)pieces);
      for (int i = tid; i < p.T * pieces; i += MOE_EXPERT_THREADS) {
        const int m = w4_div(i, pieces, inv), v = i - m * pieces;
        const float* src = reinterpret_cast<const float*>(p.x + m * p.ldx_bytes);
        float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (v * 8 < p.D) load8<false>(reinterpret_cast<const char*>(src + v * 8), f);
        uint32_t part[8][S];
#pragma unroll
        for (int e = 0; e < 8; ++e) split_bf16<S>(f[e], part[e]);
#pragma unroll
        for (int s = 0; s < S; ++s)
          *reinterpret_cast<uint4*>(xs + (s * p.T + m) * spitch + v * 16) =
              make_uint4(part[0][s] | (part[1][s] << 16), part[2][s] | (part[3][s] << 16),
                         part[4][s] | (part[5][s] << 16), part[6][s] | (part[7][s] << 16));
      }
    }
    cp_wait<MOE_DEPTH - 1>();  // x; the ring's units are younger
    __syncthreads();

    float acc[NTM][4] = {};
    typename MoeRow<STAGED>::type rows[NTM];
    int count = 0;
    bool begin = true;
    uint32_t slot = ring, spent = ring + (MOE_DEPTH - 1) * SLOT;
    for (int left = run.units; left > 0; --left) {
      if (begin) {
        const int a = (int)(((uint32_t)t0 + p0 + tile) / (uint32_t)per_expert), s0 = l.start[a];
        count = l.start[a + 1] - s0;
#pragma unroll
        for (int n = 0; n < NTM; ++n) {
          const int2 col = moe_column<S>(n, g, count);
          const int tok = l.token[s0 + col.x];
          rows[n] = MoeRow<STAGED>::of(smem_u32(xs) + (col.y * p.T + tok) * spitch, xbase + tok * xpitch + col.y * xplane, lane);
        }
        begin = false;
      }
      cp_wait<MOE_DEPTH - 2>();
      __syncwarp();
      issue(spent);
      moe_mac<STAGED, S, GW, ASYM>(acc, slot, lane, count, rows, STAGED ? (int64_t)p.T * spitch : xplane, b, p.D);
      spent = slot;
      slot = slot == ring + (MOE_DEPTH - 1) * SLOT ? ring : slot + SLOT;
      if (++b == nb || left == 1) {
        if (S > 1 && count <= w4_fold_columns(S)) w4_fold<S>(acc[0], lane);
        if (NTM == 1 || count <= 8) w4_put_cell<1>(cell, acc, lane);
        else w4_put_cell<NTM>(cell, acc, lane);
        cell += CELL;
#pragma unroll
        for (int n = 0; n < NTM; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
        b = 0;
        ++tile;
        begin = true;
      }
    }
    __syncthreads();
    const float inv_line = __frcp_rn((float)line);
    constexpr int COLS = 8 * NTM;  // 8 rows f x COLS tokens a tile
    const int f = tid % 8, m = tid / 8 % COLS;
    for (int ti = tid / (8 * COLS); ti < n_tiles; ti += MOE_EXPERT_THREADS / (8 * COLS)) {
      const int a = (int)(((uint32_t)t0 + p0 + ti) / (uint32_t)per_expert), s0 = l.start[a];
      if (m >= l.start[a + 1] - s0) continue;
      const int from = w4_first_cell<MOE_WARPS>(runs, ti, n_tiles, line, inv_line, nb);
      const int to = w4_first_cell<MOE_WARPS>(runs, ti + 1, n_tiles, line, inv_line, nb);
      const float* q = cells + from * CELL + f * COLS + m;
      float gate = 0.0f, up = 0.0f;
      for (int c = from; c < to; ++c, q += CELL) {
        gate = __fadd_rn(gate, q[0]);
        up = __fadd_rn(up, q[8 * COLS]);
      }
      // silu(v) = v / (1 + exp(-v)); exp overflows to inf for very negative v, and v / inf is -0
      const float h = __fmul_rn(__fdiv_rn(gate, __fadd_rn(1.0f, expf(-gate))), up);
      uint32_t part[SH];
      split_bf16_stored<SH>(h, part);
      const int64_t ff = (t0 + p0 + ti - (int64_t)a * per_expert) * 8 + f;
#pragma unroll
      for (int s = 0; s < SH; ++s) p.h[((int64_t)s * p.T * p.top_k + s0 + m) * p.F + ff] = (uint16_t)part[s];
    }
  }
  cp_wait_all();  // a block without tiles has not waited for x
}

// Down: a tile is 16 rows d; its units are those of every entry in turn (a rank of a cluster takes
// a share of that line, where there are few tiles).  A cell holds sums for every token, to which an
// entry's are added with the tokens' weights when the warp leaves the entry.
template <bool STAGED, int NTM, int SH, int GW, bool ASYM>
__global__ void __launch_bounds__(MOE_EXPERT_THREADS, 1) moe_down_kernel(const MoeParams p) {
  constexpr int SLOT = W4Slot<GW, ASYM>::BYTES, RP = MOE_RP;
  extern __shared__ __align__(16) char smem[];
  __shared__ W4Runs<MOE_WARPS> runs;
  const int tid = threadIdx.x, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);
  const int cell_floats = p.T * RP;
  float* cells = reinterpret_cast<float*>(smem + p.down_cells_at);
  const uint32_t ring = smem_u32(smem + p.down_ring_at) + warp * MOE_DEPTH * SLOT;
  float* out = reinterpret_cast<float*>(smem + p.down_ring_at);  // [tile][token][row] over the ranks, after the rings
  const int nb = w4_units(p.F);
  const int rank = blockIdx.x % p.C, cluster = blockIdx.x / p.C, clusters = gridDim.x / p.C;
  const int tiles = (p.D + 15) / 16, t0 = (int)((int64_t)tiles * cluster / clusters);
  const int my_tiles = (int)((int64_t)tiles * (cluster + 1) / clusters) - t0;
  wait_for_previous_kernel();
  allow_dependent_launch();
  const int slots = p.T * p.top_k;
  const MoeLists l(reinterpret_cast<int*>(smem), p.entries, slots);
  for (int i = tid; i < MoeLists::ints(p.entries, slots); i += MOE_EXPERT_THREADS)
    reinterpret_cast<int*>(smem)[i] = p.lists[i];
  __syncthreads();
  const int all = *l.active * nb, first = (int)((int64_t)all * rank / p.C);
  const int per_tile = (int)((int64_t)all * (rank + 1) / p.C) - first;
  const int64_t hplane = (int64_t)slots * p.F * 2;
  const int spitch = moe_row_pitch(p.F);
  char* hs = smem + p.down_h_at;  // rows of every slot, part after part
  for (int p0 = 0; p0 < my_tiles; p0 += p.down_pass) {
    const int n_tiles = min(p.down_pass, my_tiles - p0), line = n_tiles * per_tile;
    if (p0 != 0) __syncthreads();
    if (line > 0) {
      const W4Run run = w4_runs<MOE_WARPS>(runs, line, per_tile, warp, lane);
      int tile = run.tile, at = run.b;  // unit of the tile's line
      int a = (first + at) / nb, b = first + at - a * nb;
      float* cell = cells + run.cell * cell_floats;

      W4Base base{};
      base.row_bytes = (uint32_t)p.rb2;
      base.pitch = p.D;
      base.groups = p.g2;
      auto place = [&](int ti, int entry, int at_b) {
        const int64_t e = l.expert[entry];
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

      if (STAGED && p0 == 0) {
        const int used = l.start[*l.active];
        for (int s = 0; s < SH; ++s)
          moe_stage_rows(hs + s * slots * spitch, used, p.F,
                         [&](int r) { return reinterpret_cast<const char*>(p.h) + s * hplane + (int64_t)r * p.F * 2; });
      }
      cp_wait_all();  // h, and the ring's first units with it
      __syncthreads();

      float acc[NTM][4] = {};
      typename MoeRow<STAGED>::type rows[NTM];
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
          s0 = l.start[a];
          count = l.start[a + 1] - s0;
#pragma unroll
          for (int n = 0; n < NTM; ++n) {
            const int2 col = moe_column<SH>(n, g, count);
            const int row = s0 + col.x;
            rows[n] = MoeRow<STAGED>::of(smem_u32(hs) + (col.y * slots + row) * spitch,
                                         reinterpret_cast<const char*>(p.h) + col.y * hplane + (int64_t)row * p.F * 2,
                                         lane);
          }
          begin = false;
        }
        cp_wait<MOE_DEPTH - 2>();
        __syncwarp();
        issue(spent);
        moe_mac<STAGED, SH, GW, ASYM>(acc, slot, lane, count, rows, STAGED ? (int64_t)slots * spitch : hplane, b, p.F);
        spent = slot;
        slot = slot == ring + (MOE_DEPTH - 1) * SLOT ? ring : slot + SLOT;
        ++at;
        if (++b == nb || at == per_tile || left == 1) {
          if (count <= w4_fold_columns(SH)) w4_fold<SH>(acc[0], lane);
#pragma unroll
          for (int n = 0; n < NTM; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int m = 8 * n + 2 * t + c;
              if (m < count) {  // an entry's tokens differ, so no two lanes meet in a place
                const float w = l.weight[s0 + m];
                float* q = cell + l.token[s0 + m] * RP + g;
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

int64_t up16(int64_t v) { return (v + 15) & ~(int64_t)15; }

constexpr int64_t kSmemBudget = 226 * 1024;  // of 227 KB; the rest covers the static arrays

// Tiles of a pass whose cells fit in `room`.
int64_t moe_pass(int64_t room, int64_t cell, int64_t tiles) {
  return std::min(tiles, room / cell - (sqk::MOE_WARPS - 1));
}

template <int NTM, int S, int SH, int GW, bool ASYM>
cudaError_t launch_experts_t(sqk::MoeParams p, cudaStream_t st) {
  const int64_t ring = (int64_t)sqk::MOE_WARPS * sqk::MOE_DEPTH * sqk::W4Slot<GW, ASYM>::BYTES;
  const int64_t slots = (int64_t)p.T * p.top_k, lists = up16(sqk::MoeLists::ints(p.entries, slots) * 4);
  const int64_t rings = std::max(ring, up16(sqk::MoeScratch::bytes(p.E, slots)));  // the lists' scratch comes before
  const int64_t sms = num_sms();
  auto prepare = [](const void* k) { return allow_shared_memory(k, kSmemBudget); };
  // gate and up: as many tiles a pass as a CTA can have, as far as their cells fit beside x, and x in
  // shared memory if sixteen tiles still have cells
  const int64_t per = ((int64_t)std::min(p.E, p.T * p.top_k) * (p.F / 8) + sms - 1) / sms;
  const int64_t cell = (int64_t)sqk::w4_cell_floats(NTM) * 4, x = (int64_t)S * p.T * sqk::moe_row_pitch(p.D);
  const bool x_staged =
      moe_pass(kSmemBudget - lists - rings - x, cell, per) >= std::min<int64_t>(per, 16);
  p.up_x_at = (int)lists;
  p.up_cells_at = (int)(lists + (x_staged ? x : 0));
  p.up_pass = (int)moe_pass(kSmemBudget - rings - p.up_cells_at, cell, per);
  p.up_ring_at = (int)(p.up_cells_at + (p.up_pass + sqk::MOE_WARPS - 1) * cell);
  cudaError_t e = cudaSuccess;
  if (S > 1 && !x_staged) {
    e = launch_dependent((const void*)sqk::moe_split_kernel, (unsigned)sms, 1, 256, 0, 1, p, st);
    if (e != cudaSuccess) return e;
  }
  const void* up = x_staged ? (const void*)sqk::moe_up_kernel<true, NTM, S, SH, GW, ASYM>
                            : (const void*)sqk::moe_up_kernel<false, NTM, S, SH, GW, ASYM>;
  e = prepare(up);
  if (e != cudaSuccess) return e;
  e = launch_dependent(up, (unsigned)sms, 1, sqk::MOE_EXPERT_THREADS, (size_t)(p.up_ring_at + rings), 1, p, st);
  if (e != cudaSuccess) return e;

  // down: 16-row tiles; clusters cut an entry line where there are few of them
  const int64_t tiles = (p.D + 15) / 16, cell2 = (int64_t)p.T * sqk::MOE_RP * 4;
  p.C = 1;
  while (p.C < 8 && tiles * p.C * 2 <= sms) p.C *= 2;
  const int64_t h = (int64_t)SH * slots * sqk::moe_row_pitch(p.F);
  const bool h_staged = moe_pass(kSmemBudget - lists - ring - h, cell2, 2) >= 2;
  const void* down = h_staged ? (const void*)sqk::moe_down_kernel<true, NTM, SH, GW, ASYM>
                              : (const void*)sqk::moe_down_kernel<false, NTM, SH, GW, ASYM>;
  e = prepare(down);
  if (e != cudaSuccess) return e;
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
  p.down_h_at = (int)lists;
  p.down_cells_at = (int)(lists + (h_staged ? h : 0));
  // the sums over the ranks take the rings' place
  p.down_pass = (int)std::min(moe_pass(kSmemBudget - p.down_cells_at - ring, cell2, per2),
                              std::max<int64_t>(1, ring / ((int64_t)p.T * 64)));
  p.down_ring_at = (int)(p.down_cells_at + (p.down_pass + sqk::MOE_WARPS - 1) * cell2);
  return launch_dependent(down, (unsigned)(clusters * p.C), 1, sqk::MOE_EXPERT_THREADS, (size_t)(p.down_ring_at + ring),
                          p.C, p, st);
}

// Entries of 8 tokens (one column tile) where an expert has few on average, else of 16.  An expert with
// more tokens than an entry is read again for the next, from L2.
template <int S, int SH, int GW, bool ASYM>
cudaError_t launch_experts(sqk::MoeParams p, cudaStream_t st) {
  return p.entry == 8 ? launch_experts_t<1, S, SH, GW, ASYM>(p, st) : launch_experts_t<2, S, SH, GW, ASYM>(p, st);
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
  q.entry = T <= 8 || T * k <= 4 * E ? 8 : 16;
  q.entries = (int)std::min(T * k, E + T * k / q.entry);  // every expert's last entry may be short
  q.arrived = (unsigned int*)take(8 * sizeof(unsigned int));
  q.logits = (double*)take((size_t)(T * E) * 8);
  // (room for entries of 8 in any case, so that the size grows with each of its arguments)
  q.lists = (int*)take((size_t)sqk::MoeLists::ints(std::min(T * k, E + T * k / 8), T * k) * 4);
  q.xparts = (uint16_t*)take((size_t)(3 * T * D) * 2);
  q.h = (uint16_t*)take((size_t)(3 * T * k * F) * 2);
  if (p) {
    p->entries = q.entries;
    p->entry = q.entry;
    p->arrived = q.arrived;
    p->logits = q.logits;
    p->lists = q.lists;
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
  p.T = (int)T;
  p.D = (int)D;
  p.F = (int)F;
  p.E = (int)E;
  p.top_k = (int)top_k;
  p.renorm = renorm;
  p.ids = ids;
  p.wts = wts;
  p.ids_in = wr ? ids : ids_in;
  p.wts_in = wr ? wts : wts_in;
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
  if (wr) {
    // one token: a block per expert; more: blocks of 4 experts and 8 tokens
    const void* k;
    if (T == 1)
      k = bf16 ? (wr_bf16 ? (const void*)sqk::moe_logits_kernel<true, true, 1, 1> : (const void*)sqk::moe_logits_kernel<true, false, 1, 1>)
               : (wr_bf16 ? (const void*)sqk::moe_logits_kernel<false, true, 1, 1> : (const void*)sqk::moe_logits_kernel<false, false, 1, 1>);
    else
      k = bf16 ? (wr_bf16 ? (const void*)sqk::moe_logits_kernel<true, true, 4, 8> : (const void*)sqk::moe_logits_kernel<true, false, 4, 8>)
               : (wr_bf16 ? (const void*)sqk::moe_logits_kernel<false, true, 4, 8> : (const void*)sqk::moe_logits_kernel<false, false, 4, 8>);
    const unsigned eb = T == 1 ? 1 : 4, tb = T == 1 ? 1 : 8;
    const cudaError_t e = launch_dependent(k, ((unsigned)E + eb - 1) / eb, ((unsigned)T + tb - 1) / tb,
                                           32 * sqk::MOE_LOGIT_WARPS, 0, 1, p, st);
    if (e != cudaSuccess) return e;
  }
  return bf16 ? launch_experts_g<1, 2>(p, group, st) : launch_experts_g<3, 3>(p, group, st);
}

}  // namespace sqh
