// sq_w4_gemm.cu -- x [M, K] times 4-bit weights [N, K] with group scales, for a few tokens.
//
// y[m, n] = sum_g scale[g, n] * sum_{k in g} (code[n, k] - zero[g, n]) * x[m, k]
//
// Bound: the weight codes' K N / 2 bytes from HBM; at a few tokens every other term is small.  So
// the codes go from memory through a small ring in shared memory to registers once, copied
// asynchronously a unit ahead (sq_w4.cuh), and are turned into bf16 operands there (exact small
// integers).  The products run on mma.sync: its operands are registers, which is where the codes are
// unpacked, and at M <= 8 one 16 x 8 x 16 step consumes 256 weights, so the tensor pipe is far from
// its limit.  (For more tokens the operands go to tensor memory and tcgen05: sq_w4_tc.cu.)
//
// One CTA per SM (or cluster of CTAs, which then cut K between them because there are few rows or
// x is long) owns a run of 16-row tiles.  Its list of (tile, unit) is cut into 16 equal runs, one a
// warp, whatever the sizes; a warp streams its run through its ring without a pause (sq_w4.cuh).
// x is staged in shared memory once, as bf16 parts (one for bf16, three for binary32, which together
// are x exactly); where it does not fit it comes in chunks of K.  A warp's sum over its part of a
// tile goes to a cell of its own, and the cells of a tile are added in order at the end (and over
// the cluster through distributed shared memory): no atomics, no workspace.
//
// Measured (bf16 x, group 128): 1 x 6144 x 4096 6.4 us, 1 x 4096 x 14336 11.1, 8 x 28672 x 4096 19.0,
// 1 x 128256 x 4096 59 us = 4.7 TB/s of codes and scales; 7 x 12288 x 12288, group 64 with zero points, 26.5.
// A block of 16 x 128 codes takes 58 to 61 clocks of an SM, against 46 in which HBM delivers it (sq_w4.cuh has why).
#include <algorithm>

#include "sq_w4.cuh"

namespace sqk {

constexpr int W4G_WARPS = 16;  // of a CTA
constexpr int W4G_DEPTH = 2;   // slots of a warp's ring

struct W4GemmParams {
  const char* x;
  int64_t ldx_bytes;
  int M, K;
  W4Base w;
  int64_t N;
  void* y;
  int64_t ldy;
  int y_bf16;
  int C;         // CTAs of a cluster, over K
  int clusters;  // of the grid, over the tiles
  int units;     // of K
  bool odd;      // the last one has one block
  int tile_q, tile_r;    // tiles / clusters and the remainder: the first tile_r clusters have one more
  int unit_q, unit_r;    // the same for the units of K over the ranks
  int chunk;     // units of x staged at a time
  int pass;      // tiles whose partial sums fit
  int out_at, cell_at, ring_at;  // shared memory: x, then sums over chunks or ranks, cells, rings (sums
                                 // that no chunk adds to take the rings' place when those are empty)
};

template <int NT, int S, int GW, bool ASYM, bool ALIGNED>
__global__ void __launch_bounds__(32 * W4G_WARPS, 1) w4_gemm_kernel(const W4GemmParams p) {
  constexpr int WARPS = W4G_WARPS, THREADS = 32 * WARPS, DEPTH = W4G_DEPTH, SLOT = W4Slot<GW, ASYM>::BYTES, CELL = w4_cell_floats(NT);
  extern __shared__ __align__(16) char smem[];
  __shared__ W4Runs<WARPS> runs;
  const int tid = threadIdx.x, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);  // the same in every lane, and known to be
  const int rank = blockIdx.x % p.C, cluster = blockIdx.x / p.C;
  const int m0 = blockIdx.y * 8 * NT, Mr = min(8 * NT, p.M - m0);
  const int b0 = (int)w4_part(rank, p.unit_q, p.unit_r), b1 = b0 + p.unit_q + (rank < p.unit_r);
  const int64_t t0 = w4_part(cluster, p.tile_q, p.tile_r);
  const int my_tiles = p.tile_q + (cluster < p.tile_r);
  const uint32_t last_row = (uint32_t)min(p.N - 1 - t0 * 16, (int64_t)my_tiles * 16 - 1);
  float* out = reinterpret_cast<float*>(smem + p.out_at);     // [tile of the pass][token][row]
  float* cells = reinterpret_cast<float*>(smem + p.cell_at);  // [cell][row][8 NT]
  const uint32_t ring = smem_u32(smem + p.ring_at) + warp * DEPTH * SLOT;
  W4Base base = p.w;
  base.codes += t0 * 16 * base.row_bytes;
  base.scales += t0 * 16;
  if (ASYM) base.zeros += t0 * 16;

  wait_for_previous_kernel();
  allow_dependent_launch();

  const int pitch = p.chunk * (2 * W4_UNIT) + 64;  // bytes per staged token: rows 64 bytes apart modulo 128
  uint32_t xs[NT];                       // this lane's columns (addresses); absent tokens read the last one
#pragma unroll
  for (int n = 0; n < NT; ++n) xs[n] = smem_u32(smem) + min(8 * n + g, Mr - 1) * pitch + t * 16;
  const bool fold = S > 1 && NT == 1 && Mr <= w4_fold_columns(S);  // the parts of x beside each other
  if (fold) xs[0] = smem_u32(smem) + (w4_part_column<S>(g).y * Mr + min(w4_part_column<S>(g).x, Mr - 1)) * pitch + t * 16;
  const int plane = Mr * pitch;
  const bool whole = p.chunk >= b1 - b0;

  for (int p0 = 0; p0 < my_tiles; p0 += p.pass) {
    const int n_tiles = min(p.pass, my_tiles - p0);
    for (int c0 = b0; c0 < b1; c0 += p.chunk) {
      const int units = min(p.chunk, b1 - c0), line = n_tiles * units;
      if (c0 != b0 || p0 != 0) __syncthreads();  // x, the cells and the sums of the last turn have been read
      const bool stage = !whole || p0 == 0;
      const int vecs = units * (W4_UNIT / 8);  // 8-value pieces per token
      const float inv_vecs = __frcp_rn((float)vecs);
      if (S == 1 && stage) {
        const char* src = p.x + m0 * p.ldx_bytes + (int64_t)c0 * W4_UNIT * 2;
        for (int i = tid; i < Mr * vecs; i += THREADS) {
          const int m = w4_div(i, vecs, inv_vecs), v = i - m * vecs;
          if (c0 * W4_UNIT + v * 8 < p.K) cp_async16(smem_u32(smem + m * pitch + v * 16), src + m * p.ldx_bytes + v * 16);
          else *reinterpret_cast<uint4*>(smem + m * pitch + v * 16) = make_uint4(0, 0, 0, 0);
        }
      }
      cp_commit();
      {
        const W4Run run = w4_runs<WARPS>(runs, line, units, warp, lane);
        int b = run.b, left = run.units;
        float* cell = cells + run.cell * CELL;

        int to_load = left, load_tile = run.tile, load_b = units - b;
        W4Cursor cur = w4_place<GW, ASYM, ALIGNED>(base, (p0 + load_tile) * 16, (p0 + load_tile) * 16 + 8, last_row, c0 + b, lane);
        const bool odd = p.odd && c0 + units == p.units;  // the last unit of a row is half a one
        auto issue = [&](uint32_t into) {
          if (to_load > 0) {
            w4_issue<GW, ASYM, ALIGNED>(into, base, cur, odd && load_b == 1, lane);
            --to_load;
            if (--load_b == 0) {
              load_b = units;
              ++load_tile;
              const uint32_t row = (p0 + load_tile) * 16;
              cur = w4_place<GW, ASYM, ALIGNED>(base, row, row + 8, last_row, c0, lane);
            }
          }
          cp_commit();
        };
#pragma unroll 1
        for (int u = 0; u < DEPTH - 1; ++u) issue(ring + u * SLOT);
        if (S > 1 && stage) {
          const char* src = p.x + m0 * p.ldx_bytes + (int64_t)c0 * W4_UNIT * 4;
          for (int i = tid; i < Mr * vecs; i += THREADS) {
            const int m = w4_div(i, vecs, inv_vecs), v = i - m * vecs;
            float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (c0 * W4_UNIT + v * 8 < p.K) {
              const float4* at = reinterpret_cast<const float4*>(src + m * p.ldx_bytes + v * 32);
              *reinterpret_cast<float4*>(f) = at[0];
              *reinterpret_cast<float4*>(f + 4) = at[1];
            }
            uint32_t part[8][S];
#pragma unroll
            for (int e = 0; e < 8; ++e) split_bf16<S>(f[e], part[e]);
#pragma unroll
            for (int s = 0; s < S; ++s)
              *reinterpret_cast<uint4*>(smem + m * pitch + v * 16 + s * plane) =
                  make_uint4(part[0][s] | (part[1][s] << 16), part[2][s] | (part[3][s] << 16),
                             part[4][s] | (part[5][s] << 16), part[6][s] | (part[7][s] << 16));
          }
        }
        cp_wait<DEPTH - 1>();  // x; the ring's units are younger
        __syncthreads();

        float acc[NT][4];
#pragma unroll
        for (int k = 0; k < NT; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.0f;
        uint32_t slot = ring, spent = ring + (DEPTH - 1) * SLOT;  // the next unit's, the last one's
        uint32_t xo = b * (2 * W4_UNIT);
        while (left > 0) {
          const int part = min(left, units - b);  // of the tile
          left -= part;
#pragma unroll 1
          for (int i = 0; i < part; ++i) {
            cp_wait<DEPTH - 2>();
            __syncwarp();
            issue(spent);
            auto x = [&](int k, int s, int w) { return lds128(xs[k] + xo + s * plane + w * 64); };
            if (S > 1 && NT == 1 && fold) w4_mac<1, 1, GW, ASYM>(acc, slot, lane, x);
            else w4_mac<NT, S, GW, ASYM>(acc, slot, lane, x);
            spent = slot;
            slot = slot == ring + (DEPTH - 1) * SLOT ? ring : slot + SLOT;
            xo += 2 * W4_UNIT;
          }
          {  // the end of this warp's part of the tile
            if (S > 1 && NT == 1 && fold) w4_fold<S>(acc[0], lane);
            w4_put_cell<NT>(cell, acc, lane);
            cell += CELL;
#pragma unroll
            for (int k = 0; k < NT; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.0f;
            b = 0;
            xo = 0;
          }
        }
      }
      __syncthreads();
      // 16 rows x 8 NT tokens a tile
      const float inv_line = __frcp_rn((float)line);
      const bool last = c0 + p.chunk >= b1;
      const int row = tid % 16, m = tid / 16 % (8 * NT);
      for (int ti = tid / (128 * NT); ti < n_tiles; ti += THREADS / (128 * NT)) {
        const int from = w4_first_cell<WARPS>(runs, ti, n_tiles, line, inv_line, units);
        const int to = w4_first_cell<WARPS>(runs, ti + 1, n_tiles, line, inv_line, units);
        if (m >= Mr) continue;
        const float* q = cells + from * CELL + row * (8 * NT) + m;
        const int o = (ti * Mr + m) * 16 + row;
        float v = c0 == b0 ? 0.0f : out[o];
        for (int c = from; c < to; ++c, q += CELL) v = __fadd_rn(v, *q);
        const int64_t n = (t0 + p0 + ti) * 16 + row;
        if (p.C > 1 || !last) out[o] = v;
        else if (n < p.N) store_out(p.y, (m0 + m) * p.ldy + n, v, p.y_bf16);
      }
    }
    if (p.C > 1) {
      cluster_sync();
      const int outs = n_tiles * Mr * 16;
      const float inv_Mr = __frcp_rn((float)Mr);
      for (int o = rank * THREADS + tid; o < outs; o += p.C * THREADS) {
        const int row = o % 16, mt = o / 16, ti = w4_div(mt, Mr, inv_Mr), m = mt - ti * Mr;
        float v = ld_dsmem_f32(out + o, 0);
        for (int c = 1; c < p.C; ++c) v = __fadd_rn(v, ld_dsmem_f32(out + o, c));
        const int64_t n = (t0 + p0 + ti) * 16 + row;
        if (n < p.N) store_out(p.y, (m0 + m) * p.ldy + n, v, p.y_bf16);
      }
      cluster_sync();  // no CTA leaves, or reuses its sums, while they are read
    }
  }
}

}  // namespace sqk

namespace sqh {
cudaError_t launch_w4_tc(const void* x, bool bf16, int64_t M, int64_t K, int64_t ldx, const uint8_t* wq,
                         const uint16_t* sg, const uint8_t* zp, int64_t N, int group, void* y, bool y_bf16, int64_t ldy,
                         bool* taken, cudaStream_t st);

namespace {

constexpr int64_t kSmemBudget = 226 * 1024;  // of 227 KB; the rest covers the static arrays

template <int NT, int S, int GW, bool ASYM, bool ALIGNED>
cudaError_t launch_w4_gemm_t(sqk::W4GemmParams p, cudaStream_t st) {
  constexpr int WARPS = sqk::W4G_WARPS;
  auto kern = sqk::w4_gemm_kernel<NT, S, GW, ASYM, ALIGNED>;
  const int64_t tiles = (p.N + 15) / 16, mt = (p.M + 8 * NT - 1) / (8 * NT);
  const int nu = sqk::w4_units(p.K), mr = std::min(p.M, 8 * NT);
  cudaError_t e = allow_shared_memory((const void*)kern, kSmemBudget);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(32 * WARPS);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  const int64_t ring = (int64_t)WARPS * sqk::W4G_DEPTH * sqk::W4Slot<GW, ASYM>::BYTES;
  const int64_t cell = (int64_t)sqk::w4_cell_floats(NT) * 4, out = (int64_t)mr * 16 * 4;  // bytes per cell, per tile
  const int64_t x_unit = (int64_t)S * mr * (2 * sqk::W4_UNIT), x_fixed = (int64_t)S * mr * 64;
  // The cluster: as few CTAs as hold x and the sums of their tiles whole, or, with few tiles, as many
  // as still give every CTA an SM; each keeps at least two units of a tile.
  const int sms = (int)std::max<int64_t>(1, num_sms() / mt);
  int64_t used = 0;
  for (int C = 1;; C *= 2) {
    const int64_t units = (nu + C - 1) / C;
    const bool more = C < 8 && units >= 4;
    p.C = C;
    // (offsets within a CTA's tiles are 32-bit)
    const int64_t least = (tiles * 16 * p.w.row_bytes) / (int64_t)(UINT32_MAX - 16 * p.w.row_bytes) + 1;
    p.clusters = (int)std::min<int64_t>(tiles, std::max(sms / C, 1));
    if (C > 1) {
      attr[0].val.clusterDim.x = (unsigned)C;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      cfg.gridDim = dim3((unsigned)(p.clusters * C), 1);
      cfg.dynamicSmemBytes = (size_t)kSmemBudget;
      int active = 0;
      e = max_active_clusters((const void*)kern, &cfg, &active);
      if (e != cudaSuccess) return e;
      p.clusters = (int)std::min<int64_t>(p.clusters, std::max<int64_t>(1, active / mt));
    }
    p.clusters = (int)std::min(tiles, std::max<int64_t>(p.clusters, least));
    const int64_t per = (tiles + p.clusters - 1) / p.clusters;
    // tiles whose cells fit beside x, the whole of it: all of them, or passes of at least 16
    const int64_t x_all = x_fixed + units * x_unit;
    int64_t cap = (kSmemBudget - x_all - ring) / cell - (WARPS - 1);
    if (C > 1) cap = std::min(cap, ring / out);  // their sums take the rings' place
    const bool fits = cap >= std::min<int64_t>(per, 16);
    if (more && (!fits || tiles * C * 2 <= sms)) continue;
    if (fits) {
      const int64_t passes = (per + cap - 1) / cap;
      p.pass = (int)((per + passes - 1) / passes);
      p.chunk = (int)units;
      p.cell_at = (int)x_all;
      p.ring_at = p.out_at = (int)(x_all + (p.pass + WARPS - 1) * cell);
      used = p.ring_at + ring;
      break;
    }
    // x in chunks, tiles in passes: a pass of t tiles has at most t + WARPS - 1 cells
    const int64_t room = kSmemBudget - ring - x_fixed - (WARPS - 1) * cell;
    p.pass = (int)std::max<int64_t>(1, std::min(per, (room / 2) / (out + cell)));
    p.chunk = (int)std::min<int64_t>(units, (room - p.pass * (out + cell)) / x_unit);
    if (p.chunk < 1) return cudaErrorInvalidConfiguration;
    p.out_at = (int)(x_fixed + p.chunk * x_unit);
    p.cell_at = (int)(p.out_at + p.pass * out);
    p.ring_at = (int)(p.cell_at + (p.pass + WARPS - 1) * cell);
    used = p.ring_at + ring;
    break;
  }
  p.tile_q = (int)(tiles / p.clusters);
  p.tile_r = (int)(tiles % p.clusters);
  p.unit_q = nu / p.C;
  p.unit_r = nu % p.C;
  p.units = nu;
  p.odd = sqk::w4_blocks(p.K) % 2 != 0;
  cfg.dynamicSmemBytes = (size_t)used;
  cfg.gridDim = dim3((unsigned)(p.clusters * p.C), (unsigned)mt);
  cfg.attrs = p.C > 1 ? attr : attr + 1;
  cfg.numAttrs = p.C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int NT, int S, int GW, bool ASYM>
cudaError_t launch_w4_gemm_a(const sqk::W4GemmParams& p, cudaStream_t st) {
  const bool aligned = p.N % 8 == 0 && (uintptr_t)p.w.scales % 16 == 0 && (uintptr_t)p.w.zeros % 8 == 0;
  return aligned ? launch_w4_gemm_t<NT, S, GW, ASYM, true>(p, st)
                 : launch_w4_gemm_t<NT, S, GW, ASYM, false>(p, st);
}

template <int NT, int S>
cudaError_t launch_w4_gemm_g(const sqk::W4GemmParams& p, int group, cudaStream_t st) {
  if (p.w.zeros) {
    if (group == 32) return launch_w4_gemm_a<NT, S, 1, true>(p, st);
    if (group == 64) return launch_w4_gemm_a<NT, S, 2, true>(p, st);
    return launch_w4_gemm_a<NT, S, 4, true>(p, st);
  }
  if (group == 32) return launch_w4_gemm_a<NT, S, 1, false>(p, st);
  if (group == 64) return launch_w4_gemm_a<NT, S, 2, false>(p, st);
  return launch_w4_gemm_a<NT, S, 4, false>(p, st);
}

// Whether the kernel that unpacks a code once for a batch of tokens (sq_w4_tc.cu) is the faster one.  Its fixed
// costs want 4 M codes and 8 tiles of 128 channels; this file's takes a block of 16 tokens at a time.  Measured, us,
// this file's and that one:
//   bf16, groups of 128, 32 tokens: 1024 x 4096 8.4 and 6.9, 4096 x 4096 13.0 and 9.4, 28672 x 4096 41.5 and 27.2
//   (2048 x 768 4.8 and 6.3); 64 tokens: 4096 x 4096 16.5 and 13.3, 28672 x 4096 76 and 40
//   16 tokens: 2048 x 4096 10.0 and 7.5, 4096 x 4096 11.3 and 8.3, 28672 x 4096 24.9 and 25.3 (9 tokens 22.8 and 25.1)
//   (16384 x 4096 17.9 and 17.3, 24576 x 4096 23.1 and 23.0, 12288 x 12288 32.2 and 31.4; at 9 tokens 2048 x 4096 7.3
//   and 7.9, 4096 x 4096 9.8 and 8.7, 16384 x 4096 16.6 and 16.1, 24576 x 4096 21.1 and 22.3)
//   groups of 64, 9 / 16 / 32 tokens: 4096 x 4096 10.0 / 12.0 / 13.4 and 9.2 / 9.4 / 10.5, 6144 x 4096 11.7 / 12.7 / 16.2 and
//   12.2 / 12.8 / 14.1, 16384 x 4096 16.6 / 18.7 / 27.3 and 18.1 / 19.4 / 22.0, 28672 x 4096 24.0 / 26.1 / 47.5 and
//   29.3 / 29.4 / 33.0: up to 16 tokens the larger weights decide
//   binary32, 16 tokens: 2048 x 2048 9.5 and 7.1, 28672 x 4096 56 and 29; groups of 32 61 and 49 (2048 x 4096 11.2
//   and 12.6); 9 tokens: 2048 x 2048 8.6 and 7.2, 28672 x 4096 42 and 28, groups of 32 46 and 49
//   N = 512, 8192 channels, bf16, 16 / 32 / 64 tokens: 6.7 / 8.8 / 10.0 and 11.1 / 8.9 / 9.2
// Groups of 32 are four sums a block there, which the adding warps do not keep up with: bf16, 64 tokens, 4096 x 4096
// 17.5 and 21.5; 16 tokens, 28672 x 4096 29 and 40.
bool batch_kernel_pays(bool bf16, int64_t M, int64_t N, int64_t K, int group) {
  const int64_t codes = N * K;
  if (M <= 8 || N < 1024) return false;
  if (!bf16) return codes >= (group == 32 ? 1 << 24 : 1 << 22);
  if (group == 32) return false;
  if (M <= 16) return group == 128 && N >= 2048 && codes >= 1 << 23 && codes <= 1 << 26;
  return codes >= 1 << 22;
}

}  // namespace

cudaError_t launch_w4_gemm(const void* x, bool bf16, int64_t M, int64_t K, int64_t ldx, const uint8_t* wq,
                           const uint16_t* sg, const uint8_t* zp, int64_t N, int group, void* y, bool y_bf16,
                           int64_t ldy, cudaStream_t st) {
  if (batch_kernel_pays(bf16, M, N, K, group) && N % 8 == 0 && (uintptr_t)sg % 16 == 0 && (uintptr_t)zp % 8 == 0) {
    bool taken = false;
    const cudaError_t e = launch_w4_tc(x, bf16, M, K, ldx, wq, sg, zp, N, group, y, y_bf16, ldy, &taken, st);
    if (e != cudaSuccess || taken) return e;
  }
  sqk::W4GemmParams p{};
  p.x = (const char*)x;
  p.ldx_bytes = ldx * (bf16 ? 2 : 4);
  p.M = (int)M;
  p.K = (int)K;
  p.w.codes = (const char*)wq;
  p.w.scales = sg;
  p.w.zeros = zp;
  p.w.row_bytes = (uint32_t)(sqk::w4_blocks(K) * sqk::W4_BLOCK_BYTES);
  p.w.pitch = (uint32_t)N;
  p.w.groups = (int)((K + group - 1) / group);
  p.N = N;
  p.y = y;
  p.ldy = ldy;
  p.y_bf16 = y_bf16;
  // up to 8 tokens fill a column tile; more (where the other kernel does not pay, or does not fit) come in blocks of
  // 16 (grid y), each reading the weights again, from L2
  if (bf16) return M <= 8 ? launch_w4_gemm_g<1, 1>(p, group, st) : launch_w4_gemm_g<2, 1>(p, group, st);
  return M <= 8 ? launch_w4_gemm_g<1, 3>(p, group, st) : launch_w4_gemm_g<2, 3>(p, group, st);
}

}  // namespace sqh
