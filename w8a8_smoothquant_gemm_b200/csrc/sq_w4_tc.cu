// sq_w4_tc.cu -- x [M, K] times 4-bit weights [N, K] with group scales for a batch of tokens, on the
// 5th-generation tensor cores (tcgen05).
//
// y[m, n] = sum_g scale[g, n] * sum_{k in g} (code[n, k] - zero[g, n]) * x[m, k]
//
// Beyond two column tiles of mma.sync, what costs is no longer the weights' bytes but turning codes
// into operands again for every 16 tokens.  Here a code is unpacked once for all tokens of a block:
// the weights are the A operand (128 output channels), which tcgen05.mma takes from tensor memory, so
// the unpacked pairs go from registers straight there (tcgen05.st, a thread per channel) and never
// through shared memory; the tokens are the N columns of B, in shared memory for the whole of the CTA's
// share of K.  A group's sum of (code - zero) x is one accumulator; a thread per channel reads it, and
// adds it times the group's scale in binary32 registers.
//
//   adding      a warpgroup per 32 tokens: tcgen05.ld of a group's sums, scale, add; at a tile's end the
//               sums go to the ranks that store them (a slice of the tokens each)
//   out         a warpgroup: adds what came from the ranks, in their order, and stores
//   unpacking   two warpgroups, a unit (128 rows x 256 codes) each in turn: asynchronous copies into a
//               ring that belongs to the warp alone, unpack, tcgen05.st into two buffers a warpgroup
//   one warp    allocates tensor memory; one lane issues tcgen05.mma (kind::f16, M = 128, K = 16)
//
// A cluster of C CTAs cuts K, so that x fits; the CTAs' sums of a tile meet through distributed shared
// memory (every rank adds, in the order of the ranks, a slice of the tokens).  Waits are bounded.
//
// Measured: 64 x 4096 x 4096 13.3 us (blocks of 16 tokens on mma.sync: 16.4), 64 x 28672 x 4096 40.0 (77),
// 32 x 28672 x 4096 26.9 (42), 64 x 12288 x 12288 65.3 (105).  A block of 128 x 128
// codes takes some 640 clocks of an SM at 16 tokens, of which the integer pipe needs 250 for the unpacking and
// the matrix instructions 224: the rest is the chain of barriers between the roles.  A third unpacking
// warpgroup and reading the next sums ahead of the additions changed nothing.  At 64 x 28672 x 4096: the exchange by
// plain stores with cluster-wide fences, and a single lane in the issuing loop, 123 us; st.async and the whole
// warp in the loop 61; a warpgroup of its own for what comes in 47; its code unrolled per cluster size 41.
#include <algorithm>
#include <type_traits>

#include "sq_tc.cuh"
#include "sq_w4.cuh"

namespace sqk {

constexpr int TC_ROWS = 128;
// Warpgroups that add (32 tokens each, if there are as many), and threads of a CTA.
__host__ __device__ constexpr int tc_adders(int TB) { return TB > 32 ? TB / 32 : 1; }
__host__ __device__ constexpr int tc_threads(int TB) { return 128 * (tc_adders(TB) + 3) + 32; }
constexpr int TC_A_COLS = 64;                   // tensor memory columns of 128 unpacked codes
constexpr int TC_A_BUFS = 4;                    // two per unpacking warpgroup
constexpr int TC_SCALE_SLOTS = 4;               // units of scales on their way
constexpr int TC_BARS = 36;                     // room for the barriers (8 bytes each)

struct W4TcParams {
  const char* x;
  int64_t ldx_bytes;
  int M, K;
  W4Base w;
  int64_t N;
  void* y;
  int64_t ldy;
  int y_bf16;
  int C, clusters;     // CTAs of a cluster, clusters in x
  int units;           // of K
  int unit_q, unit_r;  // units / C and the remainder
  int tiles;
  bool odd;            // the last unit of K has one block
  int depth;           // slots of a warp's ring
  int recv_at, ring_at, scale_at, bar_at;  // shared memory: x first
  unsigned int* err;
};

__host__ __device__ constexpr int tc_groups(int GW) { return 8 / GW; }  // of a unit
// Bytes of a ring slot of one unpacking warp (32 rows), and of a scale slot of one adding warp.
__host__ __device__ constexpr int tc_slot(int GW, bool ASYM) { return 32 * 128 + (ASYM ? tc_groups(GW) * 32 : 0); }
__host__ __device__ constexpr int tc_scale_slot(int GW) { return tc_groups(GW) * 64; }

// D[tmem] (+)= A[tmem] B[smem]^T, bf16, binary32 sums; by the lane that is `on`.  The whole warp goes through
// the loop around it, so that descriptors stay in uniform registers.
__device__ __forceinline__ void tc_mma_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void tc_commit_if(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
  return on;
}
// Instruction descriptor of kind::f16: D = f32, A and B = bf16, both K-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A wait for what other CTAs of the cluster do: what they wrote before is then visible.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
  if (limit_ns == 0) return false;
  const unsigned long long t0 = global_ns();
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 1023u) == 0 && global_ns() - t0 > limit_ns) return false;
  }
}
// Four floats into another CTA's shared memory; they count on its barrier.
__device__ __forceinline__ void st_async4(uint32_t to, float2 a, float2 b, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to), "f"(a.x),
      "f"(a.y), "f"(b.x), "f"(b.y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void store_as(float* y, float v) { *y = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }

__device__ __forceinline__ void cp_wait_n(int n) {  // all but the n youngest groups
  if (n == 0) cp_wait<0>();
  else if (n == 1) cp_wait<1>();
  else if (n == 2) cp_wait<2>();
  else cp_wait<3>();
}

template <int TB, int S, int GW, bool ASYM>
__global__ void __launch_bounds__(tc_threads(TB), 1) w4_tc_kernel(const W4TcParams p) {
  constexpr int NC = S * TB;                 // columns: the parts of x are columns of their own
  constexpr int ND = NC <= 64 ? 4 : 2;       // accumulators
  constexpr int GPB = 4 / GW, GPU = 2 * GPB;  // groups of a block, of a unit
  constexpr int DW = tc_adders(TB), TW = TB / DW, OUT_WARP = 4 * DW + 8, MMA_WARP = OUT_WARP + 4, THREADS = tc_threads(TB);
  constexpr int SLOT = tc_slot(GW, ASYM), SCALES = tc_scale_slot(GW);
  // One group a block and as many accumulators as operand buffers: one commit says both that the sums are there
  // and that the operands have been used.
  constexpr bool ONE = GPB == 1 && ND == TC_A_BUFS;
  static_assert(NC % 16 == 0 && ND * NC + TC_A_BUFS * TC_A_COLS <= 512, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(0xffffffffu, tid / 32, 0);
  const uint32_t bar0 = sbase + p.bar_at;
  auto a_full = [&](int i) { return bar0 + 8u * i; };
  auto a_empty = [&](int i) { return bar0 + 8u * (4 + i); };
  auto d_full = [&](int i) { return bar0 + 8u * (8 + i); };
  auto d_empty = [&](int i) { return bar0 + 8u * (12 + i); };
  auto recv_full = [&](int par, int q) { return bar0 + 8u * (16 + 4 * par + q); };
  auto recv_free = [&](int par, int q) { return bar0 + 8u * (24 + 4 * par + q); };
  const uint32_t done = bar0 + 8u * 32;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + p.bar_at + 8 * 34);

  const int rank = blockIdx.x % p.C, cluster = blockIdx.x / p.C;
  const int m0 = blockIdx.y * TB, Mr = min(TB, p.M - m0);
  const int b0 = (int)w4_part(rank, p.unit_q, p.unit_r), units = p.unit_q + (rank < p.unit_r);
  const int t_first = (int)((int64_t)p.tiles * cluster / p.clusters);
  const int my_tiles = (int)((int64_t)p.tiles * (cluster + 1) / p.clusters) - t_first;
  const int total = my_tiles * units;
  const unsigned long long limit = wait_limit(p.err);

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(a_full(i), 4);
      mbar_init(a_empty(i), 1);
      mbar_init(d_full(i), 1);
      mbar_init(d_empty(i), 4 * DW);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(recv_full(0, i), 1);
      mbar_init(recv_free(0, i), (uint32_t)p.C);
    }
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  wait_for_previous_kernel();
  allow_dependent_launch();

  // x: per 64 values of K a tile of NC rows x 128 bytes, the 16-byte pieces of a row swizzled
  {
    const int vecs = units * (W4_UNIT / 8);
    const float inv_vecs = __frcp_rn((float)vecs);
    const char* src = p.x + m0 * p.ldx_bytes + (int64_t)b0 * W4_UNIT * (S == 1 ? 2 : 4);
    for (int i = tid; i < Mr * vecs; i += THREADS) {
      const int m = w4_div(i, vecs, inv_vecs), v = i - m * vecs;
      const bool there = b0 * W4_UNIT + v * 8 < p.K;
      auto at = [&](int s) {
        const int r = s * TB + m;
        return (uint32_t)((v / 8) * (NC * 128) + r * 128 + (((v % 8) ^ (r % 8)) << 4));
      };
      if (S == 1) {
        if (there) cp_async16(sbase + at(0), src + m * p.ldx_bytes + v * 16);
        else *reinterpret_cast<uint4*>(smem + at(0)) = make_uint4(0, 0, 0, 0);
      } else {
        float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (there) {
          const float4* q = reinterpret_cast<const float4*>(src + m * p.ldx_bytes + v * 32);
          *reinterpret_cast<float4*>(f) = q[0];
          *reinterpret_cast<float4*>(f + 4) = q[1];
        }
        uint32_t part[8][S];
#pragma unroll
        for (int e = 0; e < 8; ++e) split_bf16<S>(f[e], part[e]);
#pragma unroll
        for (int s = 0; s < S; ++s)
          *reinterpret_cast<uint4*>(smem + at(s)) =
              make_uint4(part[0][s] | (part[1][s] << 16), part[2][s] | (part[3][s] << 16),
                         part[4][s] | (part[5][s] << 16), part[6][s] | (part[7][s] << 16));
      }
    }
    cp_commit();
  }

  // An unpacking warp's ring.  Lane l copies piece l % 8 of rows l / 8, l / 8 + 4, ..; row r's pieces are
  // swizzled by r % 8, since a thread reads a row back.
  const int q = warp % 4, wg = (warp - 4 * DW) / 4;
  const uint32_t ring = sbase + p.ring_at + (warp - 4 * DW) * p.depth * SLOT;
  int load_i = wg, load_tile = wg / max(units, 1), load_u = wg - load_tile * max(units, 1);
  auto issue = [&](uint32_t slot) {
    if (load_i < total) {
      const int64_t n0 = (int64_t)(t_first + load_tile) * TC_ROWS + q * 32;
      const bool half = p.odd && b0 + load_u == p.units - 1;
      const int piece = lane % 8;
      if (n0 < p.N) {
        const char* src = p.w.codes + n0 * p.w.row_bytes + (int64_t)(b0 + load_u) * 128 + piece * 16;
        const uint32_t bytes = half && piece >= 4 ? 0u : 16u;
        if (!bytes) src -= 64;  // nothing is read there
        const uint32_t even = slot + (lane / 8) * 128 + ((piece ^ (lane / 8)) << 4);  // row r's pieces are swizzled by r % 8
        const uint32_t odd = slot + (lane / 8 + 4) * 128 + ((piece ^ (lane / 8 + 4)) << 4);
        if (n0 + 32 <= p.N) {
          src += (lane / 8) * p.w.row_bytes;
#pragma unroll
          for (int j = 0; j < 8; ++j, src += 4 * p.w.row_bytes)
            cp_async16((j % 2 ? odd : even) + j / 2 * 1024, src, bytes);
        } else {
          const uint32_t last = (uint32_t)(p.N - 1 - n0);
#pragma unroll 1
          for (int j = 0; j < 8; ++j)
            cp_async16((j % 2 ? odd : even) + j / 2 * 1024, src + (int64_t)(min(j * 4 + lane / 8, last) * p.w.row_bytes), bytes);
        }
        if (ASYM) {  // 8 rows' zero points of a group are 8 bytes
          const int g = min((b0 + load_u) * GPU + lane / 4, p.w.groups - 1);
          const int64_t n = min(n0 + lane % 4 * 8, p.N - 8);
          cp_async8_if(lane < GPU * 4, slot + 4096 + (lane / 4) * 32 + lane % 4 * 8, p.w.zeros + (int64_t)g * p.w.pitch + n);
        }
      }
      load_i += 2;
      for (load_u += 2; load_u >= units; load_u -= units) ++load_tile;
    }
    cp_commit();
  };
  // An adding warp's scales.
  const uint32_t scales = sbase + p.scale_at + warp * TC_SCALE_SLOTS * SCALES;
  int sc_i = 0, sc_tile = 0, sc_u = 0;
  auto issue_scales = [&](uint32_t slot) {
    if (sc_i < total) {
      const int g = min((b0 + sc_u) * GPU + lane / 4, p.w.groups - 1);
      const int64_t n = min((int64_t)(t_first + sc_tile) * TC_ROWS + q * 32 + lane % 4 * 8, p.N - 8);
      cp_async16_if(lane < GPU * 4, slot + (lane / 4) * 64 + lane % 4 * 16, p.w.scales + (int64_t)g * p.w.pitch + n);
      ++sc_i;
      if (++sc_u == units) {
        sc_u = 0;
        ++sc_tile;
      }
    }
    cp_commit();
  };
  if (warp < 4 * DW) {
#pragma unroll 1
    for (int i = 0; i < TC_SCALE_SLOTS - 1; ++i) issue_scales(scales + i * SCALES);
    cp_wait<TC_SCALE_SLOTS - 1>();
  } else if (warp < OUT_WARP) {
#pragma unroll 1
    for (int i = 0; i < p.depth - 1; ++i) issue(ring + i * SLOT);
    cp_wait_n(p.depth - 1);
  } else {
    cp_wait<0>();
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // x, for the tensor cores
  tc_fence_before();
  if (p.C > 1) cluster_sync();  // barriers of every rank are ready
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_holder);
  const uint32_t d_base = tmem + TC_A_BUFS * TC_A_COLS;

  // Sums over the cluster: rank c takes tokens w0 + c slice .. of every adding warpgroup of every rank,
  // [parity of the tile][warpgroup][source rank][4 tokens][row][4]
  const int log_slice = __ffs(TW) - __ffs(p.C), slice = 1 << log_slice;
  float* recv = reinterpret_cast<float*>(smem + p.recv_at);
  constexpr int PARITY = TB * TC_ROWS;

  bool landed = true;  // all that other ranks send to this thread's part of the exchange buffer
  if (warp == MMA_WARP) {
    // ------------------------------------------------------------------ matrix instructions
    constexpr uint32_t IDESC = idesc_bf16(TC_ROWS, NC);
    const uint32_t on = elect_one();
    bool ok = true;
    uint32_t d = 0, d_par = 1, u = 0;
    for (int i = 0; ok && i < total; ++i) {
      for (int b = 0; ok && b < 2; ++b) {
        const int buf = 2 * (i & 1) + b;
        // the operands and the first group's accumulator: looked at together, the answers take a while
        const uint32_t a_par = (i >> 1) & 1;
        const bool a_there = mbar_try_wait(a_full(buf), a_par), d_there = mbar_try_wait(d_empty(d), d_par);
        ok = limit != 0 && (a_there || mbar_wait(a_full(buf), a_par, limit)) && (d_there || mbar_wait(d_empty(d), d_par, limit));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = tmem + buf * TC_A_COLS;
        const uint64_t x = sw128_desc(sbase + (u * 4 + b * 2) * (NC * 128));
        for (int g = 0; g < GPB; ++g) {
          if (g > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(d_empty(d), d_par, limit));
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll
          for (int s = 0; s < 8 / GPB; ++s) {
            const int step = g * (8 / GPB) + s;
            tc_mma_ts(on, d_base + d * NC, a + step * 8, x + (((step / 4) * (NC * 128) + (step % 4) * 32) >> 4), IDESC, s > 0);
          }
          tc_commit_if(on, d_full(d));
          if (++d == ND) {
            d = 0;
            d_par ^= 1;
          }
        }
        if (!ONE) tc_commit_if(on, a_empty(buf));
      }
      if (++u == (uint32_t)units) u = 0;
    }
    if (!ok && on) atomicOr(p.err, ERR_GEMM_MMA_WAIT);
    tc_commit_if(on, done);  // nothing is in flight when tensor memory is given back
    mbar_wait(done, 0, DRAIN_NS);
    __syncwarp();
  } else if (warp >= OUT_WARP) {
    // ------------------------------------------------------------------ the cluster's sums, out
    bool ok = true;
    auto out = [&](auto ranks) {
      constexpr int C = decltype(ranks)::value, FOURS = TB / C / 4, SL = TW / C;
      for (int tile = 0; tile < my_tiles; ++tile) {
        const int par = tile & 1;
        if (lane == 0) mbar_arrive_expect_tx(recv_full(par, q), TB * 128);
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(recv_full(par, q), (tile >> 1) & 1, limit));
        if (!ok) break;
        float4 v[FOURS];  // this rank's tokens, by fours
#pragma unroll
        for (int k = 0; k < FOURS; ++k) {
          const float* from = recv + par * PARITY + (4 * k / SL) * (TW * TC_ROWS) + (4 * k % SL) * TC_ROWS + (q * 32 + lane) * 4;
          float4 o[C];
#pragma unroll
          for (int c = 0; c < C; ++c) o[c] = *reinterpret_cast<const float4*>(from + c * SL * TC_ROWS);
          v[k] = o[0];
#pragma unroll
          for (int c = 1; c < C; ++c)
            v[k] = make_float4(__fadd_rn(v[k].x, o[c].x), __fadd_rn(v[k].y, o[c].y), __fadd_rn(v[k].z, o[c].z), __fadd_rn(v[k].w, o[c].w));
        }
        // Every lane has read: the arrivals release that to the ranks, which write here again after they have acquired
        // it.  They come before this tile's stores, so all that they can wait for is the last tile's.
        __syncwarp();
        if (lane < C) mbar_arrive_cluster(map_shared(recv_free(par, q), lane));
        const int64_t n = (int64_t)(t_first + tile) * TC_ROWS + q * 32 + lane;
        if (n < p.N) {
          auto put = [&](auto* y) {
#pragma unroll
            for (int k = 0; k < FOURS; ++k) {
              const int m = (4 * k / SL) * TW + rank * SL + 4 * k % SL;
              auto* at = y + (m0 + m) * p.ldy + n;
              const float o[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (m + e < Mr) store_as(at + e * p.ldy, o[e]);
            }
          };
          if (p.y_bf16) put(reinterpret_cast<__nv_bfloat16*>(p.y));
          else put(reinterpret_cast<float*>(p.y));
        }
      }
    };
    if (p.C == 2) out(std::integral_constant<int, 2>{});
    else if (p.C == 4) out(std::integral_constant<int, 4>{});
    else if constexpr (TW >= 32) {
      if (p.C == 8) out(std::integral_constant<int, 8>{});
    }
    if (!ok && lane == 0) atomicOr(p.err, ERR_GEMM_EPILOGUE_WAIT);
    landed = ok || p.C == 1;
  } else if (warp >= 4 * DW) {
    // ------------------------------------------------------------------ codes to operands
    const uint32_t tm = tmem + ((uint32_t)(q * 32) << 16) + 2 * wg * TC_A_COLS;
    uint32_t slot = ring, spent = ring + (p.depth - 1) * SLOT;
    const uint32_t end = ring + p.depth * SLOT;
    uint32_t par = 1;
    bool ok = true;
    for (int i = wg; ok && i < total; i += 2) {
      cp_wait_n(p.depth - 2);
      __syncwarp();
      issue(spent);
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        uint32_t word[4][4];  // [piece t][w]
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint4 v = lds128(slot + lane * 128 + (((b * 4 + t) ^ (lane % 8)) << 4));
          word[t][0] = v.x;
          word[t][1] = v.y;
          word[t][2] = v.z;
          word[t][3] = v.w;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
#pragma unroll
          for (int w = 2 * h; w < 2 * h + 2; ++w) {
            const uint32_t zero = ASYM ? w4_zero(lds8(slot + 4096 + (b * GPB + w / GW) * 32 + lane)) : w4_zero(8);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              uint32_t pair[4];
              w4_unpack(pair, word[t][w], zero);
#pragma unroll
              for (int e = 0; e < 4; ++e) r[(w - 2 * h) * 16 + t * 4 + e] = pair[e];
            }
          }
          if (h == 0) {  // the buffer's last operands have been used
            ok = __all_sync(0xffffffffu, mbar_wait(ONE ? d_full(2 * wg + b) : a_empty(2 * wg + b), par, limit));
            if (!ok) break;
            tc_fence_after();
          }
          tmem_st32(tm + b * TC_A_COLS + h * 32, r);
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(a_full(2 * wg + b));
      }
      par ^= 1;
      spent = slot;
      slot = slot + SLOT == end ? ring : slot + SLOT;
    }
    if (!ok && lane == 0) atomicOr(p.err, ERR_GEMM_PRODUCER_WAIT);
    cp_wait<0>();
  } else {
    // ------------------------------------------------------------------ sums
    const int w0 = warp / 4 * TW;  // this warpgroup's first token
    const uint32_t tm = d_base + ((uint32_t)(q * 32) << 16) + w0;
    uint32_t slot = scales, spent = scales + (TC_SCALE_SLOTS - 1) * SCALES;
    uint32_t d = 0, d_par = 0;
    bool ok = true;
    float* to = recv + warp / 4 * (TW * TC_ROWS) + rank * slice * TC_ROWS + (q * 32 + lane) * 4;
    for (int tile = 0; ok && tile < my_tiles; ++tile) {
      float2 acc[TW / 2];
#pragma unroll
      for (int m = 0; m < TW / 2; ++m) acc[m] = make_float2(0.0f, 0.0f);
      for (int u = 0; ok && u < units; ++u) {
        cp_wait<TC_SCALE_SLOTS - 2>();
        __syncwarp();
        issue_scales(spent);
#pragma unroll 1
        for (int g = 0; g < GPU; ++g) {
          const float scale = bf16lo(lds16(slot + g * 64 + lane * 2));
          const float2 s2 = make_float2(scale, scale);
          ok = __all_sync(0xffffffffu, mbar_wait(d_full(d), d_par, limit));
          if (!ok) break;
          tc_fence_after();
          if constexpr (S == 1) {
            uint32_t r[TW];
            tmem_ld<TW>(tm + d * NC, r);
            tmem_wait_ld();
#pragma unroll
            for (int m = 0; m < TW / 2; ++m)
              acc[m] = __ffma2_rn(s2, make_float2(__uint_as_float(r[2 * m]), __uint_as_float(r[2 * m + 1])), acc[m]);
          } else {  // the parts' sums first
#pragma unroll
            for (int c = 0; c < TW; c += 16) {
              uint32_t r[3][16];
#pragma unroll
              for (int s = 0; s < 3; ++s) tmem_ld<16>(tm + d * NC + s * TB + c, r[s]);
              tmem_wait_ld();
#pragma unroll
              for (int m = 0; m < 8; ++m) {
                float2 v[3];
#pragma unroll
                for (int s = 0; s < 3; ++s) v[s] = make_float2(__uint_as_float(r[s][2 * m]), __uint_as_float(r[s][2 * m + 1]));
                acc[c / 2 + m] = __ffma2_rn(s2, __fadd2_rn(v[0], __fadd2_rn(v[1], v[2])), acc[c / 2 + m]);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(d_empty(d));
          if (++d == ND) {
            d = 0;
            d_par ^= 1;
          }
        }
        spent = slot;
        slot = slot + SCALES == scales + TC_SCALE_SLOTS * SCALES ? scales : slot + SCALES;
      }
      if (!ok) break;
      if (p.C == 1) {
        const int64_t n = (int64_t)(t_first + tile) * TC_ROWS + q * 32 + lane;
        if (n < p.N) {
#pragma unroll
          for (int m = 0; m < TW; ++m)
            if (w0 + m < Mr) store_out(p.y, (m0 + w0 + m) * p.ldy + n, m % 2 ? acc[m / 2].y : acc[m / 2].x, p.y_bf16);
        }
        continue;
      }
      const int par = tile & 1;
      ok = __all_sync(0xffffffffu, mbar_wait_cluster(recv_free(par, q), ((tile >> 1) & 1) ^ 1, limit));
      if (!ok) break;
      const uint32_t at = smem_u32(to + par * PARITY);
#pragma unroll
      for (int m = 0; m < TW / 4; ++m) {
        const uint32_t c = (uint32_t)(4 * m) >> log_slice, off = ((uint32_t)(4 * m) & (slice - 1)) * (TC_ROWS * 4);
        st_async4(map_shared(at + off, c), acc[2 * m], acc[2 * m + 1], map_shared(recv_full(par, q), c));
      }
    }
    if (!ok && lane == 0) atomicOr(p.err, ERR_GEMM_EPILOGUE_WAIT);
    cp_wait<0>();
  }

  tc_fence_before();
  if (p.C > 1) cluster_sync();  // no CTA leaves while others write to it
  else __syncthreads();
  if (warp == MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
  if (!landed) {
    // A wait ran out, and sums that the others sent may still be on their way.  All were sent before the barrier
    // above, which does not wait for them: this CTA's memory stays until they have come.
    const unsigned long long t0 = global_ns();
    for (uint32_t i = 0; i < (1u << 20) && global_ns() - t0 < 1000000ull; ++i) __nanosleep(1000);
  }
}

}  // namespace sqk

namespace sqh {
namespace {

constexpr int64_t kSmemBudget = 227 * 1024;

template <int TB, int S, int GW, bool ASYM>
cudaError_t launch_w4_tc_t(sqk::W4TcParams p, bool* taken, cudaStream_t st) {
  constexpr int NC = S * TB;
  auto kern = sqk::w4_tc_kernel<TB, S, GW, ASYM>;
  const int nu = sqk::w4_units(p.K);
  const int64_t mt = (p.M + TB - 1) / TB;
  p.tiles = (int)((p.N + sqk::TC_ROWS - 1) / sqk::TC_ROWS);
  p.units = nu;
  p.odd = sqk::w4_blocks(p.K) % 2 != 0;
  const int64_t fixed = 1024 + 4 * sqk::tc_adders(TB) * sqk::TC_SCALE_SLOTS * sqk::tc_scale_slot(GW) + 8 * sqk::TC_BARS;
  const int64_t slot = 8 * sqk::tc_slot(GW, ASYM);
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(sqk::tc_threads(TB));
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  *taken = false;
  // the cluster with the least work per CTA, in units, a tile's exchange counted as half a unit
  double best = 0;
  int best_c = 0, best_clusters = 0;
  for (int C = 1; C <= 8 && C <= nu && C * 4 * sqk::tc_adders(TB) <= TB; C *= 2) {
    const int64_t part = (nu + C - 1) / C;
    const int64_t room = kSmemBudget - fixed - part * NC * 512 - (C > 1 ? 2 * TB * 512 : 0);
    if (room < 2 * slot) continue;
    int64_t clusters = std::max<int64_t>(1, num_sms() / C);
    if (C > 1) {
      cudaError_t e = allow_shared_memory((const void*)kern, kSmemBudget);
      if (e != cudaSuccess) return e;
      attr[1].val.clusterDim.x = (unsigned)C;
      cfg.attrs = attr + 1;
      cfg.numAttrs = 1;
      cfg.gridDim = dim3((unsigned)(clusters * C));
      cfg.dynamicSmemBytes = (size_t)kSmemBudget;
      int active = 0;
      e = max_active_clusters((const void*)kern, &cfg, &active);
      if (e != cudaSuccess) return e;
      clusters = std::max(1, std::min((int)clusters, active));
    }
    clusters = std::max<int64_t>(1, std::min<int64_t>(p.tiles, clusters / mt));
    const double cost = (double)((p.tiles + clusters - 1) / clusters) * (part + (C > 1 ? 0.5 : 0.0));
    if (!best_c || cost < best) {
      best = cost;
      best_c = C;
      best_clusters = (int)clusters;
    }
  }
  if (!best_c) return cudaSuccess;
  *taken = true;
  p.C = best_c;
  p.clusters = best_clusters;
  p.unit_q = nu / p.C;
  p.unit_r = nu % p.C;
  const int64_t x = (int64_t)(p.unit_q + (p.unit_r > 0)) * NC * 512, recv = p.C > 1 ? 2 * TB * 512 : 0;
  p.depth = (int)std::min<int64_t>(4, (kSmemBudget - fixed - x - recv) / slot);
  p.recv_at = (int)x;
  p.ring_at = (int)(x + recv);
  p.scale_at = (int)(p.ring_at + p.depth * slot);
  p.bar_at = p.scale_at + 4 * sqk::tc_adders(TB) * sqk::TC_SCALE_SLOTS * sqk::tc_scale_slot(GW);
  cudaError_t e = allow_shared_memory((const void*)kern, kSmemBudget);
  if (e != cudaSuccess) return e;
  attr[1].val.clusterDim.x = (unsigned)p.C;
  cfg.gridDim = dim3((unsigned)(p.clusters * p.C), (unsigned)mt);
  // All of an SM's shared memory, whatever is used of it: no other kernel that allocates tensor memory may share
  // the SM, since two clusters that each held an SM the other waits for would never go on.
  cfg.dynamicSmemBytes = (size_t)kSmemBudget;
  cfg.attrs = attr;
  cfg.numAttrs = p.C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int TB, int S>
cudaError_t launch_w4_tc_g(const sqk::W4TcParams& p, int group, bool* taken, cudaStream_t st) {
  if constexpr (S > 1) {  // (groups of 32 come here with binary32 x alone)
    if (group == 32)
      return p.w.zeros ? launch_w4_tc_t<TB, S, 1, true>(p, taken, st) : launch_w4_tc_t<TB, S, 1, false>(p, taken, st);
  }
  if (p.w.zeros) {
    if (group == 64) return launch_w4_tc_t<TB, S, 2, true>(p, taken, st);
    return launch_w4_tc_t<TB, S, 4, true>(p, taken, st);
  }
  if (group == 64) return launch_w4_tc_t<TB, S, 2, false>(p, taken, st);
  return launch_w4_tc_t<TB, S, 4, false>(p, taken, st);
}

}  // namespace

// *taken: whether some block of tokens fits; if not, nothing is launched.
cudaError_t launch_w4_tc(const void* x, bool bf16, int64_t M, int64_t K, int64_t ldx, const uint8_t* wq,
                         const uint16_t* sg, const uint8_t* zp, int64_t N, int group, void* y, bool y_bf16, int64_t ldy,
                         bool* taken, cudaStream_t st) {
  sqk::W4TcParams p{};
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
  p.err = error_word_ptr();
  *taken = false;
  if (!p.err) return cudaErrorInvalidDevice;
  cudaError_t e = cudaSuccess;
  if (bf16) {
    if (M > 32) e = launch_w4_tc_g<64, 1>(p, group, taken, st);
    if (e == cudaSuccess && !*taken && M > 16) e = launch_w4_tc_g<32, 1>(p, group, taken, st);
    if (e == cudaSuccess && !*taken) e = launch_w4_tc_g<16, 1>(p, group, taken, st);
  } else {
    if (M > 16) e = launch_w4_tc_g<32, 3>(p, group, taken, st);
    if (e == cudaSuccess && !*taken) e = launch_w4_tc_g<16, 3>(p, group, taken, st);
  }
  return e;
}

}  // namespace sqh
