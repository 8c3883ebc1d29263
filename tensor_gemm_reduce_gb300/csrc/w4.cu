// w4.cu -- the row-parallel layer for 1 to 32 tokens with 4-bit weights
// (gemm_rs_w4_* in include/gemm_rs_ops.h):
//   out[m][n] = sum_r sum_k x[r][m][k] (code[r][k][n] - zero[r][g][n]) scale[r][g][n]
//
// The weights are read once and there are few tokens, so the product is bound
// by HBM: 0.5 bytes a weight and 2 (2.5 with zero points) for each group.
// The layout makes every lane's weights of four MMA steps one 16-byte load and
// a warp's 512 consecutive bytes.  The MMA is mma.sync m16n8k16 with the
// weights as the 16-row operand: the codes are unpacked in registers straight
// into its fragments (tcgen05 would need them written to shared memory as bf16,
// four times the bytes read from HBM), and its rate is not the limit.
//
// Unpacking: a bf16 pattern below 256 stands for 2^-133 times its value (bf16's
// subnormals and its first binade lie on one line), so a code masked out of a
// word is a number already, wherever it lies in the low byte of a half word.
// One bf16x2 FMA, exact, scales it and subtracts the zero point: the tensor core
// multiplies the exact values (code - zero) 2^-6 with the bf16 inputs.  Each
// group's sum is scaled in fp32 and added to the total, which takes 2^6 at the end.  The masks
// and shifts keep the integer pipe the busiest: 5 instructions for 8 weights.
//
// Split: a cluster of 8 CTAs computes up to 128 columns, CTA r rank r's share of
// the sum; each CTA hands the others their columns of its share through
// distributed shared memory and adds the eight (in rank order) that it is handed:
// the layer's reduce-scatter, inside one cluster.  Inside a CTA the warps take
// columns, and where there are few columns also parts of the inner dimension.
//
// Measured, us, calls in a row over weights of 12 layers in turn, which L2 does not
// hold: one token, 8192 columns, K = 28672 with zero points (122 MB) 24.8, 4.9 TB/s,
// 0.72 of a copy's rate; K = 8192 10.0, where the clusters' start and joins count as
// much as the weights.  16 tokens, 6144 columns, K = 16384, groups of 64 19.3; 32
// tokens 37.6, in groups of 128 32.7: 12 to 16 warps an SM hide too little of the
// latency of unpacking, MMA and scaling.  (Three layers in turn, of which L2 holds much:
// 24.3, 8.6, 18.4, 37.2 and 32.3.)
#include "ops_common.cuh"

using namespace grs;

namespace {

constexpr int kRanks = 8;
constexpr int kBlockN = 32;         // columns that lie together in the packed weights, in two halves
constexpr int kCell = 64;           // inner elements of a lane's 16-byte load
constexpr int kUnit = 128;          // inner elements of a step: two cells of each half
constexpr int kMaxTokens = 32;
constexpr int kPrefetchUnits = 8;   // units of a warp asked for before the previous grid ends
constexpr int kMaxSmem = 227 * 1024;
constexpr int kSmWarps = 16;        // that an SM holds at 128 registers a thread

// Halves of a block that a warp multiplies (one set of input fragments serves
// both, but 3 and 4 token tiles leave no registers for a second one), and units
// of weights in flight for each warp: what leaves the fewest spills, which go to L2
// where shared memory takes most of L1 (32 tokens, 6144 columns, K = 16384: 37 us
// with 4 units, 33 with 3).
__host__ __device__ constexpr int halves_of(int tiles) { return tiles <= 2 ? 2 : 1; }
__host__ __device__ constexpr int depth_of(int tiles) { return tiles == 2 ? 2 : 3; }

// Tokens of a column of the shares: eight (32 bytes, what one store of a warp
// writes of a column) or a multiple, or 2 or 4.
__host__ __device__ constexpr int share_pitch(int M) { return M <= 2 ? 2 : M <= 4 ? 4 : (M + 7) / 8 * 8; }

// Packed buffer: weights [N/32][8][units][2 halves][2 cells][32 lanes] of 16
// bytes, then scales [N/32][8][groups][2 halves][8] of two bf16 (columns g and
// g + 8), then zero points of the same shape, two bytes each; N/32 and units =
// K/8/128 rounded up, groups those of whole units.  What lies beyond the layer's
// sizes is zero.
// A cell's 64 inner elements: step j of part h holds, in lane 4 g + q, inner
// elements 32 h + 8 q + 4 j + {0, 1, 2, 3} of columns g and g + 8, four bits
// each, at bits 0, 16 (column g, elements 0, 1), 4, 20 (g + 8), 8, 24 (column
// g, elements 2, 3) and 12, 28 of word 2 h + j.
struct Layout {
  long long blocks, units, groups;
  long long scale_off, zero_off, bytes;
};
Layout layout_of(int64_t N, int64_t K, int group, bool zeros) {
  Layout l;
  const int64_t Kr = K / kRanks;
  l.blocks = (N + kBlockN - 1) / kBlockN;
  l.units = (Kr + kUnit - 1) / kUnit;
  l.groups = l.units * (kUnit / group);
  l.scale_off = l.blocks * kRanks * l.units * 2048;
  l.zero_off = l.scale_off + l.blocks * kRanks * l.groups * 64;
  l.bytes = l.zero_off + (zeros ? l.blocks * kRanks * l.groups * 32 : 0);
  return l;
}

struct W4Params {
  int M, N, Kr, group;
  int blocks, units, groups;   // units and groups of a rank
  int wn, wk;                  // warps of a CTA: wn of columns x wk parts of the units
  int part_units;              // units of a part
  int prefetch_units;          // of each warp, before the previous grid ends
  int chunks, chunk_units, pitch;  // a part's inputs arrive in chunks: units, row pitch in bytes
  const uint16_t* x;           // [8][M][Kr]
  const uint4* weights;
  const uint32_t* scales;
  const uint16_t* zeros;
  uint16_t* out;               // [M][N]
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b: the same without an addend.
__device__ __forceinline__ void mma_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Multiples of 16 bytes.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, float a, float b) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

// kTiles tiles of 8 tokens, groups of kGroup inner elements.
template <int kTiles, int kGroup, bool kZeros>
__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(256, 2)
    w4_kernel(const W4Params p) {
  // for each part two chunks of the inputs [token][chunk]; then the ranks' and
  // parts' shares of this CTA's columns [rank][part][column][token], which the
  // cluster's CTAs write
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kHalves = halves_of(kTiles), kDepth = depth_of(kTiles);
  constexpr int kPerUnit = kUnit / kGroup;  // groups in a unit
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp / p.wn, wn = warp - part * p.wn;
  const int rank = blockIdx.x, tile = blockIdx.y;
  const int g = lane >> 2, q = lane & 3;
  const int cols = 16 * kHalves * p.wn, share = cols / kRanks;  // of the cluster, of a CTA
  const int u0 = part * p.part_units < p.units ? part * p.part_units : p.units;
  const int u1 = u0 + p.part_units < p.units ? u0 + p.part_units : p.units;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t inputs = (uint32_t)(part * 2 * p.M * p.pitch);  // this part's chunks
  // The next launch's blocks may take the places that this one's leave; they
  // read and write no memory before this grid is complete, but bring their first
  // weights to L2 (a hint, which sees whatever is written until they are read).
  griddep_launch_dependents();
  // every CTA of the cluster is running before any writes into another's memory
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  // inputs of units [u, u + chunk_units) into buffer `buf`; zero beyond the row's
  // end.  A row takes a warp, or with more than 8 tokens half of one where a chunk
  // is one unit (16 tokens, 512 columns, K = 28672: 16.5 -> 10.4 us).
  auto stage_inputs = [&](int u, int buf) {
    const int row_log = kTiles > 1 && p.chunk_units == 1 ? 4 : 5, row_lanes = 1 << row_log;
    const int first = kTiles > 1 ? (int)(threadIdx.x - 32 * part * p.wn) >> row_log : wn;
    const int vectors = (u1 - u < p.chunk_units ? u1 - u : p.chunk_units) * (kUnit / 8);
    for (int m = first; m < p.M; m += (32 * p.wn) >> row_log) {
      const uint16_t* src = p.x + ((long long)rank * p.M + m) * p.Kr;
      for (int v = lane & (row_lanes - 1); v < vectors; v += row_lanes) {
        const int k = u * kUnit + 8 * v;
        const bool in = k < p.Kr;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(
                         sbase + inputs + (uint32_t)((buf * p.M + m) * p.pitch + 16 * v)),
                     "l"(in ? src + k : p.x), "r"(in ? 16 : 0)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  float acc[kHalves][kTiles][4];
#pragma unroll
  for (int b = 0; b < kHalves; ++b)
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[b][t][i] = 0.f;

  // A unit's weights, scales and zero points.  Lane 4 g + q holds those of the
  // unit's group q (columns g and g + 8); the others ask it by a shuffle.
  struct Unit {
    uint4 w[kHalves][2];
    uint32_t s[kHalves], z[kHalves];
  };
  // columns beyond the last block read the last one's weights and are not stored
  const int half_at = tile * (p.wn * kHalves) + wn * kHalves;  // this warp's first half of a block
  const int block_at = half_at / 2, half0 = half_at % 2;
  const int block = block_at < p.blocks ? block_at : p.blocks - 1;
  const long long at = (long long)block * kRanks + rank;
  const long long group0 = at * p.groups + (long long)u0 * kPerUnit + q % kPerUnit;
  const uint4* wp = p.weights + (at * p.units + u0) * 128 + half0 * 64 + lane;
  const uint32_t* sp = p.scales + group0 * 16 + 8 * half0 + g;
  const uint16_t* zp = kZeros ? p.zeros + group0 * 16 + 8 * half0 + g : nullptr;
  // unit `d` beyond the pointers
  auto fetch = [&](Unit& v, int d, bool in) {
    if (!in) return;
#pragma unroll
    for (int b = 0; b < kHalves; ++b) {
      v.w[b][0] = load_v4_stream(wp + d * 128 + b * 64);
      v.w[b][1] = load_v4_stream(wp + d * 128 + b * 64 + 32);
      v.s[b] = load_u32_stream(sp + d * kPerUnit * 16 + 8 * b);
      if (kZeros) v.z[b] = load_u16_stream(zp + d * kPerUnit * 16 + 8 * b);
    }
  };
  const int early = u1 - u0 < p.prefetch_units ? u1 - u0 : p.prefetch_units;
  if (lane == 0 && half0 == 0 && early > 0) {
    prefetch_l2(wp, (uint32_t)early * 2048);
    prefetch_l2(p.scales + (at * p.groups + (long long)u0 * kPerUnit) * 16, (uint32_t)(early * kPerUnit * 64));
  }
  griddep_wait();
  Unit ring[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d) fetch(ring[d], d, u0 + d < u1);
  if (u0 < u1) stage_inputs(u0, 0);

  // tokens beyond the last read its row; their columns are not stored
  uint32_t row[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) row[t] = (uint32_t)((8 * t + g < p.M ? 8 * t + g : p.M - 1) * p.pitch + 16 * q);

  int buf = 0;
  uint32_t xu = 0;  // the unit's inputs
  int chunk_end = u0, synced = 0;
#pragma unroll 1
  for (int base = u0; base < u1; base += kDepth) {
    wp += kDepth * 128;
    sp += kDepth * kPerUnit * 16;
    if (kZeros) zp += kDepth * kPerUnit * 16;
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int u = base + d;
      if (u >= u1) break;
      if (u == chunk_end) {  // the chunk has arrived; the next one takes the other buffer
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        ++synced;
        xu = inputs + (uint32_t)(buf * p.M * p.pitch);
        buf ^= 1;
        chunk_end += p.chunk_units;
        if (chunk_end < u1) stage_inputs(chunk_end, buf);
      } else {
        xu += 2 * kUnit;
      }
      const Unit& cur = ring[d];
#pragma unroll
      for (int grp = 0; grp < kPerUnit; ++grp) {
        float sum[kHalves][kTiles][4];
        uint32_t nz[kHalves][2];  // -(zero point) 2^-6 of columns g and g + 8, in both halves
#pragma unroll
        for (int b = 0; b < kHalves; ++b) {
          nz[b][0] = nz[b][1] = 0xBE00BE00u;  // -8 2^-6
          if (kZeros) {
            const uint32_t z = kPerUnit == 1 ? cur.z[b] : __shfl_sync(0xffffffffu, cur.z[b], (lane & 28) + grp);
            // z as a number (its pattern is 2^-133 z) times -2^127
            nz[b][0] = fma_bf16x2((z & 0xFFu) * 0x10001u, 0xFF00FF00u, 0u);
            nz[b][1] = fma_bf16x2((z >> 8) * 0x10001u, 0xFF00FF00u, 0u);
          }
        }
#pragma unroll
        for (int hh = 0; hh < kGroup / 32; ++hh) {  // 32 inner elements
          const int h = grp * (kGroup / 32) + hh;
          uint4 xv[kTiles];
#pragma unroll
          for (int t = 0; t < kTiles; ++t) xv[t] = *reinterpret_cast<const uint4*>(smem + xu + row[t] + 64 * h);
#pragma unroll
          for (int b = 0; b < kHalves; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint4& v = cur.w[b][h >> 1];
              const uint32_t word = (h & 1) ? (j ? v.w : v.z) : (j ? v.y : v.x), high = word >> 8;
              const uint32_t a[4] = {fma_bf16x2(word & 0x000F000Fu, 0x7F007F00u, nz[b][0]),   // 2^127
                                     fma_bf16x2(word & 0x00F000F0u, 0x7D007D00u, nz[b][1]),   // 2^123
                                     fma_bf16x2(high & 0x000F000Fu, 0x7F007F00u, nz[b][0]),
                                     fma_bf16x2(high & 0x00F000F0u, 0x7D007D00u, nz[b][1])};
#pragma unroll
              for (int t = 0; t < kTiles; ++t) {
                if (hh == 0 && j == 0)
                  mma_16816_first(sum[b][t], a, xv[t].x, xv[t].y);
                else
                  mma_16816(sum[b][t], a, j ? xv[t].z : xv[t].x, j ? xv[t].w : xv[t].y);
              }
            }
        }
#pragma unroll
        for (int b = 0; b < kHalves; ++b) {
          const uint32_t s = kPerUnit == 1 ? cur.s[b] : __shfl_sync(0xffffffffu, cur.s[b], (lane & 28) + grp);
          const float s0 = bf16lo_to_f32(s), s1 = bf16hi_to_f32(s);
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            acc[b][t][0] = fmaf(s0, sum[b][t][0], acc[b][t][0]);
            acc[b][t][1] = fmaf(s0, sum[b][t][1], acc[b][t][1]);
            acc[b][t][2] = fmaf(s1, sum[b][t][2], acc[b][t][2]);
            acc[b][t][3] = fmaf(s1, sum[b][t][3], acc[b][t][3]);
          }
        }
      }
      fetch(ring[d], d, u + kDepth < u1);  // into the registers just used
    }
  }
  // A shorter last part keeps the others company at their chunks' barriers.  (One
  // barrier for each part would do, but a kernel that names barriers at run time
  // holds all 16 of a CTA, and an SM has 64: no more than 4 CTAs.)
  for (; synced < p.chunks; ++synced) __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  // Hand each CTA this warp's sums for its columns, two tokens a lane and whole 32
  // bytes a column: with only the tokens there are (5 tokens, 12288 columns, K =
  // 4096) 11.6 instead of 11.0 us; 4-byte stores for each token, 13.7 instead of
  // 10.2 at 16 tokens, 512 columns, K = 28672.
  const uint32_t shares = (uint32_t)(p.wk * 2 * p.M * p.pitch);
  const int tokens = share_pitch(p.M);
#pragma unroll
  for (int b = 0; b < kHalves; ++b)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = (wn * kHalves + b) * 16 + g + 8 * i, owner = col / share;
      const uint32_t to = mapa_shared(sbase + shares, owner) +
                          4u * (uint32_t)(((rank * p.wk + part) * share + col - owner * share) * tokens + 2 * q);
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        if (8 * t + 2 * q < tokens) st_cluster_v2(to + 32u * t, 64.f * acc[b][t][2 * i], 64.f * acc[b][t][2 * i + 1]);
    }
  cluster_sync();  // the shares of all ranks are here

  const float* from = reinterpret_cast<const float*>(smem + shares);
  // eight tokens of a column in eight lanes, then the next column
  const int low = tokens < 8 ? tokens : 8;
  for (int i = threadIdx.x; i < share * tokens; i += blockDim.x) {
    const int c = i / low, block = c / share, col = c - block * share, m = block * low + i - c * low;
    const int n = tile * cols + rank * share + col;
    if (m >= p.M || n >= p.N) continue;
    float s = 0.f;
    for (int r = 0; r < kRanks * p.wk; ++r) s += from[(r * share + col) * tokens + m];  // in order
    p.out[(long long)m * p.N + n] = (uint16_t)(pack_bf16x2(s, 0.f) & 0xFFFFu);
  }
}

struct PackParams {
  int N, Kr, group, blocks, units, groups, in_groups;
  const uint8_t* codes;    // [8][Kr][N]
  const uint16_t* scales;  // [8][groups][N]
  const uint8_t* zeros;    // [8][groups][N] or null
  uint32_t* weights;
  uint32_t* out_scales;
  uint16_t* out_zeros;
};

// A block takes 64 inner elements x 128 columns at a time through shared memory:
// rows come in whole 128-byte lines, each warp packs one cell of 16 columns.
// Then the groups' scales and zero points.
__global__ void __launch_bounds__(256) w4_pack_kernel(const PackParams p) {
  constexpr int kCols = 128, kPitch = kCols + 4;  // 4 bytes beyond, so that rows 8 apart lie in other banks
  __shared__ uint8_t tile[kCell * kPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cells = 2 * p.units;
  const long long items = (long long)((p.N + kCols - 1) / kCols) * kRanks * cells;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int c = (int)(item % cells), r = (int)(item / cells % kRanks);
    const int n0 = (int)(item / cells / kRanks) * kCols;
    __syncthreads();  // the previous item's tile has been read
    for (int i = threadIdx.x; i < kCell * kCols / 8; i += blockDim.x) {
      const int row = i / (kCols / 8), seg = i % (kCols / 8);
      const int k = c * kCell + row, n = n0 + 8 * seg;  // N is a multiple of 8
      uint2 v = make_uint2(0, 0);
      if (k < p.Kr && n < p.N) v = __ldcs(reinterpret_cast<const uint2*>(p.codes + ((long long)r * p.Kr + k) * p.N + n));
      uint32_t* to = reinterpret_cast<uint32_t*>(tile + row * kPitch + 8 * seg);
      to[0] = v.x & 0x0F0F0F0Fu;
      to[1] = v.y & 0x0F0F0F0Fu;
    }
    __syncthreads();
    const int block = n0 / kBlockN + warp / 2, half = warp & 1;
    if (block >= p.blocks) continue;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int step = 0; step < 4; ++step)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int reg = e >> 1;  // MMA register: column g or g + 8, inner pair 0 or 1
        const int k = 32 * (step >> 1) + 8 * (lane & 3) + 4 * (step & 1) + 2 * (reg >> 1) + (e & 1);
        const int n = warp * 16 + (lane >> 2) + 8 * (reg & 1);
        w[step] |= (uint32_t)tile[k * kPitch + n] << (4 * reg + 16 * (e & 1));
      }
    const long long at = ((((long long)block * kRanks + r) * p.units + c / 2) * 2 + half) * 2 + (c & 1);
    reinterpret_cast<uint4*>(p.weights)[at * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  const long long stride = (long long)gridDim.x * blockDim.x;
  const long long first = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long metas = (long long)p.blocks * kRanks * p.groups * 16;
  for (long long i = first; i < metas; i += stride) {
    const int g = (int)(i & 7), half = (int)(i >> 3) & 1;
    const long long t = i >> 4;
    const int grp = (int)(t % p.groups);
    const int r = (int)(t / p.groups % kRanks);
    const int n = (int)(t / p.groups / kRanks) * kBlockN + half * 16 + g;
    const long long row = ((long long)r * p.in_groups + grp) * p.N;
    const bool lo_in = grp < p.in_groups && n < p.N, hi_in = grp < p.in_groups && n + 8 < p.N;
    const uint32_t lo = lo_in ? p.scales[row + n] : 0u, hi = hi_in ? p.scales[row + n + 8] : 0u;
    p.out_scales[i] = lo | hi << 16;
    if (p.zeros) {
      const uint32_t zl = lo_in ? p.zeros[row + n] & 127u : 0u, zh = hi_in ? p.zeros[row + n + 8] & 127u : 0u;
      p.out_zeros[i] = (uint16_t)(zl | zh << 8);
    }
  }
}

// Symmetric round-to-nearest codes of one group and column a thread.
__global__ void __launch_bounds__(256) w4_quantize_kernel(const uint16_t* W, uint8_t* codes, uint16_t* scales,
                                                          int N, int Kr, int group, int groups) {
  const long long total = (long long)kRanks * groups * N;
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int n = (int)(i % N);
    const int grp = (int)(i / N % groups), r = (int)(i / N / groups);
    const int k0 = grp * group, k1 = k0 + group < Kr ? k0 + group : Kr;
    const long long at = (long long)r * Kr * N + n;
    float top = 0.f;
    bool finite = true;
    for (int k = k0; k < k1; ++k) {
      const float a = fabsf(__uint_as_float((uint32_t)W[at + (long long)k * N] << 16));
      finite = finite && a < __uint_as_float(0x7F800000u);
      top = fmaxf(top, a);
    }
    const uint32_t s = finite ? pack_bf16x2(__fdiv_rn(top, 7.f), 0.f) & 0xFFFFu : 0x7FC0u;
    const float sf = __uint_as_float(s << 16);
    scales[i] = (uint16_t)s;
    for (int k = k0; k < k1; ++k) {
      const float v = __uint_as_float((uint32_t)W[at + (long long)k * N] << 16);
      float c = sf > 0.f ? rintf(__fdiv_rn(v, sf)) : 0.f;
      c = fminf(fmaxf(c, -8.f), 7.f);
      codes[at + (long long)k * N] = (uint8_t)((int)c + 8);
    }
  }
}

int check(int64_t M, int64_t N, int64_t K, int group) {
  if (group != 32 && group != 64 && group != 128) return GEMM_RS_ERR_INVALID_ARG;
  if (M < 0 || M > kMaxTokens || N < 0 || K < 0 || N % 8 || K % 64 || N > (1ll << 19) || K > (1ll << 30))
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  return GEMM_RS_OK;
}

// How the columns and the inner dimension are cut: clusters of 128 columns, and
// fewer columns where that leaves under 32 clusters (256 CTAs), down to a warp's,
// or two warps' from 17 tokens on (every CTA copies all its rank's inputs: 32
// tokens, 512 columns, K = 28672: 16 columns x 8 parts 30.8 us, 32 x 4 15.7).  Then
// parts of the inner dimension: CTAs of 8 warps where two of them fit each SM at
// once, else of 4, which fit four times (2560 columns, K = 8192, one token: 64
// columns x 3 parts in two waves 7.3, 64 x 2 at once 4.9).  A warp's columns and up
// to 4 tokens take 4 parts (1024 columns, K = 8192, one token 3.4 against 3.8 with
// 8; 512 columns, K = 28672, 3 tokens 5.7 against 5.9, 6 tokens 7.8 against 6.8).
// (Narrower clusters for an even load of the SMs gained nothing at 8192 columns:
// 112 columns on 148 SMs as long as 128 on 128.)
struct Split {
  int wn, wk, clusters, part_units, chunk_units, pitch, smem;
  bool at_once;  // every cluster runs from the start
};
// Clusters of 8 CTAs that run at once with n CTAs an SM.
constexpr int kMaxPerSm = 4;
struct Slots {
  int at[kMaxPerSm + 1];
};
// Dynamic shared memory with which n CTAs fit an SM and n + 1 do not.
int smem_for(int n) { return 228 * 1024 / (n + 1) - 1024 + 128; }
Split split_of(int64_t M, int64_t N, int units, int tiles, const Slots& slots) {
  Split s = {};
  const int half_cols = 16 * halves_of(tiles);
  s.wn = 128 / half_cols;
  while (s.wn > (tiles > 2 ? 2 : 1) && N <= 31ll * half_cols * s.wn) s.wn /= 2;
  s.clusters = (int)((N + half_cols * s.wn - 1) / (half_cols * s.wn));
  const bool eight = s.clusters <= slots.at[kSmWarps / 8] && !(M <= 4 && s.wn == 1);
  s.wk = (eight ? 8 : 4) / s.wn;
  if (s.wk > units) s.wk = units;
  if (s.wk < 1) s.wk = 1;
  s.part_units = (units + s.wk - 1) / s.wk;
  s.wk = (units + s.part_units - 1) / s.part_units;
  // the inputs' chunks: up to 32 units, an even number (a warp copies two at a time),
  // within the shared memory of as many CTAs as an SM's registers hold
  const int room = kMaxSmem / (kSmWarps / (s.wn * s.wk)) - 2 * 1024;
  for (int most = s.part_units < 32 ? s.part_units : 32;; most = most > 2 ? (most - 1) / 2 * 2 : 1) {
    s.chunk_units = most;
    s.pitch = s.chunk_units * kUnit * 2 + 64;  // two rows that 8 lanes read lie in different banks
    s.smem = (int)(s.wk * (2 * M * s.pitch + share_pitch((int)M) * half_cols * s.wn * 4));  // and the shares
    if (most == 1 || s.smem <= room) break;
  }
  // The hardware packs clusters as densely as they fit and leaves the last SMs
  // without work: no more CTAs an SM than the clusters need to run at once (6144
  // columns, K = 16384: 3 on 128 SMs instead of 4 on 96, one token 15.8 -> 13.8 us,
  // 16 tokens 24.3 -> 20.5).
  for (int n = 1; n <= kMaxPerSm; ++n)
    if (slots.at[n] >= s.clusters) {
      if (n < kMaxPerSm && s.smem < smem_for(n)) s.smem = smem_for(n);
      s.at_once = true;
      break;
    }
  return s;
}

// Looked up once for each device, with a kernel of one warp (registers and warps
// do not bound it).
bool slots_of(Slots* out) {
  static std::atomic<int> known[64][kMaxPerSm + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  const auto kernel = w4_kernel<1, 128, false>;
  for (int n = 1; n <= kMaxPerSm; ++n) {
    int clusters = known[dev][n].load(std::memory_order_relaxed);
    if (clusters == 0) {
      static SmemAllowed allowed;
      if (!allowed.set(kernel, kMaxSmem)) return false;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(kRanks, 1024);
      cfg.blockDim = dim3(32);
      cfg.dynamicSmemBytes = (size_t)smem_for(n);
      if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters < 1) {
        cudaGetLastError();
        return false;
      }
      known[dev][n].store(clusters, std::memory_order_relaxed);
    }
    out->at[n] = clusters;
  }
  return true;
}

template <int kTiles, int kGroup>
int launch(const W4Params& p, const Split& sp, cudaStream_t st) {
  const auto kernel = p.zeros ? w4_kernel<kTiles, kGroup, true> : w4_kernel<kTiles, kGroup, false>;
  static SmemAllowed allowed[2];
  if (!allowed[p.zeros != nullptr].set(kernel, kMaxSmem)) return GEMM_RS_ERR_CUDA;
  return launch_overlapped(kernel, dim3(kRanks, (unsigned)sp.clusters), 32 * sp.wn * sp.wk, (size_t)sp.smem, st, p);
}

template <int kTiles>
int launch(const W4Params& p, const Split& sp, cudaStream_t st) {
  if (p.group == 32) return launch<kTiles, 32>(p, sp, st);
  if (p.group == 64) return launch<kTiles, 64>(p, sp, st);
  return launch<kTiles, 128>(p, sp, st);
}

}  // namespace

extern "C" int gemm_rs_w4_bytes(int64_t N, int64_t K, int group, int has_zeros, size_t* weight_bytes) {
  const int rc = check(0, N, K, group);
  if (rc) return rc;
  if (!weight_bytes) return GEMM_RS_ERR_INVALID_ARG;
  *weight_bytes = (size_t)layout_of(N, K, group, has_zeros != 0).bytes;
  return GEMM_RS_OK;
}

extern "C" int gemm_rs_w4_quantize(int64_t N, int64_t K, int group, const void* W, void* codes, void* scales,
                                   void* stream) {
  int rc = check(0, N, K, group);
  if (rc) return rc;
  if (N == 0 || K == 0) return GEMM_RS_OK;
  if (!W || !codes || !scales) return GEMM_RS_ERR_INVALID_ARG;
  if (misaligned16(W) || misaligned16(codes) || misaligned16(scales)) return GEMM_RS_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  const int groups = (int)((K / kRanks + group - 1) / group);
  w4_quantize_kernel<<<8 * sms, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(W), static_cast<uint8_t*>(codes), static_cast<uint16_t*>(scales), (int)N,
      (int)(K / kRanks), group, groups);
  return launch_status();
}

extern "C" int gemm_rs_w4_pack(int64_t N, int64_t K, int group, const void* codes, const void* scales,
                               const void* zeros, void* weight, void* stream) {
  int rc = check(0, N, K, group);
  if (rc) return rc;
  if (N == 0 || K == 0) return GEMM_RS_OK;
  if (!codes || !scales || !weight) return GEMM_RS_ERR_INVALID_ARG;
  for (const void* q : {codes, scales, zeros, (const void*)weight})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  const Layout l = layout_of(N, K, group, zeros != nullptr);
  uint8_t* base = static_cast<uint8_t*>(weight);
  PackParams p = {(int)N, (int)(K / kRanks), group, (int)l.blocks, (int)l.units, (int)l.groups,
                  (int)((K / kRanks + group - 1) / group),
                  static_cast<const uint8_t*>(codes), static_cast<const uint16_t*>(scales),
                  static_cast<const uint8_t*>(zeros), reinterpret_cast<uint32_t*>(base),
                  reinterpret_cast<uint32_t*>(base + l.scale_off), reinterpret_cast<uint16_t*>(base + l.zero_off)};
  w4_pack_kernel<<<8 * sms, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return launch_status();
}

extern "C" int gemm_rs_w4_run(int64_t M, int64_t N, int64_t K, int group, int has_zeros, const void* x,
                              const void* weight, void* out, void* stream) {
  int rc = check(M, N, K, group);
  if (rc) return rc;
  if (M == 0 || N == 0) return GEMM_RS_OK;
  if (!out || (K > 0 && (!x || !weight))) return GEMM_RS_ERR_INVALID_ARG;
  for (const void* q : {x, weight, (const void*)out})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (K == 0) {
    if (cudaMemsetAsync(out, 0, (size_t)M * N * 2, st) == cudaSuccess) return GEMM_RS_OK;
    cudaGetLastError();
    return GEMM_RS_ERR_CUDA;
  }
  const Layout l = layout_of(N, K, group, has_zeros != 0);
  const uint8_t* base = static_cast<const uint8_t*>(weight);
  W4Params p;
  p.M = (int)M;
  p.N = (int)N;
  p.Kr = (int)(K / kRanks);
  p.group = group;
  p.blocks = (int)l.blocks;
  p.groups = (int)l.groups;
  p.units = (int)l.units;
  const int tiles = (int)((M + 7) / 8);
  Slots slots;
  if (!slots_of(&slots)) return GEMM_RS_ERR_CUDA;
  const Split sp = split_of(M, N, p.units, tiles, slots);
  p.wn = sp.wn;
  p.wk = sp.wk;
  p.part_units = sp.part_units;
  p.chunk_units = sp.chunk_units;
  p.chunks = (sp.part_units + sp.chunk_units - 1) / sp.chunk_units;
  p.pitch = sp.pitch;
  // (in a second wave the request would come when the weights are read anyway)
  p.prefetch_units = sp.at_once ? kPrefetchUnits : 0;
  p.x = static_cast<const uint16_t*>(x);
  p.weights = reinterpret_cast<const uint4*>(base);
  p.scales = reinterpret_cast<const uint32_t*>(base + l.scale_off);
  p.zeros = has_zeros ? reinterpret_cast<const uint16_t*>(base + l.zero_off) : nullptr;
  p.out = static_cast<uint16_t*>(out);
  switch (tiles) {
    case 1: return launch<1>(p, sp, st);
    case 2: return launch<2>(p, sp, st);
    case 3: return launch<3>(p, sp, st);
    default: return launch<4>(p, sp, st);
  }
}
