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
// Unpacking: code c in the low bits of 0x4300 is the bf16 128 + c; subtracting
// 128 + zero is exact, so the tensor core multiplies exact integers with the
// bf16 inputs.  Each group's sum is scaled in fp32 and added to the total.
//
// Split: a cluster of 8 CTAs computes 128 columns, CTA r rank r's share of the
// sum; the eight fp32 partial sums are exchanged through distributed shared
// memory and CTA r writes columns [16 r, 16 r + 16) of the 128, added in rank
// order: the layer's reduce-scatter, inside one cluster.
#include "ops_common.cuh"

using namespace grs;

namespace {

constexpr int kRanks = 8;
constexpr int kWarps = 8;           // each 16 columns
constexpr int kTileN = 16 * kWarps;
constexpr int kCell = 64;           // inner elements of a lane's 16-byte load
constexpr int kMaxTokens = 32;
constexpr int kDepth = 3;           // units (2 cells) of weights in flight per warp
constexpr int kMaxParts = 8;

// Packed buffer: weights [N/16][8][cells][32 lanes] of 16 bytes, then scales
// [N/16][8][groups][8] of two bf16 (columns g and g + 8), then zero points
// [N/16][8][groups][8] of two bytes; N/16 rounded up, cells = K/8/64 rounded up.
// A cell's 64 inner elements: step j of half h holds, in lane 4 g + q, inner
// elements 32 h + 8 q + 4 j + {0, 1, 2, 3} of columns g and g + 8, four bits
// each, at bits 0, 16 (column g, elements 0, 1), 4, 20 (g + 8), 8, 24 (column
// g, elements 2, 3) and 12, 28 of word 2 h + j.
struct Layout {
  long long blocks, cells, groups;
  long long scale_off, zero_off, bytes;
};
Layout layout_of(int64_t N, int64_t K, int group, bool zeros) {
  Layout l;
  const int64_t Kr = K / kRanks;
  l.blocks = (N + 15) / 16;
  l.cells = (Kr + kCell - 1) / kCell;
  l.groups = (Kr + group - 1) / group;
  l.scale_off = l.blocks * kRanks * l.cells * 512;
  l.zero_off = l.scale_off + l.blocks * kRanks * l.groups * 32;
  l.bytes = l.zero_off + (zeros ? l.blocks * kRanks * l.groups * 16 : 0);
  return l;
}

struct W4Params {
  int M, N, Kr, group;
  int blocks, cells, groups;
  int parts, part_cells;       // the cells of a rank are cut into parts of part_cells
  const uint16_t* x;           // [8][M][Kr]
  const uint4* weights;
  const uint32_t* scales;
  const uint16_t* zeros;
  uint16_t* out;               // [M][N]
  float* partial;              // parts > 1: [parts][M][tiles * 128]
  uint32_t* arrived;           // parts > 1: one count for each CTA of a cluster
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// kTiles tiles of 8 tokens, groups of kGroup inner elements.
template <int kTiles, int kGroup, bool kZeros>
__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(32 * kWarps)
    w4_kernel(const W4Params p) {
  __shared__ float sums[kTiles * 8 * kTileN];  // this rank's share: [token][column]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x, tile = blockIdx.y, part = blockIdx.z;
  const int g = lane >> 2, q = lane & 3;
  const int block = tile * kWarps + warp;
  const int c0 = part * p.part_cells;
  const int c1 = c0 + p.part_cells < p.cells ? c0 + p.part_cells : p.cells;

  float acc[kTiles][4];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;

  if (block < p.blocks && c0 < c1) {
    const long long at = (long long)block * kRanks + rank;
    const uint4* w = p.weights + at * p.cells * 32 + lane;
    const uint32_t* sc = p.scales + at * p.groups * 8 + g;
    const uint16_t* zp = kZeros ? p.zeros + at * p.groups * 8 + g : nullptr;
    const uint16_t* x = p.x + (long long)rank * p.M * p.Kr + 8 * q;
    uint4 buf[kDepth][2];
    const uint4 none = make_uint4(0, 0, 0, 0);
    auto fetch = [&](uint4 (&u)[2], int c) {
      u[0] = c < c1 ? __ldcs(w + (long long)c * 32) : none;
      u[1] = c + 1 < c1 ? __ldcs(w + (long long)(c + 1) * 32) : none;
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) fetch(buf[d], c0 + 2 * d);
#pragma unroll 1
    for (int base = c0; base < c1; base += 2 * kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int c = base + 2 * d;
        if (c >= c1) break;
        const uint4 cur[2] = {buf[d][0], buf[d][1]};
        fetch(buf[d], c + 2 * kDepth);
        float sum[kTiles][4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {  // 32 inner elements
          const int k = c * kCell + 32 * h;
          const int grp = k / kGroup;
          if (h % (kGroup / 32) == 0) {
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[t][i] = 0.f;
          }
          // 128 + zero point of columns g and g + 8, in both halves
          uint32_t z0 = 0x43084308u, z1 = 0x43084308u;
          if (kZeros && grp < p.groups) {
            const uint32_t z = __ldg(zp + grp * 8);
            z0 = 0x43004300u | (z & 0xFFu) * 0x10001u;
            z1 = 0x43004300u | (z >> 8) * 0x10001u;
          }
          uint4 xv[kTiles];
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            const int m = 8 * t + g;
            xv[t] = m < p.M && k + 8 * q < p.Kr
                        ? __ldg(reinterpret_cast<const uint4*>(x + (long long)m * p.Kr + k))
                        : none;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4& v = cur[h >> 1];
            const uint32_t word = (h & 1) ? (j ? v.w : v.z) : (j ? v.y : v.x);
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              a[i] = sub_bf16x2(((word >> (4 * i)) & 0x000F000Fu) | 0x43004300u, (i & 1) ? z1 : z0);
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
              mma_16816(sum[t], a, j ? xv[t].z : xv[t].x, j ? xv[t].w : xv[t].y);
          }
          if ((h + 1) % (kGroup / 32) == 0) {
            const uint32_t s = grp < p.groups ? __ldg(sc + grp * 8) : 0u;
            const float s0 = bf16lo_to_f32(s), s1 = bf16hi_to_f32(s);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              acc[t][0] = fmaf(s0, sum[t][0], acc[t][0]);
              acc[t][1] = fmaf(s0, sum[t][1], acc[t][1]);
              acc[t][2] = fmaf(s1, sum[t][2], acc[t][2]);
              acc[t][3] = fmaf(s1, sum[t][3], acc[t][3]);
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sums[(8 * t + 2 * q + (i & 1)) * kTileN + warp * 16 + g + 8 * (i >> 1)] = acc[t][i];
  cluster_sync();  // every rank's share is in its shared memory

  // CTA r adds columns [16 r, 16 r + 16) in rank order
  const uint32_t mine = smem_u32(sums);
  for (int i = threadIdx.x; i < 16 * p.M; i += blockDim.x) {
    const int m = i >> 4, col = rank * 16 + (i & 15);
    const int n = tile * kTileN + col;
    float s = 0.f;
#pragma unroll
    for (uint32_t r = 0; r < kRanks; ++r) s += ld_cluster_f32(mapa_shared(mine, r) + 4u * (m * kTileN + col));
    if (p.parts > 1)
      __stcg(p.partial + ((long long)part * p.M + m) * (gridDim.y * kTileN) + n, s);
    else if (n < p.N)
      p.out[(long long)m * p.N + n] = (uint16_t)(pack_bf16x2(s, 0.f) & 0xFFFFu);
  }
  cluster_sync();  // no CTA leaves while its share is being read
  if (p.parts == 1) return;

  // the last part to arrive adds the parts in order
  __shared__ uint32_t last;
  __threadfence();
  __syncthreads();
  uint32_t* count = p.arrived + tile * kRanks + rank;
  if (threadIdx.x == 0) last = atomicAdd(count, 1u) == (uint32_t)p.parts - 1u;
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int i = threadIdx.x; i < 16 * p.M; i += blockDim.x) {
    const int m = i >> 4, n = tile * kTileN + rank * 16 + (i & 15);
    if (n >= p.N) continue;
    float s = 0.f;
    for (int z = 0; z < p.parts; ++z)
      s += __ldcg(p.partial + ((long long)z * p.M + m) * (gridDim.y * kTileN) + n);
    p.out[(long long)m * p.N + n] = (uint16_t)(pack_bf16x2(s, 0.f) & 0xFFFFu);
  }
  if (threadIdx.x == 0) *count = 0;  // ready for the next call
}

struct PackParams {
  int N, Kr, group, blocks, cells, groups;
  const uint8_t* codes;    // [8][Kr][N]
  const uint16_t* scales;  // [8][groups][N]
  const uint8_t* zeros;    // [8][groups][N] or null
  uint32_t* weights;
  uint32_t* out_scales;
  uint16_t* out_zeros;
};

// One 32-bit word (8 codes) a thread, then the groups' scales and zero points.
__global__ void __launch_bounds__(256) w4_pack_kernel(const PackParams p) {
  const long long stride = (long long)gridDim.x * blockDim.x;
  const long long first = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long words = (long long)p.blocks * kRanks * p.cells * 128;
  for (long long i = first; i < words; i += stride) {
    const int step = (int)(i & 3), lane = (int)(i >> 2) & 31;
    const long long cell = i >> 7;
    const int c = (int)(cell % p.cells);
    const int r = (int)(cell / p.cells % kRanks);
    const int block = (int)(cell / p.cells / kRanks);
    const int k0 = c * kCell + 32 * (step >> 1) + 8 * (lane & 3) + 4 * (step & 1);
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i4 = e >> 1;  // MMA register: column g or g + 8, inner pair 0 or 1
      const int n = block * 16 + (lane >> 2) + 8 * (i4 & 1);
      const int k = k0 + 2 * (i4 >> 1) + (e & 1);
      if (n < p.N && k < p.Kr)
        w |= (uint32_t)(p.codes[((long long)r * p.Kr + k) * p.N + n] & 15u) << (4 * i4 + 16 * (e & 1));
    }
    p.weights[i] = w;
  }
  const long long metas = (long long)p.blocks * kRanks * p.groups * 8;
  for (long long i = first; i < metas; i += stride) {
    const int g = (int)(i & 7);
    const long long t = i >> 3;
    const int grp = (int)(t % p.groups);
    const int r = (int)(t / p.groups % kRanks);
    const int n = (int)(t / p.groups / kRanks) * 16 + g;
    const long long row = ((long long)r * p.groups + grp) * p.N;
    const uint32_t lo = n < p.N ? p.scales[row + n] : 0u, hi = n + 8 < p.N ? p.scales[row + n + 8] : 0u;
    p.out_scales[i] = lo | hi << 16;
    if (p.zeros) {
      const uint32_t zl = n < p.N ? p.zeros[row + n] & 127u : 0u, zh = n + 8 < p.N ? p.zeros[row + n + 8] & 127u : 0u;
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
  if (M < 0 || M > kMaxTokens || N < 0 || K < 0 || N % 8 || K % 64 || N > (1ll << 22) || K > (1ll << 30))
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  return GEMM_RS_OK;
}

// Few columns leave SMs idle: the inner dimension is then cut into parts (of
// an even number of cells, so that a group stays whole).
void split_of(const Layout& l, int64_t N, int* parts, int* part_cells) {
  const long long ctas = (N + kTileN - 1) / kTileN * kRanks;
  long long want = ctas > 0 ? 304 / ctas : 1;
  const long long units = (l.cells + 1) / 2;
  if (want > kMaxParts) want = kMaxParts;
  if (want > units / 4) want = units / 4;  // at least 8 cells (4 KiB a warp) in a part
  if (want < 1) want = 1;
  const long long per = (units + want - 1) / want;
  *part_cells = (int)(2 * per);
  *parts = (int)(per > 0 ? (units + per - 1) / per : 1);
  if (*parts < 1) *parts = 1;
}

template <int kTiles, int kGroup>
void launch(const W4Params& p, dim3 grid, cudaStream_t st) {
  if (p.zeros)
    w4_kernel<kTiles, kGroup, true><<<grid, 32 * kWarps, 0, st>>>(p);
  else
    w4_kernel<kTiles, kGroup, false><<<grid, 32 * kWarps, 0, st>>>(p);
}
template <int kTiles>
void launch(const W4Params& p, dim3 grid, cudaStream_t st) {
  if (p.group == 32)
    launch<kTiles, 32>(p, grid, st);
  else if (p.group == 64)
    launch<kTiles, 64>(p, grid, st);
  else
    launch<kTiles, 128>(p, grid, st);
}

}  // namespace

extern "C" int gemm_rs_w4_bytes(int64_t N, int64_t K, int group, int has_zeros, size_t* weight_bytes,
                                size_t* workspace_bytes) {
  const int rc = check(0, N, K, group);
  if (rc) return rc;
  const Layout l = layout_of(N, K, group, has_zeros != 0);
  if (weight_bytes) *weight_bytes = (size_t)l.bytes;
  if (workspace_bytes) {
    int parts = 1, cells = 0;
    split_of(l, N, &parts, &cells);
    const size_t tiles = (size_t)(N + kTileN - 1) / kTileN;
    *workspace_bytes = tiles * kRanks * 4 + (parts > 1 ? (size_t)parts * kMaxTokens * tiles * kTileN * 4 : 0);
  }
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
  const Layout l = layout_of(N, K, group, false);
  w4_quantize_kernel<<<8 * sms, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(W), static_cast<uint8_t*>(codes), static_cast<uint16_t*>(scales), (int)N,
      (int)(K / kRanks), group, (int)l.groups);
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
  PackParams p = {(int)N, (int)(K / kRanks), group, (int)l.blocks, (int)l.cells, (int)l.groups,
                  static_cast<const uint8_t*>(codes), static_cast<const uint16_t*>(scales),
                  static_cast<const uint8_t*>(zeros), reinterpret_cast<uint32_t*>(base),
                  reinterpret_cast<uint32_t*>(base + l.scale_off), reinterpret_cast<uint16_t*>(base + l.zero_off)};
  w4_pack_kernel<<<8 * sms, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return launch_status();
}

extern "C" int gemm_rs_w4_run(int64_t M, int64_t N, int64_t K, int group, int has_zeros, const void* x,
                              const void* weight, void* out, void* workspace, void* stream) {
  int rc = check(M, N, K, group);
  if (rc) return rc;
  if (M == 0 || N == 0) return GEMM_RS_OK;
  if (!out || (K > 0 && (!x || !weight))) return GEMM_RS_ERR_INVALID_ARG;
  if (!workspace) return GEMM_RS_ERR_WORKSPACE;
  for (const void* q : {x, weight, (const void*)out, (const void*)workspace})
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
  const int tiles = (int)((N + kTileN - 1) / kTileN);
  W4Params p;
  p.M = (int)M;
  p.N = (int)N;
  p.Kr = (int)(K / kRanks);
  p.group = group;
  p.blocks = (int)l.blocks;
  p.cells = (int)l.cells;
  p.groups = (int)l.groups;
  split_of(l, N, &p.parts, &p.part_cells);
  p.x = static_cast<const uint16_t*>(x);
  p.weights = reinterpret_cast<const uint4*>(base);
  p.scales = reinterpret_cast<const uint32_t*>(base + l.scale_off);
  p.zeros = has_zeros ? reinterpret_cast<const uint16_t*>(base + l.zero_off) : nullptr;
  p.out = static_cast<uint16_t*>(out);
  p.arrived = static_cast<uint32_t*>(workspace);
  p.partial = reinterpret_cast<float*>(p.arrived + tiles * kRanks);
  const dim3 grid(kRanks, (unsigned)tiles, (unsigned)p.parts);
  if (M <= 8)
    launch<1>(p, grid, st);
  else if (M <= 16)
    launch<2>(p, grid, st);
  else
    launch<4>(p, grid, st);
  return launch_status();
}
