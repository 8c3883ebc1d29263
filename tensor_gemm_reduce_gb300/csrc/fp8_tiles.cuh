// fp8_tiles.cuh -- what the two product kernels of e4m3 operands share (fp8_gemm.cu: scales that are powers
// of two; fp8_gemm_f32.cu: fp32): tiles and their order, the loads of their operands, whole-line
// stores and launches.
//
// Tiles of 256 x 256, one at a time for each pair of CTAs (cta_group::2).  Operands are read as
// they lie in memory, K-major or MN-major, through TMA.  dA and dW are independent, so a
// backward pass may multiply both in one launch, dA's tiles first.
#pragma once
#include <cuda.h>

#include <cstring>

#include "fp8.cuh"
#include "mx.cuh"
#include "tensor_pipe.cuh"

namespace grs {
namespace tiles {

constexpr int kTile = 256;
constexpr int kStages = 6;
constexpr int kOperand = 128 * kBlk;  // bytes of one CTA's half of an operand in a stage
constexpr int kEpiWarps = 8;
constexpr int kWarps = 4 + kEpiWarps;
constexpr int kThreads = 32 * kWarps;
constexpr int kSmemB = kStages * kOperand;
constexpr int kSmemScales = 2 * kStages * kOperand;
constexpr int kBufBytes = 16 * 128;  // of an epilogue warp
constexpr uint64_t kLimitNs = 2000000000ull;  // of every wait

constexpr int kBothGrads = 3;  // Fp8Kind of a launch with the tiles of dA, then of dW

// One of a launch's products.
struct Side {
  CUtensorMap a, b;
  const void* a_scale;  // a word for each row and step, bytes' for four steps
  const void* b_scale;  // weight grad: likewise for columns; else the weight's
  void* out_ptr;
  long long a_stride, b_stride;  // words from one step's scales (bytes: four steps') to the next
  int nt;          // tiles along the output's columns, planes included
  int band;
  // One expert, or weight grad: every expert has mt x nt tiles in bands of `band`, the last one
  // of `last`; each division by these is a multiplication.
  int mt, last;
  Divider by_expert, by_band, by_band_rows, by_last_rows, by_plane;
};
struct Shared {
  const int* offsets;
  uint32_t* status;
  int M, N, Kr, experts, KB, NB, out_f32, parts;
  int blocks;      // weight grad: of 128 tokens in the operands
};
template <int kKind>
struct Params : Shared {
  Side sides[kKind == kBothGrads ? 2 : 1];
};

// A pair's tiles.  All warps walk them alike.
struct Tile {
  int kind;
  int e;                // expert
  int plane;            // rank, where the output has one for each; forward: part of the contraction
  int row0, row_end;    // output rows: the tile's first, the first behind the expert's last
  int col0;             // output column within the plane
  int steps, step0;     // steps of 128; weight grad: the first one's token block
};

// What a tile belongs to: constants in a launch of one product.
template <int kKind>
__device__ __forceinline__ int kind_of(const Tile& t) {
  return kKind == kBothGrads ? t.kind : kKind;
}
template <int kKind>
__device__ __forceinline__ const Side& side_of(const Params<kKind>& p, const Tile& t) {
  return p.sides[kKind == kBothGrads && t.kind == kFp8WeightGrad ? 1 : 0];
}

template <int kKind>
struct Walk {
  const Params<kKind>& p;
  const int* start;   // [experts + 1] first tile of each expert
  const int* blocks;  // weight grad: [experts + 1] first token block
  int idx, tiles, total;  // tiles: those in front of the weight grad's
  const int stride;
  __device__ Walk(const Params<kKind>& params, const int* s, const int* b, int pair, int pairs)
      : p(params), start(s), blocks(b), idx(pair), stride(pairs) {
    const Side& w = p.sides[kKind == kBothGrads ? 1 : 0];
    tiles = kKind == kFp8WeightGrad ? 0 : start[p.experts];
    total = tiles * (kKind == kFp8Forward ? p.parts : 1) + (kKind == kFp8WeightGrad || kKind == kBothGrads ? p.experts * w.mt * w.nt : 0);
  }
  // Tile `i` of an expert with the launch's mt x nt tiles, in the order of region_at (four divisions
  // by run-time values took longer than a short tile's products).
  __device__ Region region(const Side& d, uint32_t i) const {
    const uint32_t b = divided(i, d.by_band), rem = i - b * (uint32_t)(d.band * d.nt);
    const int mt0 = (int)b * d.band;
    const bool whole = mt0 + d.band <= d.mt;
    const uint32_t q = divided(rem, whole ? d.by_band_rows : d.by_last_rows);
    return Region{mt0 + (int)(rem - q * (uint32_t)(whole ? d.band : d.last)), (int)q};
  }
  __device__ bool next(Tile* t) {
    if (idx >= total) return false;
    t->kind = kKind != kBothGrads ? kKind : idx < tiles ? kFp8InputGrad : kFp8WeightGrad;
    const int kind = kind_of<kKind>(*t);
    const Side& d = side_of(p, *t);
    if (kind == kFp8WeightGrad) {
      const int i = idx - tiles;
      t->e = (int)divided((uint32_t)i, d.by_expert);
      const Region g = region(d, (uint32_t)(i - t->e * d.mt * d.nt));
      t->plane = (int)divided((uint32_t)g.mt, d.by_plane);
      t->row0 = (g.mt - t->plane * (d.mt / kWorld)) * kTile;
      t->row_end = p.Kr;
      t->col0 = g.nt * kTile;
      t->step0 = blocks[t->e];
      t->steps = blocks[t->e + 1] - t->step0;
    } else {
      Region g;
      int r0 = 0, r1 = p.M, part = 0;
      t->e = 0;
      if (!p.offsets) {
        if (kind == kFp8Forward) part = (int)divided((uint32_t)idx, d.by_expert);
        g = region(d, (uint32_t)(idx - part * d.mt * d.nt));
      } else {
        int lo = 0, hi = p.experts;  // the last expert whose first tile is not behind idx
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (start[mid] <= idx) lo = mid; else hi = mid;
        }
        t->e = lo;
        r0 = expert_row(p.offsets, lo, p.M);
        r1 = expert_row(p.offsets, lo + 1, p.M);
        const int mt = (r1 - r0 + kTile - 1) / kTile;
        g = region_at(idx - start[lo], mt, d.nt, d.band < mt ? d.band : mt);
      }
      t->row0 = r0 + g.mt * kTile;
      t->row_end = r1;
      t->step0 = 0;
      if (kind == kFp8Forward) {
        t->plane = part;
        t->col0 = g.nt * kTile;
        t->steps = kWorld * p.KB;
        if (p.parts > 1) {
          const int all = t->steps;
          t->step0 = all * part / p.parts;
          t->steps = all * (part + 1) / p.parts - t->step0;
        }
      } else {
        t->plane = (int)divided((uint32_t)g.nt, d.by_plane);
        t->col0 = (g.nt - t->plane * (d.nt / kWorld)) * kTile;
        t->steps = p.NB;
      }
    }
    idx += stride;
    return true;
  }
};

// The plane of the weight's map that is its 128 columns from 128 nb on.  A tile's second half may
// lie behind the last: that plane's values go to columns that are not stored.
__device__ __forceinline__ int weight_block(const Shared& p, int plane, int nb) {
  return plane * p.NB + (nb < p.NB ? nb : p.NB - 1);
}

// A warp's 32 rows of 128 bytes (w: a lane's row) to global memory in whole lines, 16 rows
// at a time through its buffer: lanes that each store their own row write sectors one by
// one, which took 512 x 8192 x 28672 dW from 123 us without stores to 178.  Row i of `rows` goes to
// out + i * pitch; of a row, the first `bytes`.
__device__ __forceinline__ void store_rows(uint32_t buf, const uint32_t (&w)[32], int lane, char* out, long long pitch, int rows,
                                           int bytes) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if ((lane >> 4) == h) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        st_shared_v4(buf + (lane & 15) * 128 + (uint32_t)((j ^ (lane & 7)) << 4), w[4 * j], w[4 * j + 1], w[4 * j + 2],
                     w[4 * j + 3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * i + (lane >> 3), c = lane & 7;
      uint4 v;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(buf + r * 128 + (uint32_t)((c ^ (r & 7)) << 4))
                   : "memory");
      if (16 * h + r < rows && c * 16 < bytes) st_global_v4(out + (16 * h + r) * pitch + c * 16, v);
    }
    __syncwarp();
  }
}

// A warp's 32 rows x 128 columns of the tile (v: a lane's row) to the output, rounded where it is bf16.
template <int kKind>
__device__ __forceinline__ void store_tile(const Params<kKind>& p, const Tile& t, int cta, int q, int half, int lane,
                                           uint32_t buf, const uint32_t (&v)[4][32]) {
  const int row0 = t.row0 + cta * 128 + q * 32, col0 = t.col0 + half * 128;
  const int rows = t.row_end - row0;
  if (rows > 0) {
    const int kind = kind_of<kKind>(t), cols = kind == kFp8InputGrad ? p.Kr : p.N;
    const int plane = kind == kFp8WeightGrad ? t.e * kWorld + t.plane : t.plane;
    const int rows_all = kind == kFp8WeightGrad ? p.Kr : p.M;  // of a plane
    void* const out = side_of(p, t).out_ptr;
    const long long at = ((long long)plane * rows_all + row0) * cols + col0;
    if (kKind == kFp8Forward && p.out_f32) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (col0 + 32 * c < cols)
          store_rows(buf, v[c], lane, reinterpret_cast<char*>(static_cast<float*>(out) + at + 32 * c),
                     (long long)cols * 4, rows, (cols - col0 - 32 * c) * 4);
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (col0 + 64 * c >= cols) break;
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i)
          w[i] = pack_bf16x2(__uint_as_float(v[2 * c + (i >> 4)][2 * (i & 15)]),
                             __uint_as_float(v[2 * c + (i >> 4)][2 * (i & 15) + 1]));
        store_rows(buf, w, lane, reinterpret_cast<char*>(static_cast<uint16_t*>(out) + at + 64 * c),
                   (long long)cols * 2, rows, (cols - col0 - 64 * c) * 2);
      }
    }
  }
}

// Where each expert's tiles (or token blocks) start: rows in units, `per` tiles for each.  A whole warp.
__device__ __forceinline__ void count_starts(const Shared& p, int lane, int* first, int unit, int per, int most) {
  int before = 0;
  for (int e0 = 0; e0 < p.experts; e0 += 32) {
    const int e = e0 + lane;
    int n = 0;
    if (e < p.experts) {
      const int rows = p.offsets ? expert_row(p.offsets, e + 1, p.M) - expert_row(p.offsets, e, p.M) : p.M;
      n = rows > 0 ? (rows + unit - 1) / unit * per : 0;
    }
    int sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += up;
    }
    const int at = before + sum - n;
    if (e < p.experts) first[e] = at < most ? at : most;
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (lane == 0) first[p.experts] = before < most ? before : most;
}

// One thread loads this CTA's half of an operand (is_a: of A) for every step of the pair's tiles; the
// first CTA's barriers count both CTAs' bytes.
template <int kKind>
__device__ __forceinline__ void load_operand(const Params<kKind>& p, Walk<kKind>& walk, bool is_a, int cta, uint32_t sbase,
                                             uint32_t bar_full, volatile uint32_t* cta_abort, uint32_t abort_addr) {
  Tile t;
  const uint32_t base = sbase + (is_a ? 0 : kSmemB), bar_empty = bar_full + 8 * kStages;
  int stage = 0;
  uint32_t phase = 0, issued = 0, issued_par = 0;
  bool ok = true;
  while (ok && walk.next(&t)) {
    const int x0 = (is_a ? t.row0 : t.col0) + cta * 128;  // this CTA's half
    const int kind = kind_of<kKind>(t);
    const Side& d = side_of(p, t);
    const CUtensorMap* map = is_a ? &d.a : &d.b;
    int r = 0, kb = 0;
    if (kKind == kFp8Forward && p.parts > 1) {
      r = t.step0 / p.KB;
      kb = t.step0 - r * p.KB;
    }
    for (int s = 0; s < t.steps; ++s) {
      if (!wait_bar(bar_empty + 8 * stage, phase ^ 1u, kLimitNs, cta_abort)) {
        give_up(abort_addr);
        ok = false;
        break;
      }
      const uint32_t fb = bar_full + 8 * stage, fb0 = mapa_shared(fb, 0);
      const uint32_t dst = base + stage * kOperand;
      if (cta == 0) mbar_arrive_expect_tx(fb, 2 * kOperand);
      if (kind == kFp8Forward) {
        if (is_a)
          tma_load_3d_pair(dst, map, fb0, kb * kBlk, x0, r);
        else
          tma_load_3d_pair(dst, map, fb0, 0, kb * kBlk, weight_block(p, t.e * kWorld + r, x0 / kBlk));
        if (++kb == p.KB) {
          kb = 0;
          ++r;
        }
      } else if (kind == kFp8InputGrad) {
        if (is_a)
          tma_load_3d_pair(dst, map, fb0, s * kBlk, x0, 0);
        else
          tma_load_3d_pair(dst, map, fb0, 0, x0, weight_block(p, t.e * kWorld + t.plane, s));
      } else {
        tma_load_3d_pair(dst, map, fb0, x0, (t.step0 + s) * kBlk, is_a ? t.plane : 0);
      }
      issued |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  // every copy lands before the CTA can exit (the first CTA's barriers
  // count both CTAs' bytes; a pair that gave up waits in settle() below)
  if (cta == 0)
    for (int s = 0; s < kStages; ++s)
      if ((issued & (1u << s)) && !wait_bar(bar_full + 8 * s, (issued_par >> s) & 1u, kDrainNs, cta_abort))
        give_up(abort_addr);
}

inline bool map8(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t planes, int64_t pitch) {
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, cols, rows, planes, kBlk, kBlk, pitch);
}

// Pairs of a kernel that run at the same time on the current device.  kRegs: what the warps of a CTA hold
// after they exchange registers, where they do; with fewer at launch they would wait for ever.
template <int kKind, void (*kKernel)(Params<kKind>), int kSmem, int kRegs>
int max_pairs(int sms, int* pairs) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return GEMM_RS_ERR_CUDA;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaFuncAttributes attr;
    if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaFuncGetAttributes(&attr, kKernel) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_RS_ERR_CUDA;
    }
    if (attr.numRegs * kThreads < kRegs) return GEMM_RS_ERR_UNSUPPORTED_DEVICE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u * (unsigned)(sms / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    if (cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_RS_ERR_CUDA;
    }
    if (n < 1) return GEMM_RS_ERR_UNSUPPORTED_DEVICE;
    if (n > sms / 2) n = sms / 2;
    known[dev].store(n, std::memory_order_relaxed);
  }
  *pairs = n;
  return GEMM_RS_OK;
}

inline int64_t tiles_of_dim(int64_t n) { return (n + kTile - 1) / kTile; }

template <int kKind, void (*kKernel)(Params<kKind>), int kSmem, int kRegs>
int launch(const Params<kKind>& p, int64_t most_tiles, cudaStream_t st) {
  int sms = 0, pairs = 0;
  int rc = current_device_sms(&sms);
  if (rc) return rc;
  rc = max_pairs<kKind, kKernel, kSmem, kRegs>(sms, &pairs);
  if (rc) return rc;
  if (pairs > most_tiles) pairs = (int)most_tiles;
  return launch_overlapped(kKernel, dim3(2u * (unsigned)pairs), kThreads, kSmem, st, p);
}

// What all products of these rows share.
inline void fill(Shared* p, const Fp8Product& d) {
  p->offsets = d.rows.offsets;
  p->status = d.status;
  p->M = (int)d.rows.M;
  p->N = (int)d.N;
  p->Kr = (int)d.Kr;
  p->experts = (int)d.rows.experts;
  p->KB = (int)blocks_of(d.Kr);
  p->NB = (int)blocks_of(d.N);
  p->out_f32 = d.out_f32;
  p->parts = d.parts;
  p->blocks = (int)(padded_rows(d.rows.M, d.rows.offsets ? d.rows.experts : 1) / kBlk);
}

// One product, and its tiles at most; 0: the maps cannot be encoded.
inline int64_t fill(Side* s, const Fp8Product& d) {
  const int64_t M = d.rows.M, N = d.N, Kr = d.Kr, E = d.rows.experts;
  const int64_t pk = fp8_pitch(Kr), pn = fp8_pitch(N), padded = padded_rows(M, d.rows.offsets ? E : 1);
  s->a_scale = d.a_scale;
  s->b_scale = d.b_scale;
  s->out_ptr = d.out;
  int64_t per_plane = 1;  // tiles of a plane along the axis that planes share
  bool ok;
  if (d.kind == kFp8WeightGrad) {
    s->nt = (int)tiles_of_dim(N);
    s->mt = (int)(kWorld * tiles_of_dim(Kr));
    per_plane = s->mt / kWorld;
    s->a_stride = kWorld * pk;
    s->b_stride = pn;
    s->band = auto_band(kWorld * tiles_of_dim(Kr) * kTile, M / 2, kTile);
    ok = map8(&s->a, d.a, Kr, padded, kWorld, pk) && map8(&s->b, d.b, N, padded, 1, pn);
  } else {
    const bool fwd = d.kind == kFp8Forward;
    s->nt = (int)(fwd ? tiles_of_dim(N) : kWorld * tiles_of_dim(Kr));
    s->mt = (int)tiles_of_dim(M);
    if (!fwd) per_plane = s->nt / kWorld;
    s->a_stride = row_scale_pitch(M);
    // bytes of the codes of a band's rows, as auto_band counts them for two-byte elements
    s->band = auto_band(M, fwd ? kWorld * Kr / 2 : N / 2, kTile);
    ok = (fwd ? map8(&s->a, d.a, Kr, M, kWorld, pk) : map8(&s->a, d.a, N, M, 1, pn)) &&
         map8(&s->b, d.b, kBlk, Kr, kWorld * E * blocks_of(N), kBlk);
  }
  s->last = s->mt - (s->mt - 1) / s->band * s->band;
  s->by_expert = divider_of((uint32_t)(s->mt * s->nt));
  s->by_band = divider_of((uint32_t)(s->band * s->nt));
  s->by_band_rows = divider_of((uint32_t)s->band);
  s->by_last_rows = divider_of((uint32_t)s->last);
  s->by_plane = divider_of((uint32_t)per_plane);
  if (!ok) return 0;
  return d.kind == kFp8WeightGrad ? E * s->mt * s->nt : (s->mt + (d.rows.offsets ? E : 0)) * s->nt;
}

}  // namespace tiles
}  // namespace grs
