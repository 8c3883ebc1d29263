// backward.cu -- backward pass of the row-parallel layer from an 8-bit
// checkpoint of its input (gemm_rs_bwd_* in include/gemm_rs_ops.h):
//   dA_r = dY W_r^T   (rows M, columns K/8, contraction over N)
//   dW_r = A_r^T dY   (rows K/8, columns N, contraction over M)
//
// One persistent kernel computes both products in 256 x 256 tiles, one tile at
// a time for each pair of CTAs (tcgen05 cta_group::2, fp32 accumulators in
// TMEM, two of them so that one tile's epilogue overlaps the next tile's
// MMAs).  dA's operands are K-major as they lie in memory (dY's rows and W's
// rows both run along N); dW's are both MN-major (A's rows run along K/8, dY's
// along N, and the contraction runs over tokens), so nothing is transposed.
// Warp roles in each CTA: 0 loads the A operand, 6 the B operand, 1 issues the
// MMAs (first CTA of the pair), 2 to 5 run the epilogue.
//
// Bound by the tensor cores and, in a row of launches, by the card's power: 2048 x
// 8192 x 8192 (550 GFLOP) takes 276 us alone at the full clock (tensor pipe active
// 94%) and 330 us repeated, restore included: 1.65 PFLOP/s, 0.98 of what a plain
// library product sustains and 0.86 of its burst; 512 x 8192 x 28672 338 us,
// 1.42 PFLOP/s (its dW tiles contract over 8 steps, so what a tile costs besides,
// 500 to 1000 cycles, and 1 GB of operands and outputs weigh more).
// Every wait is bounded; on expiry both CTAs of the pair stop, leave their copies and
// MMAs the time to end, free TMEM and return.  Each CTA says at its end, in a word of
// its own, whether it gave up, so nothing has to be cleared before a run, whatever the
// workspace held.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>
#include <new>

#include "act8.cuh"
#include "ops_common.cuh"
#include "schedule.h"

using namespace grs;

namespace {

constexpr int kTile = 256;  // rows and columns of a pair's tile
constexpr int kStages = 6;
constexpr int kOperand = 128 * kBK * 2;  // bytes of one CTA's half of an operand in a stage
constexpr int kEpiWarps = 4;
constexpr int kEpiBufBytes = 32 * 64 * 2;  // a warp's 32 rows x 64 columns of bf16
constexpr int kWarps = 7;
constexpr int kSmemB = kStages * kOperand;
constexpr int kSmemEpi = 2 * kStages * kOperand;
constexpr int kSmemBar = kSmemEpi + kEpiWarps * 2 * kEpiBufBytes;
constexpr int kNumBars = 2 * kStages + 5;  // full, empty, acc_full[2], acc_empty[2], drain
constexpr int kSmemMisc = kSmemBar + kNumBars * 8;
constexpr int kSmemAlloc = kSmemMisc + 16 + 1024;  // slack to align the base to 1024 bytes
static_assert(kSmemAlloc <= 232448, "shared memory per CTA");
// Elements of a checkpoint up to which it is restored beside the dA tiles (M x N x K:
// 392 x 776 x 1600 11.7 -> 11.1 us, 128 x 8192 x 8192 59.3 -> 57.7; above, 480 x 256 x
// 12928 16.0 -> 17.0, 1000 x 1032 x 6400 35.8 -> 37.1, the largest no difference).
constexpr int64_t kRestoreBeside = 2 << 20;
constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
// What is in flight when a CTA has nothing more to issue ends within microseconds.
constexpr uint64_t kDrainNs = 100000000ull;   // bound of the waits for it, whatever the caller's limit
constexpr uint64_t kSettleNs = 10000000ull;   // time that a pair leaves it after giving up
// The workspace: a status word for each CTA, then the restored activations.  The words
// come first so that plans of any sizes which share a workspace agree on the place.
constexpr int kStatusWords = 256;
constexpr size_t kStatusBytes = kStatusWords * sizeof(uint32_t);

// One of the two products: 8 ranks of mt x nt tiles, kb steps of kBK each.
struct Product {
  int mt, nt, kb, band;
  __host__ __device__ int per_rank() const { return mt * nt; }
  __host__ __device__ int tiles() const { return kWorld * mt * nt; }
};

// Which tiles a pair computes: the dA tiles c, c + pairs, ... first (their
// contraction is usually the longer one), then dW tiles.  When the dA tiles do
// not divide evenly, pairs from `extra` on have one fewer: each of them takes
// `early` dW tiles while the others work on their last dA tile; the remaining
// dW tiles are dealt in turn, starting with those pairs.
struct Schedule {
  Product da, dw;
  int pairs, extra, early;
};

struct Tile {
  bool is_dw;
  int rank, mt, nt;
};

struct TileWalk {
  int c, i = 0;
  __host__ __device__ explicit TileWalk(int pair) : c(pair) {}
  __host__ __device__ bool next(const Schedule& s, Tile* t) {
    int idx = c + i * s.pairs;
    const int mine = s.da.tiles() > c ? (s.da.tiles() - c + s.pairs - 1) / s.pairs : 0;
    const Product* p = &s.da;
    t->is_dw = i >= mine;
    if (t->is_dw) {
      p = &s.dw;
      int j = i - mine;
      const bool is_short = s.extra > 0 && c >= s.extra;
      const int spare = s.extra > 0 ? s.pairs - s.extra : 0;
      if (is_short && j < s.early) {
        idx = (c - s.extra) + j * spare;
      } else {
        if (is_short) j -= s.early;
        const int turn = c >= s.extra ? c - s.extra : c + s.pairs - s.extra;
        idx = s.early * spare + turn + j * s.pairs;
      }
      if (idx >= s.dw.tiles()) {
        // an early tile may be past the end only if every later one is too
        return false;
      }
    }
    ++i;
    t->rank = idx / p->per_rank();
    const Region g = region_at(idx - t->rank * p->per_rank(), p->mt, p->nt, p->band);
    t->mt = g.mt;
    t->nt = g.nt;
    return true;
  }
};

struct BwdParams {
  // Loads: dY and W K-major (box 64 along N x 128 rows), A and dY MN-major
  // (box 64 columns x 64 tokens).  Stores: 64 columns x 32 rows.
  CUtensorMap dy_k, w_k, a_mn, dy_mn, out_da, out_dw;
  Schedule s;
  int M, N, Kr;
  uint32_t* status;  // [CTA] written at its end: non-zero if a wait gave up
  int restored_before;  // the launch before this one restores A and lets this one start early
  unsigned long long timeout_ns;
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                         volatile uint32_t* cta_abort, bool cluster = false) {
  auto probe = [&]() {
    return cluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
  };
  if (probe()) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 128; ++i)
      if (probe()) return true;
    if (*cta_abort || globaltimer_ns() - t0 > limit_ns) return false;
  }
}

// A wait ran out: both CTAs of the pair stop at their next wait that does not succeed.
__device__ __forceinline__ void give_up(uint32_t abort_addr) {
#pragma unroll
  for (uint32_t cta = 0; cta < 2; ++cta)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(abort_addr, cta)), "r"(1) : "memory");
}

// Time for the copies and MMAs of a pair that gave up.  Waiting for their barriers does
// not do: a stage that one of the pair's four loaders never filled never completes, and
// the others' bytes for it may still be on their way.
__device__ __noinline__ void settle() {
  const uint64_t t0 = globaltimer_ns();
  for (int i = 0; i < (1 << 20) && globaltimer_ns() - t0 < kSettleNs; ++i) __nanosleep(1000);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(32 * kWarps, 1)
    backward_kernel(const __grid_constant__ BwdParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = (int)cluster_ctarank();
  const int pair = blockIdx.x >> 1;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_full = sbase + kSmemBar;
  const uint32_t bar_empty = bar_full + 8 * kStages;
  const uint32_t bar_acc_full = bar_empty + 8 * kStages;
  const uint32_t bar_acc_empty = bar_acc_full + 16;
  const uint32_t bar_drain = bar_acc_empty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmemMisc);
  volatile uint32_t* cta_abort = reinterpret_cast<volatile uint32_t*>(smem + kSmemMisc + 4);
  const uint32_t abort_addr = sbase + kSmemMisc + 4;
  const uint64_t limit = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_full + 8 * s, 2);   // the first CTA's two loaders (+ both CTAs' bytes)
      mbar_init(bar_empty + 8 * s, 1);  // one MMA commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_acc_full + 8 * b, 1);
      mbar_init(bar_acc_empty + 8 * b, 2 * kEpiWarps);
    }
    mbar_init(bar_drain, 1);
    *cta_abort = 0;
    fence_mbar_init();
    fence_proxy_async_shared();
  }
  if (warp == 1) {
    tmem_alloc<2>(smem_u32(tmem_slot), 512);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  // restored_before: the kernel before this one is the checkpoint's restoration,
  // which lets this grid start when everything before it is complete, so the dA
  // tiles need not wait; the A loader waits for it before the first dW tile.
  if (!p.restored_before) griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const uint32_t tmem_base = *tmem_slot;
  TileWalk walk(pair);
  Tile t;

  if (warp == 0 || warp == 6) {
    // ---------------------------------------------------------------- loaders
    if (lane == 0) {
      const bool is_a = warp == 0;
      const uint32_t base = sbase + (is_a ? 0 : kSmemB);
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_par = 0;
      bool ok = true, waited = !p.restored_before;
      while (ok && walk.next(p.s, &t)) {
        if (is_a && t.is_dw && !waited) {
          griddep_wait();
          fence_proxy_async_global();  // the restored values, before TMA reads them
          waited = true;
        }
        const int kb_count = t.is_dw ? p.s.dw.kb : p.s.da.kb;
        // first row (A) or column (B) of this CTA's half of the operand
        const int x0 = (is_a ? t.mt : t.nt) * kTile + cta * 128;
        for (int kb = 0; kb < kb_count; ++kb) {
          if (!wait_bar(bar_empty + 8 * stage, phase ^ 1u, limit, cta_abort)) {
            give_up(abort_addr);
            ok = false;
            break;
          }
          const uint32_t fb = bar_full + 8 * stage, fb0 = mapa_shared(fb, 0);
          const uint32_t dst = base + stage * kOperand;
          if (cta == 0) mbar_arrive_expect_tx(fb, 2 * kOperand);
          if (!t.is_dw) {
            if (is_a)
              tma_load_3d_pair(dst, &p.dy_k, fb0, kb * kBK, x0, 0);
            else
              tma_load_3d_pair(dst, &p.w_k, fb0, kb * kBK, x0, t.rank);
          } else {
            const CUtensorMap* map = is_a ? &p.a_mn : &p.dy_mn;
            const int plane = is_a ? t.rank : 0;
            tma_load_3d_pair(dst, map, fb0, x0, kb * kBK, plane);
            tma_load_3d_pair(dst + kOperand / 2, map, fb0, x0 + 64, kb * kBK, plane);
          }
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the grid does not end before the restoration (a pair without dW tiles has not waited)
      if (is_a && !waited) griddep_wait();
      // every copy lands before the CTA can exit (the first CTA's barriers
      // count both CTAs' bytes; a pair that gave up waits in settle() below)
      if (cta == 0)
        for (int s = 0; s < kStages; ++s)
          if ((issued & (1u << s)) && !wait_bar(bar_full + 8 * s, (issued_par >> s) & 1u, kDrainNs, cta_abort))
            give_up(abort_addr);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    if (lane == 0 && cta == 0) {
      constexpr uint32_t idesc_k = idesc_bf16_f32(kTile, kTile, 0);
      constexpr uint32_t idesc_mn = idesc_bf16_f32(kTile, kTile, 1) | (1u << 15);  // A MN-major too
      // K-major: 128-byte rows, 8-row groups 1024 bytes apart, a 16-element step
      // is 32 bytes.  MN-major: 64-column boxes half an operand apart, 8-token
      // groups 1024 bytes apart, a 16-token step is 2 KiB.
      const uint64_t k0 = smem_desc_sw128(sbase, 16, 1024);
      const uint64_t mn0 = smem_desc_sw128(sbase, kOperand / 2, 1024);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      while (ok && walk.next(p.s, &t)) {
        if (!wait_bar(bar_acc_empty + 8 * acc, acc_phase ^ 1u, limit, cta_abort, true)) {
          give_up(abort_addr);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * kTile;
        const uint32_t idesc = t.is_dw ? idesc_mn : idesc_k;
        const uint64_t desc0 = t.is_dw ? mn0 : k0;
        const uint32_t hi = (uint32_t)(desc0 >> 32), step = t.is_dw ? 128u : 2u;
        const int kb_count = t.is_dw ? p.s.dw.kb : p.s.da.kb;
        for (int kb = 0; kb < kb_count; ++kb) {
          if (!wait_bar(bar_full + 8 * stage, phase, limit, cta_abort)) {
            give_up(abort_addr);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = (uint32_t)desc0 + (uint32_t)(stage * (kOperand >> 4));
          const uint32_t b = a + (uint32_t)(kSmemB >> 4);
#pragma unroll
          for (uint32_t s = 0; s < kBK / 16; ++s)
            mma_bf16<2>(d, desc_join(a + step * s, hi), desc_join(b + step * s, hi), idesc,
                        (kb | (int)s) != 0 ? 1u : 0u);
          mma_commit_pair_multicast(bar_empty + 8 * stage, 0x3);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit_pair_multicast(bar_acc_full + 8 * acc, 0x3);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      mma_commit<2>(bar_drain);  // every MMA completes before TMEM is released
      if (!wait_bar(bar_drain, 0, kDrainNs, cta_abort)) give_up(abort_addr);
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    // Lane = row of the warp's 32; 64 columns at a time through a shared buffer
    // in the 128-byte swizzle and one TMA store, which clips ragged edges.
    const int q = warp & 3;
    const uint32_t ebuf = sbase + kSmemEpi + (uint32_t)(warp - 2) * 2 * kEpiBufBytes;
    int acc = 0, nbuf = 0;
    uint32_t acc_phase = 0;
    while (walk.next(p.s, &t)) {
      int got = 0;
      if (lane == 0) got = wait_bar(bar_acc_full + 8 * acc, acc_phase, limit, cta_abort) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) {
        if (lane == 0) give_up(abort_addr);
        break;
      }
      tc_fence_after();
      const CUtensorMap* map = t.is_dw ? &p.out_dw : &p.out_da;
      const int rows = t.is_dw ? p.Kr : p.M, cols = t.is_dw ? p.N : p.Kr;
      const int row0 = t.mt * kTile + cta * 128 + q * 32;
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kTile);
      uint32_t v0[32], v1[32];
      tmem_ld_32x32b_x32(taddr, v0);
      tmem_ld_32x32b_x32(taddr + 32, v1);
#pragma unroll 1
      for (int c = 0; c < kTile / 64; ++c) {
        tmem_ld_wait(v0);
        tmem_ld_wait(v1);
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          w[i] = pack_bf16x2(__uint_as_float(v0[2 * i]), __uint_as_float(v0[2 * i + 1]));
          w[16 + i] = pack_bf16x2(__uint_as_float(v1[2 * i]), __uint_as_float(v1[2 * i + 1]));
        }
        if (c == kTile / 64 - 1) {  // accumulator read: back to the MMA warp
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (cta == 0)
              mbar_arrive(bar_acc_empty + 8 * acc);
            else
              mbar_arrive_remote(mapa_shared(bar_acc_empty + 8 * acc, 0));
          }
        } else {
          tmem_ld_32x32b_x32(taddr + (c + 1) * 64, v0);
          tmem_ld_32x32b_x32(taddr + (c + 1) * 64 + 32, v1);
        }
        const int col = t.nt * kTile + c * 64;
        if (row0 < rows && col < cols) {
          const uint32_t src = ebuf + (uint32_t)nbuf * kEpiBufBytes;
          if (lane == 0) bulk_wait_group_read<1>();  // the buffer's previous store has read it
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_shared_v4(src + lane * 128 + (uint32_t)((j ^ (lane & 7)) << 4), w[4 * j], w[4 * j + 1],
                         w[4 * j + 2], w[4 * j + 3]);
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(map, src, col, row0, t.rank);
            bulk_commit_group();
          }
          nbuf ^= 1;
        }
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA issues anything more, and what it issued has ended
  const uint32_t gave_up = *cta_abort;  // the same in both CTAs
  if (gave_up) settle();                // or has now
  if (threadIdx.x == 0) p.status[blockIdx.x] = gave_up;
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem_base, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// bf16 [planes][rows][cols], rows `pitch` elements apart (0: cols), 128-byte
// swizzle, zero fill out of bounds.
bool make_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t planes, uint32_t box_cols,
              uint32_t box_rows, int64_t pitch = 0) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t row_bytes = (cuuint64_t)(pitch ? pitch : cols) * 2;
  const cuuint64_t strides[2] = {row_bytes, row_bytes * (cuuint64_t)rows};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int tiles_of_dim(int64_t n) { return (int)((n + kTile - 1) / kTile); }

// rows x cols outputs per rank, contraction over `depth`
Product product_of(int64_t rows, int64_t cols, int64_t depth) {
  Product p;
  p.mt = tiles_of_dim(rows);
  p.nt = tiles_of_dim(cols);
  p.kb = (int)((depth + kBK - 1) / kBK);
  p.band = auto_band(rows, depth, kTile);
  return p;
}

// Estimated cycles of a tile: dA's steps, with the loads behind the tensor cores'
// 512 cycles; dW's, of which a short one is as long as its 128 KB of output take.
int da_tile_cycles(int kb) { return 600 * kb + 1000; }
int dw_tile_cycles(int kb) { return (512 * kb > 2500 ? 512 * kb : 2500) + 500; }

Schedule schedule_of(const Product& da, const Product& dw, int max_pairs) {
  Schedule s;
  s.da = da;
  s.dw = dw;
  const int tiles = da.tiles() + dw.tiles();
  s.pairs = tiles < max_pairs ? tiles : max_pairs;
  s.extra = da.tiles() % s.pairs;
  s.early = 0;
  if (s.extra > 0 && dw.tiles() > 0) {
    s.early = da_tile_cycles(da.kb) / dw_tile_cycles(dw.kb);
    const int spare = s.pairs - s.extra;
    // as many whole rounds of early tiles as there are tiles for
    if (s.early > dw.tiles() / spare) s.early = dw.tiles() / spare;
  }
  return s;
}

}  // namespace

struct gemm_rs_bwd_plan_s {
  int64_t M, N, K, Kr;
  uint64_t timeout_ns;
  int max_pairs;
  size_t total;
  const void* last_ws = nullptr;  // of the last run; null if it launched no kernel
  int last_ctas = 0;
};

extern "C" int gemm_rs_bwd_create(int64_t M, int64_t N, int64_t K, uint64_t timeout_ns, gemm_rs_bwd_t* plan,
                                  size_t* workspace_bytes) {
  if (!plan) return GEMM_RS_ERR_INVALID_ARG;
  *plan = nullptr;
  if (M < 0 || N < 0 || K < 0 || M % 8 || N % 8 || K % 64) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  // TMA coordinates and tile indices are 32-bit
  const int64_t Kr = K / kWorld;
  if (M > (1ll << 30) || N > (1ll << 30) || Kr > (1ll << 30)) return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  const int64_t most = (1ll << 30) / kWorld;
  if ((M / kTile + 1) * (Kr / kTile + 1) >= most || (Kr / kTile + 1) * (N / kTile + 1) >= most)
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  int sms = 0;
  int rc = current_device_sms(&sms);
  if (rc) return rc;
  if (cudaFuncSetAttribute(backward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc) !=
      cudaSuccess) {
    cudaGetLastError();
    return GEMM_RS_ERR_CUDA;
  }
  // pairs that run at the same time (an SM without a free neighbour is left out)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(sms / 2));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = kSmemAlloc;
  int pairs = 0;
  if (cudaOccupancyMaxActiveClusters(&pairs, backward_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_RS_ERR_CUDA;
  }
  if (pairs < 1) return GEMM_RS_ERR_UNSUPPORTED_DEVICE;
  gemm_rs_bwd_plan_s* h = new (std::nothrow) gemm_rs_bwd_plan_s();
  if (!h) return GEMM_RS_ERR_CUDA;
  h->M = M;
  h->N = N;
  h->K = K;
  h->Kr = Kr;
  h->timeout_ns = timeout_ns ? timeout_ns : kDefaultTimeoutNs;
  h->max_pairs = pairs < sms / 2 ? pairs : sms / 2;
  if (h->max_pairs > kStatusWords / 2) h->max_pairs = kStatusWords / 2;
  h->total = kStatusBytes + (size_t)kWorld * M * act8_pitch(Kr) * 2;  // whole 256-byte lines: TMA reads boxes of 128
  if (workspace_bytes) *workspace_bytes = h->total;
  *plan = h;
  return GEMM_RS_OK;
}

extern "C" int gemm_rs_bwd_run(gemm_rs_bwd_t h, const void* dY, const void* W, const void* codes,
                               const void* scales, void* dA, void* dW, void* workspace, void* stream) {
  if (!h) return GEMM_RS_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool da = dA && h->M > 0 && h->Kr > 0, dw = dW && h->N > 0 && h->Kr > 0;
  if (!da && !dw) {
    h->last_ws = nullptr;
    return GEMM_RS_OK;
  }
  if (h->M > 0 && h->N > 0 && (!dY || (da && !W) || (dw && (!codes || !scales)))) return GEMM_RS_ERR_INVALID_ARG;
  for (const void* q : {dY, W, codes, scales, (const void*)dA, (const void*)dW, (const void*)workspace})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  if (!workspace) return GEMM_RS_ERR_WORKSPACE;
  if (h->M == 0 || h->N == 0) {  // an empty contraction
    void* out = h->M == 0 ? dW : dA;
    const size_t bytes = (size_t)kWorld * h->Kr * (h->M == 0 ? h->N : h->M) * 2;
    if (cudaMemsetAsync(out, 0, bytes, st) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_RS_ERR_CUDA;
    }
    h->last_ws = nullptr;
    return GEMM_RS_OK;
  }
  BwdParams p;
  memset(&p, 0, sizeof(p));
  p.status = static_cast<uint32_t*>(workspace);
  void* const restored = static_cast<uint8_t*>(workspace) + kStatusBytes;
  p.M = (int)h->M;
  p.N = (int)h->N;
  p.Kr = (int)h->Kr;
  p.timeout_ns = h->timeout_ns;
  const Product none = {0, 0, 0, 1};
  bool ok = true;
  if (da)
    ok = ok && make_map(&p.dy_k, dY, h->N, h->M, 1, kBK, 128) && make_map(&p.w_k, W, h->N, h->Kr, kWorld, kBK, 128) &&
         make_map(&p.out_da, dA, h->Kr, h->M, kWorld, 64, 32);
  if (dw) {
    ok = ok && make_map(&p.a_mn, restored, h->Kr, h->M, kWorld, 64, kBK, act8_pitch(h->Kr)) &&
         make_map(&p.dy_mn, dY, h->N, h->M, 1, 64, kBK) && make_map(&p.out_dw, dW, h->N, h->Kr, kWorld, 64, 32);
    // A small checkpoint is restored beside the first dA tiles; a large one is
    // faster with the whole GPU to itself.
    p.restored_before = da && h->M * h->K <= kRestoreBeside;
    const int rc = act8_restore_padded(h->M, h->K, codes, scales, restored, p.restored_before, stream);
    if (rc) return rc;
  }
  if (!ok) return GEMM_RS_ERR_CUDA;
  p.s = schedule_of(da ? product_of(h->M, h->Kr, h->N) : none, dw ? product_of(h->Kr, h->N, h->M) : none,
                    h->max_pairs);
  const int ctas = 2 * p.s.pairs;
  const int rc = launch_overlapped(backward_kernel, dim3((unsigned)ctas), 32 * kWarps, kSmemAlloc, st, p);
  if (rc) return rc;
  h->last_ws = workspace;
  h->last_ctas = ctas;
  return GEMM_RS_OK;
}

extern "C" int gemm_rs_bwd_status(gemm_rs_bwd_t h, void* stream) {
  if (!h) return GEMM_RS_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t words[kStatusWords];
  cudaError_t e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && h->last_ws) {
    e = cudaMemcpyAsync(words, h->last_ws, h->last_ctas * sizeof(uint32_t), cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_RS_ERR_CUDA;
  }
  for (int i = 0; h->last_ws && i < h->last_ctas; ++i)
    if (words[i]) return GEMM_RS_ERR_TIMEOUT;
  return GEMM_RS_OK;
}

extern "C" int gemm_rs_bwd_destroy(gemm_rs_bwd_t h) {
  if (!h) return GEMM_RS_ERR_INVALID_ARG;
  delete h;
  return GEMM_RS_OK;
}
