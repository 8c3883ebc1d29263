// fp8_gemm.cu -- products of e4m3 operands with a power of two for each block of 128
// (gemm_rs_fp8_*_e8m0 and gemm_rs_moe_*_e8m0 in include/gemm_rs_ops.h).
//
// A step multiplies 128 inner elements.  The elements of a row of A share a power of
// two in it, and so do those of a column of B, so the tensor cores apply both scales
// themselves (tcgen05 kind::mxf8f6f4, whose scales are of 32 elements each: a block's
// byte serves four of them) and sums stay in TMEM for the whole contraction.
//
// Scales go from registers to shared memory in the layout that tcgen05.cp expects, four steps at a
// time, and by tcgen05.cp to TMEM.  One accumulator of 256 columns: two would leave no
// TMEM for scales.  The epilogue therefore first reads all of it into registers (128 of a
// thread), hands it back, and rounds and stores while the next tile is multiplied.
// Warps in each CTA: 0 loads A, 2 loads B, 3 brings scales, 1 issues the MMAs (first
// CTA of the pair), 4 to 11 round and store.
// Bound by the tensor cores and, repeated, by the power limit: 8192 x 8192 x 28672 forward 1.21 to 1.41 ms
// with its quantisation, 2.7 to 3.2 PFLOP/s; 2048 x 8192 x 8192 89 us, 256 tiles in four waves of 76.
// dA and dW are independent, so a backward pass multiplies both in one launch, dA's tiles
// first: 392 x 776 x 1600 19.4 -> 12.0 us, 2048 x 8192 x 8192 187 -> 181.
#include "fp8_tiles.cuh"

using namespace grs;
using namespace grs::tiles;

namespace {

constexpr int kSlots = 4;            // of scales, kPerSlot steps each, in shared memory and in TMEM
constexpr int kPerSlot = 4;          // bytes of a word of scales
constexpr int kSfBytes = 512;        // scales of 128 rows or columns for the steps of a slot
constexpr int kSlotBytes = 3 * kSfBytes;  // this CTA's 128 rows of A, the pair's 256 columns of B
constexpr int kScaleBatch = 4;
constexpr int kTmemScales = 256, kSlotColumns = 16;
constexpr int kSmemBuf = kSmemScales + kSlots * kSlotBytes;
constexpr int kSmemBar = kSmemBuf + kEpiWarps * kBufBytes;
constexpr int kNumBars = 2 * kStages + 2 * kSlots + 3;  // full, empty, sf_full, sf_empty, acc_full, acc_empty, drain
constexpr int kSmemMisc = kSmemBar + kNumBars * 8;
constexpr int kSmemStart = kSmemMisc + 16;
constexpr int kSmemAlloc = kSmemStart + 2 * (kMaxExperts + 1) * 4 + 1024;  // slack to align the base to 1024 bytes
static_assert(kSmemAlloc <= 232448, "shared memory per CTA");

// A slot's scales of the tile: this CTA's rows and the pair's columns.
struct Scales {
  uint32_t a[4], b[2][4];
  int kind;
};

// Steps 4 slot .. 4 slot + 3, counted from the tensor's first (weight grad: token blocks;
// a tile's first step may be in the middle of a slot).
template <int kKind>
__device__ __forceinline__ void load_scales(const Params<kKind>& p, const Tile& t, int cta, int lane, int slot, Scales* s) {
  const int kind = s->kind = kind_of<kKind>(t);
  const Side& d = side_of(p, t);
  const int rows_max = kind == kFp8WeightGrad ? p.Kr : p.M;
  const uint32_t* a = static_cast<const uint32_t*>(d.a_scale) + slot * d.a_stride;
  if (kind == kFp8WeightGrad) a += (long long)t.plane * (d.a_stride / kWorld);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = t.row0 + cta * 128 + lane + 32 * j;
    s->a[j] = load_u32(a + (row < rows_max ? row : rows_max - 1));
  }
  if (kind == kFp8WeightGrad) {
    const uint32_t* b = static_cast<const uint32_t*>(d.b_scale) + slot * d.b_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = t.col0 + h * 128 + lane + 32 * j;
        s->b[h][j] = load_u32(b + (col < p.N ? col : p.N - 1));
      }
  } else {
    // lanes 0 to 3 the bytes of the first 128 columns, 4 to 7 of the others
    const int h = (lane >> 2) & 1, step = 4 * slot + (lane & 3);
    const uint8_t* b = static_cast<const uint8_t*>(d.b_scale);
    uint32_t byte;
    if (kind == kFp8Forward) {
      const int steps = kWorld * p.KB, nb = t.col0 / kBlk + h;
      byte = load_u8(b + ((long long)t.e * steps + (step < steps ? step : steps - 1)) * p.NB +
                     (nb < p.NB ? nb : p.NB - 1));
    } else {
      const int kb = t.col0 / kBlk + h;
      byte = load_u8(b + ((long long)(t.e * kWorld + t.plane) * p.KB + (kb < p.KB ? kb : p.KB - 1)) * p.NB +
                     (step < p.NB ? step : p.NB - 1));
    }
    s->b[0][0] = byte;
  }
}

template <int kKind>
__device__ __forceinline__ void store_scales(uint32_t dst, int lane, Scales& s) {
  if ((kKind == kBothGrads ? s.kind : kKind) != kFp8WeightGrad) {
    const uint32_t byte = s.b[0][0];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t word = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, byte, 4 * h + i) << (8 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) s.b[h][j] = word;
    }
  }
  st_shared_v4(dst + lane * 16, s.a[0], s.a[1], s.a[2], s.a[3]);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    st_shared_v4(dst + (1 + h) * kSfBytes + lane * 16, s.b[h][0], s.b[h][1], s.b[h][2], s.b[h][3]);
}

template <int kKind>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_product_kernel(const __grid_constant__ Params<kKind> p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cta = (int)cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_full = sbase + kSmemBar;
  const uint32_t bar_empty = bar_full + 8 * kStages;
  const uint32_t bar_sf_full = bar_empty + 8 * kStages;
  const uint32_t bar_sf_empty = bar_sf_full + 8 * kSlots;
  const uint32_t bar_acc_full = bar_sf_empty + 8 * kSlots;
  const uint32_t bar_acc_empty = bar_acc_full + 8;
  const uint32_t bar_drain = bar_acc_empty + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmemMisc);
  volatile uint32_t* cta_abort = reinterpret_cast<volatile uint32_t*>(smem + kSmemMisc + 4);
  const uint32_t abort_addr = sbase + kSmemMisc + 4;
  int* start = reinterpret_cast<int*>(smem + kSmemStart);
  int* blocks = start + kMaxExperts + 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_full + 8 * s, 2);   // the first CTA's two loaders (+ both CTAs' bytes)
      mbar_init(bar_empty + 8 * s, 1);  // one MMA commit
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar_sf_full + 8 * s, 2);   // both CTAs' scale warps
      mbar_init(bar_sf_empty + 8 * s, 1);  // one MMA commit
    }
    mbar_init(bar_acc_full, 1);
    mbar_init(bar_acc_empty, 2 * kEpiWarps);
    mbar_init(bar_drain, 1);
    *cta_abort = 0;
    fence_mbar_init();
    fence_proxy_async_shared();
  }
  if (warp == 1) {
    tmem_alloc<2>(smem_u32(tmem_slot), 512);
    tmem_relinquish<2>();
  }
  griddep_wait();
  if (kKind != kFp8WeightGrad && warp == 3) count_starts(p, lane, start, kTile, p.sides[0].nt, 0x7FFFFFFF);
  // offsets that do not ascend may count more blocks than the tensors have
  if (kKind >= kFp8WeightGrad && warp == 2) count_starts(p, lane, blocks, kBlk, 1, p.blocks);
  tc_fence_before();
  __syncthreads();
  cluster_sync_shared();  // barriers and TMEM of both
  tc_fence_after();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const uint32_t tmem_base = *tmem_slot;
  Walk<kKind> walk(p, start, blocks, pair, pairs);
  Tile t;

  if (warp == 0 || warp == 2) {
    // -------------------------------------------------------------- loaders
    if (lane == 0) load_operand<kKind>(p, walk, warp == 0, cta, sbase, bar_full, cta_abort, abort_addr);
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer
    if (cta == 0) {
      const bool leader = elect_one();
      // K-major: rows of 128 bytes, groups of 8 of them 1024 bytes apart, 32 inner
      // elements further are 32 bytes.  MN-major: an inner element's 128 rows (or
      // columns) are 128 bytes, groups of 8 inner elements 1024 bytes apart, 32
      // further are 4 KiB.
      const uint64_t desc0 = smem_desc_sw128(sbase, 16, 1024);
      const uint32_t hi = (uint32_t)(desc0 >> 32);
      const uint64_t sf_desc = scales_desc(sbase + kSmemScales);
      int stage = 0, slot = 0, buf = 0;  // buf: slot whose scales are in use
      uint32_t phase = 0, sf_phase = 0, acc_phase = 0;
      bool ok = true;
      while (ok && walk.next(&t)) {
        const bool a_mn = kind_of<kKind>(t) == kFp8WeightGrad, b_mn = kind_of<kKind>(t) != kFp8InputGrad;
        const uint32_t idesc = idesc_mx(kTile, kTile, a_mn, b_mn);
        const uint32_t a_step = a_mn ? 256 : 2, b_step = b_mn ? 256 : 2;
        for (int s = 0; s < t.steps; ++s) {
          const uint32_t id = (uint32_t)(t.step0 + s) & (kPerSlot - 1);
          const bool fetch = s == 0 || id == 0;
          if (!wait_bar(bar_full + 8 * stage, phase, kLimitNs, cta_abort) ||
              (fetch && !wait_bar(bar_sf_full + 8 * slot, sf_phase, kLimitNs, cta_abort, true))) {
            give_up(abort_addr);
            ok = false;
            break;
          }
          tc_fence_after();
          if (fetch) buf = slot;
          if (fetch && leader) {
#pragma unroll
            for (int i = 0; i < 3; ++i)
              copy_scales<2>(tmem_base + kTmemScales + buf * kSlotColumns + 4 * i,
                               sf_desc + (uint32_t)((buf * kSlotBytes + i * kSfBytes) >> 4));
          }
          if (fetch && ++slot == kSlots) {
            slot = 0;
            sf_phase ^= 1u;
          }
          if (s == 0) {  // the operands and scales are there: only now wait for the accumulator
            if (!wait_bar(bar_acc_empty, acc_phase ^ 1u, kLimitNs, cta_abort, true)) {
              give_up(abort_addr);
              ok = false;
              break;
            }
            acc_phase ^= 1u;
            tc_fence_after();
          }
          const uint32_t a = (uint32_t)desc0 + (uint32_t)(stage * (kOperand >> 4));
          const uint32_t b = a + (uint32_t)(kSmemB >> 4);
          const uint32_t sf = tmem_base + kTmemScales + buf * kSlotColumns;
          if (leader) {
#pragma unroll
            for (uint32_t i = 0; i < kBlk / 32; ++i)
              mma_scaled<2>(tmem_base, desc_join(a + a_step * i, hi), desc_join(b + b_step * i, hi),
                              idesc_step(idesc, id), sf, sf + 4, (s | (int)i) != 0 ? 1u : 0u);
            mma_commit_pair_multicast(bar_empty + 8 * stage, 0x3);
            // the slot's last step: its words in shared memory and in TMEM are free once it is done
            if (id == kPerSlot - 1 || s == t.steps - 1) mma_commit_pair_multicast(bar_sf_empty + 8 * buf, 0x3);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (leader && t.steps > 0) mma_commit_pair_multicast(bar_acc_full, 0x3);
      }
      if (leader) mma_commit<2>(bar_drain);  // every MMA completes before TMEM is released
      if (!wait_bar(bar_drain, 0, kDrainNs, cta_abort)) give_up(abort_addr);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------------ scales
    // kScaleBatch slots' words are loaded, then written one by one: the fence behind each
    // write waits for every load on its way, so none is while slots are written.
    int slot = 0, c = 0, last = -1;
    uint32_t phase = 0;
    auto fetch = [&](Scales* sf) {  // the next slot's of this tile or the next one
      while (c > last) {
        if (!walk.next(&t)) return false;
        c = t.step0 / kPerSlot;
        last = t.steps > 0 ? (t.step0 + t.steps - 1) / kPerSlot : c - 1;
      }
      load_scales<kKind>(p, t, cta, lane, c++, sf);
      return true;
    };
    Scales sf[kScaleBatch];
    bool ok = true, more = true;
    while (ok && more) {
      int n = 0;
#pragma unroll
      for (int j = 0; j < kScaleBatch; ++j)
        if (more) {
          more = fetch(&sf[j]);
          n += more;
        }
#pragma unroll
      for (int j = 0; j < kScaleBatch; ++j) {
        if (!ok || j >= n) continue;
        int got = 0;
        if (lane == 0) got = wait_bar(bar_sf_empty + 8 * slot, phase ^ 1u, kLimitNs, cta_abort) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          if (lane == 0) give_up(abort_addr);
          ok = false;
          continue;
        }
        store_scales<kKind>(sbase + kSmemScales + slot * kSlotBytes, lane, sf[j]);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          if (cta == 0)
            mbar_arrive(bar_sf_full + 8 * slot);
          else  // releasing all memory takes 1700 cycles, more with the next scales on their way (dA of
                // 2048 x 8192 x 8192 113 us against 93)
            mbar_arrive_remote_release_shared(mapa_shared(bar_sf_full + 8 * slot, 0));
        }
        if (++slot == kSlots) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    // ----------------------------------------------------------- round and store
    // Lane = row of the warp's 32, 128 of the tile's columns.
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * 128);
    const uint32_t buf = sbase + kSmemBuf + (uint32_t)(warp - 4) * kBufBytes;
    uint32_t acc_phase = 0;
    while (walk.next(&t)) {
      uint32_t v[4][32];
      if (t.steps > 0) {
        int got = 0;
        if (lane == 0) got = wait_bar(bar_acc_full, acc_phase, kLimitNs, cta_abort) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          if (lane == 0) give_up(abort_addr);
          break;
        }
        acc_phase ^= 1u;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(taddr + 32 * c, v[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(v[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (cta == 0)
            mbar_arrive(bar_acc_empty);
          else
            mbar_arrive_remote(mapa_shared(bar_acc_empty, 0));
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) v[c][i] = 0;
      }
      store_tile(p, t, cta, q, half, lane, buf, v);
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA issues anything more, and what it issued has ended
  const uint32_t gave_up = *cta_abort;  // the same in both CTAs
  if (gave_up) settle();                // or has now
  if (threadIdx.x == 0 && gave_up) *p.status = 1;
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem_base, 512);
  }
}

template <int kKind>
int one(const Fp8Product& d, cudaStream_t st) {
  Params<kKind> p;
  memset(&p, 0, sizeof(p));
  fill(&p, d);
  const int64_t tiles = fill(&p.sides[0], d);
  return tiles ? launch<kKind, fp8_product_kernel<kKind>, kSmemAlloc, 0>(p, tiles * d.parts, st) : GEMM_RS_ERR_CUDA;
}

}  // namespace

int grs::fp8_product_e8m0(const Fp8Product& d, cudaStream_t st) {
  return d.kind == kFp8Forward     ? one<kFp8Forward>(d, st)
         : d.kind == kFp8InputGrad ? one<kFp8InputGrad>(d, st)
                                   : one<kFp8WeightGrad>(d, st);
}

int grs::fp8_products_e8m0(const Fp8Product& input, const Fp8Product& weight, cudaStream_t st) {
  Params<kBothGrads> p;
  memset(&p, 0, sizeof(p));
  fill(&p, input);
  const int64_t a = fill(&p.sides[0], input), w = fill(&p.sides[1], weight);
  return a && w ? launch<kBothGrads, fp8_product_kernel<kBothGrads>, kSmemAlloc, 0>(p, a + w, st) : GEMM_RS_ERR_CUDA;
}
