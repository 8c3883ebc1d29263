// fp8_gemm_f32.cu -- products of e4m3 operands with an fp32 scale for each block of 128
// (gemm_rs_fp8_* and gemm_rs_moe_* in include/gemm_rs_ops.h).
//
// A product is a sum over steps of 128 inner elements.  In a step the elements of a row of A
// share a scale, and so do those of a column of B (of a weight: of 128 columns), so the step's
// product of codes is scaled as a whole:
//   out[m][n] = sum_s a_scale[s][m] b_scale[s][n] (sum over the step of products of codes)
// The tensor cores apply powers of two only, so a step's product (kind::f8f6f4) lands in one of
// two accumulators in TMEM, and while the next step is multiplied eight warps of each CTA read it,
// scale it and add it to sums in fp32, rounded to nearest, that stay in their registers: 128
// of a thread's 216, which the other four warps give up with setmaxnreg.
// Scales go through two slots in shared memory, of four steps each: for weights a row's scale
// times its columns', for dW rows' and columns' apart.
// Warps in each CTA: 0 loads A, 2 loads B, 3 brings scales, 1 issues the MMAs (first
// CTA of the pair), 4 to 11 scale, sum and store.
// Bound by the additions, and by a step's way from MMA to sums and back, which two accumulators do not hide
// whole: an accumulator is handed back as soon as its last columns are in registers, before they are added
// (in that order 2048 x 8192 x 8192 forward took 158 us in place of 190, with every part added before the
// next is read 198).
#include <type_traits>

#include "fp8_tiles.cuh"

using namespace grs;
using namespace grs::tiles;

namespace {

constexpr int kSlots = 2, kPerSlot = 4;   // of scales, and steps in a slot, counted from a tile's first
constexpr int kStepBytes = 384 * 4;       // 128 rows' for each half of the columns; dW: 128 rows' and 256 columns'
constexpr int kSlotBytes = kPerSlot * kStepBytes;
constexpr int kSmemBuf = kSmemScales + kSlots * kSlotBytes;
constexpr int kSmemBar = kSmemBuf + kEpiWarps * kBufBytes;
constexpr int kNumBars = 2 * kStages + 2 * kSlots + 5;  // full, empty, sf_full, sf_empty, acc_full[2], acc_empty[2], drain
constexpr int kSmemMisc = kSmemBar + kNumBars * 8;
constexpr int kSmemStart = kSmemMisc + 16;
constexpr int kSmemAlloc = kSmemStart + 2 * (kMaxExperts + 1) * 4 + 1024;  // slack to align the base to 1024 bytes
static_assert(kSmemAlloc <= 232448, "shared memory per CTA");
// Registers of a thread at launch, and after the exchange.
constexpr int kRegsLaunch = 168, kRegsOther = 72, kRegsSum = 216;
constexpr int kRegsHeld = 128 * kRegsOther + 32 * kEpiWarps * kRegsSum;
static_assert(kRegsHeld <= kThreads * kRegsLaunch, "setmaxnreg would wait for ever");

__device__ __forceinline__ void mma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// sums[0..15] += scaled v[0..31]: by one factor, or by the row's and the columns' own.  Packed additions run on
// one of the two pipes that single ones share, so every third pair is added by single ones: 2048 x 8192 x 8192
// forward 156 us with packed ones alone, 142 with a quarter single, 140 with a third, 165 with half.
__device__ __forceinline__ void add_scaled(uint64_t* sums, const uint32_t (&v)[32], uint64_t factor) {
  const float f = __uint_as_float((uint32_t)factor);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (i % 3 != 2) {
      sums[i] = fma2(pack2(v[2 * i], v[2 * i + 1]), factor, sums[i]);
    } else {
      const float x = fmaf(__uint_as_float(v[2 * i]), f, __uint_as_float((uint32_t)sums[i]));
      const float y = fmaf(__uint_as_float(v[2 * i + 1]), f, __uint_as_float((uint32_t)(sums[i] >> 32)));
      sums[i] = pack2(__float_as_uint(x), __float_as_uint(y));
    }
  }
}
__device__ __forceinline__ void add_scaled_columns(uint64_t* sums, const uint32_t (&v)[32], uint64_t factor, uint32_t columns) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint64_t c, d;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(c), "=l"(d) : "r"(columns + 16 * i));
    sums[2 * i] = fma2(pack2(v[4 * i], v[4 * i + 1]), mul2(c, factor), sums[2 * i]);
    sums[2 * i + 1] = fma2(pack2(v[4 * i + 2], v[4 * i + 3]), mul2(d, factor), sums[2 * i + 1]);
  }
}

// A step's scales of the tile, by the whole scale warp: rows lane + 32 j of this CTA's 128, columns
// 128 h + lane + 32 j of the pair's 256 (for weights one for each half).
struct Scales {
  float a[4], b[2][4];
  bool columns;
};

// step: counted from the tensor's first (weight grad: the token block).
template <int kKind>
__device__ __forceinline__ void load_scales(const Params<kKind>& p, const Tile& t, int cta, int lane, int step, Scales* s) {
  const int kind = kind_of<kKind>(t);
  const Side& d = side_of(p, t);
  const int rows_max = kind == kFp8WeightGrad ? p.Kr : p.M;
  const float* a = static_cast<const float*>(d.a_scale) + step * d.a_stride;
  if (kind == kFp8WeightGrad) a += (long long)t.plane * (d.a_stride / kWorld);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = t.row0 + cta * 128 + lane + 32 * j;
    s->a[j] = load_f32(a + (row < rows_max ? row : rows_max - 1));
  }
  s->columns = kind == kFp8WeightGrad;
  const float* b = static_cast<const float*>(d.b_scale);
  if (kind == kFp8WeightGrad) {
    b += step * d.b_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = t.col0 + h * 128 + lane + 32 * j;
        s->b[h][j] = load_f32(b + (col < p.N ? col : p.N - 1));
      }
  } else {
    // a tile's second half may lie behind the last block: its columns are not stored
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (kind == kFp8Forward) {
        const int nb = t.col0 / kBlk + h;
        s->b[h][0] = load_f32(b + ((long long)t.e * (kWorld * p.KB) + step) * p.NB + (nb < p.NB ? nb : p.NB - 1));
      } else {
        const int kb = t.col0 / kBlk + h;
        s->b[h][0] = load_f32(b + ((long long)(t.e * kWorld + t.plane) * p.KB + (kb < p.KB ? kb : p.KB - 1)) * p.NB + step);
      }
    }
  }
}

template <int kKind>
__device__ __forceinline__ void store_scales(uint32_t dst, int lane, const Scales& s) {
  auto store = [&](int at, float v) { st_shared_u32(dst + 4 * (at + lane), __float_as_uint(v)); };
  if (kKind == kBothGrads ? s.columns : kKind == kFp8WeightGrad) {
#pragma unroll
    for (int j = 0; j < 4; ++j) store(32 * j, s.a[j]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) store(128 + 128 * h + 32 * j, s.b[h][j]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) store(128 * h + 32 * j, s.a[j] * s.b[h][0]);
  }
}

template <int kKind>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_product_f32_kernel(const __grid_constant__ Params<kKind> p) {
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
  const uint32_t bar_acc_empty = bar_acc_full + 16;
  const uint32_t bar_drain = bar_acc_empty + 16;
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
      mbar_init(bar_sf_full + 8 * s, 1);           // this CTA's scale warp
      mbar_init(bar_sf_empty + 8 * s, kEpiWarps);  // its summing warps
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

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 0 || warp == 2) {
      // ------------------------------------------------------------ loaders
      if (lane == 0) load_operand<kKind>(p, walk, warp == 0, cta, sbase, bar_full, cta_abort, abort_addr);
    } else if (warp == 1) {
      // --------------------------------------------------------- MMA issuer
      if (cta == 0) {
        const bool leader = elect_one();
        // K-major: rows of 128 bytes, groups of 8 of them 1024 bytes apart, 32 inner
        // elements further are 32 bytes.  MN-major: an inner element's 128 rows (or
        // columns) are 128 bytes, groups of 8 inner elements 1024 bytes apart, 32
        // further are 4 KiB.
        const uint64_t desc0 = smem_desc_sw128(sbase, 16, 1024);
        const uint32_t hi = (uint32_t)(desc0 >> 32);
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        while (ok && walk.next(&t)) {
          const bool a_mn = kind_of<kKind>(t) == kFp8WeightGrad, b_mn = kind_of<kKind>(t) != kFp8InputGrad;
          const uint32_t idesc = idesc_e4m3(kTile, kTile, a_mn, b_mn);
          const uint32_t a_step = a_mn ? 256 : 2, b_step = b_mn ? 256 : 2;
          for (int s = 0; s < t.steps; ++s) {
            if (!wait_bar(bar_full + 8 * stage, phase, kLimitNs, cta_abort) ||
                !wait_bar(bar_acc_empty + 8 * acc, acc_phase ^ 1u, kLimitNs, cta_abort, true)) {
              give_up(abort_addr);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a = (uint32_t)desc0 + (uint32_t)(stage * (kOperand >> 4));
            const uint32_t b = a + (uint32_t)(kSmemB >> 4);
            if (leader) {
#pragma unroll
              for (uint32_t i = 0; i < kBlk / 32; ++i)
                mma_e4m3_pair(tmem_base + acc * kTile, desc_join(a + a_step * i, hi), desc_join(b + b_step * i, hi), idesc,
                              i != 0 ? 1u : 0u);
              mma_commit_pair_multicast(bar_acc_full + 8 * acc, 0x3);
              mma_commit_pair_multicast(bar_empty + 8 * stage, 0x3);
            }
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
          }
        }
        if (leader) mma_commit<2>(bar_drain);  // every MMA completes before TMEM is released
        if (!wait_bar(bar_drain, 0, kDrainNs, cta_abort)) give_up(abort_addr);
      }
    } else {
      // ------------------------------------------------------------- scales
      // A slot's steps are loaded kBatch at a time; dW's have three times as many words.
      constexpr int kBatch = kKind == kFp8WeightGrad || kKind == kBothGrads ? 2 : kPerSlot;
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && walk.next(&t)) {
        for (int s0 = 0; ok && s0 < t.steps; s0 += kPerSlot) {
          Scales sf[kBatch];
#pragma unroll
          for (int j0 = 0; j0 < kPerSlot; j0 += kBatch) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
              if (s0 + j0 + j < t.steps) load_scales<kKind>(p, t, cta, lane, t.step0 + s0 + j0 + j, &sf[j]);
            if (j0 == 0) {
              int got = 0;
              if (lane == 0) got = wait_bar(bar_sf_empty + 8 * slot, phase ^ 1u, kLimitNs, cta_abort) ? 1 : 0;
              got = __shfl_sync(0xffffffffu, got, 0);
              if (!got) {
                if (lane == 0) give_up(abort_addr);
                ok = false;
                break;
              }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
              if (s0 + j0 + j < t.steps)
                store_scales<kKind>(sbase + kSmemScales + slot * kSlotBytes + (j0 + j) * kStepBytes, lane, sf[j]);
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_sf_full + 8 * slot);
          if (++slot == kSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSum));
    // ------------------------------------------------- scale, sum and store
    // Lane = row of the warp's 32, 128 of the tile's columns.
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t buf = sbase + kSmemBuf + (uint32_t)(warp - 4) * kBufBytes;
    const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * 128);
    uint32_t n = 0, m = 0;  // steps and slots so far: sums n & 1 in TMEM, slot m & 1
    bool ok = true;
    for (int at = pair;; at += pairs) {
      // what the steps do not need of the tile is looked up again behind them: registers
      if (!Walk<kKind>(p, start, blocks, at, pairs).next(&t)) break;
      uint64_t sums[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sums[i] = 0;
      auto add_steps = [&](auto columns, const int steps) {  // whether columns have scales of their own
        constexpr bool kColumns = decltype(columns)::value;
        uint32_t v[2][32];
        uint64_t factor = 0;
        uint32_t scales = 0;
        // Waits for step s's products and scales.
        auto begin = [&](int s) {
          const bool got = (s % kPerSlot != 0 || wait_bar(bar_sf_full + 8 * (m & 1), (m >> 1) & 1, kLimitNs, cta_abort)) &&
                           wait_bar(bar_acc_full + 8 * (n & 1), (n >> 1) & 1, kLimitNs, cta_abort);
          if (!__all_sync(0xffffffffu, got)) {
            if (lane == 0) give_up(abort_addr);
            return false;
          }
          tc_fence_after();
          scales = sbase + kSmemScales + (m & 1) * kSlotBytes + (uint32_t)(s % kPerSlot) * kStepBytes;
          const uint32_t own = ld_shared_u32(scales + 4 * ((kColumns ? 0 : half * 128) + q * 32 + lane));
          factor = pack2(own, own);
          return true;
        };
        auto ask = [&](int c) { tmem_ld_32x32b_x32(tbase + (n & 1) * kTile + 32 * c, v[c & 1]); };
        auto add = [&](int c) {
          if constexpr (kColumns)
            add_scaled_columns(sums + 16 * c, v[c & 1], factor, scales + 4 * (128 + half * 128 + 32 * c));
          else
            add_scaled(sums + 16 * c, v[c & 1], factor);
        };
        for (int s = 0; s < steps; ++s) {
          ok = begin(s);
          if (!ok) return;
          // two parts of 32 columns are on their way or being added at a time
          ask(0);
          ask(1);
          tmem_ld_wait(v[0]);
          tmem_ld_wait(v[1]);
          add(0);
          ask(2);
          add(1);
          ask(3);
          tmem_ld_wait(v[0]);
          tmem_ld_wait(v[1]);
          tc_fence_before();  // all read: back to the MMA warp
          __syncwarp();
          if (lane == 0) {
            if (cta == 0)
              mbar_arrive(bar_acc_empty + 8 * (n & 1));
            else
              mbar_arrive_remote(mapa_shared(bar_acc_empty + 8 * (n & 1), 0));
          }
          ++n;
          add(2);
          add(3);
          if (s % kPerSlot == kPerSlot - 1 || s == steps - 1) {  // the slot's scales have been read
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_sf_empty + 8 * (m & 1));
            ++m;
          }
        }
      };
      if (t.steps > 0) {
        if (kind_of<kKind>(t) == kFp8WeightGrad)
          add_steps(std::true_type{}, t.steps);
        else
          add_steps(std::false_type{}, t.steps);
      }
      if (!ok) break;
      Walk<kKind>(p, start, blocks, at, pairs).next(&t);
      uint32_t v[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i) v[c][i] = (uint32_t)(sums[16 * c + (i >> 1)] >> (32 * (i & 1)));
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
  return tiles ? launch<kKind, fp8_product_f32_kernel<kKind>, kSmemAlloc, kRegsHeld>(p, tiles * d.parts, st)
               : GEMM_RS_ERR_CUDA;
}

}  // namespace

int grs::fp8_product_f32(const Fp8Product& d, cudaStream_t st) {
  return d.kind == kFp8Forward     ? one<kFp8Forward>(d, st)
         : d.kind == kFp8InputGrad ? one<kFp8InputGrad>(d, st)
                                   : one<kFp8WeightGrad>(d, st);
}

// One launch where the tiles of both run at once: 392 x 776 x 1600 14.5 us against 21.8 by two, 512 x 1024 x 2048
// 14.8 against 21.4.  With more of them the launch of both, whose steps serve either kind, is the slower: 512 x 2048
// x 4096 34.3 against 32.9, 2048 x 4096 x 4096 130 against 115, 8192 x 4096 x 4096 446 against 385.
int grs::fp8_products_f32(const Fp8Product& input, const Fp8Product& weight, cudaStream_t st) {
  int sms = 0;
  const int rc = current_device_sms(&sms);
  if (rc) return rc;
  Params<kBothGrads> p;
  memset(&p, 0, sizeof(p));
  fill(&p, input);
  const int64_t a = fill(&p.sides[0], input), w = fill(&p.sides[1], weight);
  if (!a || !w) return GEMM_RS_ERR_CUDA;
  if (a + w <= sms / 2)
    return launch<kBothGrads, fp8_product_f32_kernel<kBothGrads>, kSmemAlloc, kRegsHeld>(p, a + w, st);
  const int first = fp8_product_f32(input, st);
  return first ? first : fp8_product_f32(weight, st);
}
