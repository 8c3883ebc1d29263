// fp8_few.cu -- the products of fp8.cuh with a weight for few rows: single tokens and
// small batches, of one weight or of the experts that they are routed to.
//
// Bound by reading the weights once.  They are the operand with 128 rows: a CTA
// multiplies 128 columns of W (for dA: 128 rows) by all tokens (16 to 128 columns of the
// accumulator) on tcgen05.  Scales that are powers of two are applied by the tensor cores; with fp32 scales each
// step of 128 goes to sums of its own in TMEM (four in turn), which the warps 4 to 7 scale and add up in
// their registers, unseen beside the weights' way (1 x 8192 x 28672 40.0 us against 39.9, 24 x 8192 x 8192 17.8
// against 17.1, 64 x 8192 x 28672 47).  The contraction is cut
// among the CTAs of a cluster, so that two CTAs on each SM stream weights at the same time
// (up to 64 rows: their shared memory and TMEM leave room for two); their partial sums meet in
// distributed shared memory, in the order of the CTAs, and the weighting of a token's experts
// takes place there.  One token through 8192 x 28672: 40 us; with one CTA an SM and a ring of
// twice the size 51 to 55, with runs of equal length over all tiles and sums joined in the
// workspace 47.
// The first weights are asked for before the quantisation of the rows is complete:
// that launch lets this one start only after everything before it is.
// Warps: 0 loads, 1 issues the MMAs, 2 brings scales, 4 to 7 read the sums.
#include <cuda.h>

#include <cstring>

#include "fp8.cuh"
#include "mx.cuh"
#include "tensor_pipe.cuh"

using namespace grs;

namespace {

constexpr int kThreads = 256;
// Scales.  Bytes: kSlots slots in shared memory and in TMEM, of four steps each.  fp32: kSteps slots in
// shared memory, of one step each, and as many steps' sums in TMEM as fit.
constexpr int kSlots = 4, kPerSlot = 4, kSfBytes = 512, kSlotBytes = 2 * kSfBytes;
constexpr int kSteps = 8, kSums = 4;
constexpr int kScaleBatch = 4;
constexpr int kWeightBytes = kBlk * 128;
constexpr uint64_t kLimitNs = 2000000000ull;  // of every wait

struct Params {
  CUtensorMap tok, w;
  const void *tok_scale, *w_scale;
  const int* offsets;
  void* out;
  const float* weights;
  const int* place;
  float* y;
  uint32_t* status;
  long long tok_stride;
  int M, width, experts, KB, NB, split, tokens, top_k;
};

template <int kRows>
struct Layout {
  // two CTAs an SM, for 128 rows one
  static constexpr int kStages = kRows == 16 ? 5 : kRows == 64 ? 3 : 4;
  static constexpr int kStageBytes = kWeightBytes + kRows * 128;
  static constexpr int kScales = kStages * kStageBytes;
  static constexpr int kPartial = kScales + kSlots * kSlotBytes;
  static constexpr int kBar = kPartial + kRows * 128 * 4;
  // full, empty, sf_full, sf_empty, acc_full, acc_empty, drain
  static constexpr int kNumBars = 2 * kStages + 2 * kSteps + 2 * kSums + 1;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kList = kMisc + 16;
  static constexpr int kAlloc = kList + kRows * 12 + 1024;
  static constexpr int kTmemScales = 2 * kRows;
  static constexpr int kTmemColumns = kRows == 16 ? 64 : kRows == 32 ? 128 : 256 + 256 * (kRows == 128);
  static_assert(kTmemScales + kSlots * 8 <= kTmemColumns && kSums * kRows <= kTmemColumns, "TMEM");
  static_assert(kSteps * kRows * 4 <= kSlots * kSlotBytes, "fp32 scales");
  static_assert(kRows == 128 ? kAlloc <= 232448 : 2 * (kAlloc + 1024) <= 233472, "shared memory of an SM");
};

// An expert that has rows (its index, first row, rows).
struct Active {
  int e, row0, rows;
};

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int kKind, int kRows, bool kE8m0>
__global__ void __launch_bounds__(kThreads, kRows == 128 ? 1 : 2) fp8_few_kernel(const __grid_constant__ Params p) {
  using L = Layout<kRows>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cta = (int)cluster_ctarank();
  const int tile = blockIdx.x / p.split;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_full = sbase + L::kBar;
  const uint32_t bar_empty = bar_full + 8 * L::kStages;
  const uint32_t bar_sf_full = bar_empty + 8 * L::kStages;
  const uint32_t bar_sf_empty = bar_sf_full + 8 * kSteps;
  const uint32_t bar_acc_full = bar_sf_empty + 8 * kSteps;
  const uint32_t bar_acc_empty = bar_acc_full + 8 * kSums;
  const uint32_t bar_drain = bar_acc_empty + 8 * kSums;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile uint32_t* cta_abort = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc + 4);
  int* count = reinterpret_cast<int*>(smem + L::kMisc + 8);
  Active* active = reinterpret_cast<Active*>(smem + L::kList);

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int s = 0; s < kSteps; ++s) {
      mbar_init(bar_sf_full + 8 * s, 1);
      mbar_init(bar_sf_empty + 8 * s, kE8m0 ? 1 : 4);  // an MMA commit, or the warps that read the sums
    }
    for (int b = 0; b < kSums; ++b) {
      mbar_init(bar_acc_full + 8 * b, 1);
      mbar_init(bar_acc_empty + 8 * b, 4);
    }
    mbar_init(bar_drain, 1);
    *cta_abort = 0;
    fence_mbar_init();
    fence_proxy_async_shared();
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(tmem_slot), L::kTmemColumns);
    tmem_relinquish<1>();
  }
  if (warp == 3) {
    // offsets were complete before the launch that this one may run beside
    int n = 0;
    if (!p.offsets) {
      if (lane == 0) active[0] = Active{0, 0, p.M};
      n = 1;
    } else {
      for (int e0 = 0; e0 < p.experts; e0 += 32) {
        const int e = e0 + lane;
        int first = 0, rows = 0;
        if (e < p.experts) {
          first = expert_row(p.offsets, e, p.M);
          rows = expert_row(p.offsets, e + 1, p.M) - first;
        }
        const uint32_t some = __ballot_sync(0xffffffffu, rows > 0);
        const int at = n + __popc(some & ((1u << lane) - 1));
        if (rows > 0 && at < kRows) active[at] = Active{e, first, rows};
        n += __popc(some);
      }
      n = n < kRows ? n : kRows;  // no more than there are rows
    }
    if (lane == 0) *count = n;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int n_active = *count;
  // of an expert; this CTA's are s_begin to s_end - 1
  const int steps = kKind == kFp8Forward ? kWorld * p.KB : p.NB;
  const int plane = kKind == kFp8Forward ? 0 : tile / p.KB, block = kKind == kFp8Forward ? tile : tile - plane * p.KB;
  const int s_begin = (int)((long long)steps * cta / p.split), s_end = (int)((long long)steps * (cta + 1) / p.split);

  if (warp == 0) {
    // ------------------------------------------------------------------- loader
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const int mine = s_end - s_begin, total = n_active * mine;
      const int early = total < L::kStages ? total : L::kStages;
      auto weights = [&](int e, int s, int st) {
        mbar_arrive_expect_tx(bar_full + 8 * st, L::kStageBytes);
        const int r = kKind == kFp8Forward ? s / p.KB : plane;
        const int k = kKind == kFp8Forward ? s - r * p.KB : block, n = kKind == kFp8Forward ? tile : s;
        tma_load_3d(sbase + st * L::kStageBytes, &p.w, bar_full + 8 * st, 0, k * kBlk, (e * kWorld + r) * p.NB + n);
      };
      auto rows = [&](int row0, int s, int st) {
        const int r = kKind == kFp8Forward ? s / p.KB : 0;
        tma_load_3d(sbase + st * L::kStageBytes + kWeightBytes, &p.tok, bar_full + 8 * st, (s - r * p.KB) * kBlk, row0,
                    r);
      };
      for (int g = 0, i = 0, s = s_begin; g < early; ++g) {
        weights(active[i].e, s, g);
        if (++s == s_end) {
          s = s_begin;
          ++i;
        }
      }
      griddep_wait();
      griddep_launch_dependents();
      fence_proxy_async_global();
      for (int g = 0, i = 0, s = s_begin; ok && g < total; ++g) {
        const Active a = active[i];
        if (g >= early) {
          if (!wait_bar(bar_empty + 8 * stage, phase ^ 1u, kLimitNs, cta_abort)) {
            *cta_abort = 1;
            ok = false;
            break;
          }
          weights(a.e, s, stage);
        }
        rows(a.row0, s, stage);
        if (++s == s_end) {
          s = s_begin;
          ++i;
        }
        if (++stage == L::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMA issuer
    const bool leader = elect_one();
    constexpr bool a_mn = kKind == kFp8Forward;
    constexpr uint32_t idesc = kE8m0 ? idesc_mx(kBlk, kRows, a_mn, 0) : idesc_e4m3(kBlk, kRows, a_mn, 0), a_step = a_mn ? 256 : 2;
    const uint64_t desc0 = smem_desc_sw128(sbase, 16, 1024);
    const uint32_t hi = (uint32_t)(desc0 >> 32);
    const uint64_t sf_desc = scales_desc(sbase + L::kScales);
    int stage = 0, slot = 0, buf = 0;
    uint32_t phase = 0, sf_phase = 0;
    bool ok = true;
    if constexpr (!kE8m0) {  // each step into sums of its own
      const int total = n_active * (s_end - s_begin);
      int acc = 0;
      uint32_t acc_phase = 0;
      for (int g = 0; g < total; ++g) {
        if (!wait_bar(bar_full + 8 * stage, phase, kLimitNs, cta_abort) ||
            !wait_bar(bar_acc_empty + 8 * acc, acc_phase ^ 1u, kLimitNs, cta_abort)) {
          *cta_abort = 1;
          break;
        }
        tc_fence_after();
        const uint32_t a = (uint32_t)desc0 + (uint32_t)(stage * (L::kStageBytes >> 4));
        const uint32_t b = a + (uint32_t)(kWeightBytes >> 4);
        if (leader) {
#pragma unroll
          for (uint32_t j = 0; j < kBlk / 32; ++j)
            mma_e4m3(tmem_base + acc * kRows, desc_join(a + a_step * j, hi), desc_join(b + 2 * j, hi), idesc, j != 0 ? 1u : 0u);
          mma_commit<1>(bar_acc_full + 8 * acc);
          mma_commit<1>(bar_empty + 8 * stage);
        }
        if (++stage == L::kStages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++acc == kSums) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      ok = false;
    }
    for (int i = 0; ok && i < n_active; ++i) {
      const int acc = i & 1;
      if (!wait_bar(bar_acc_empty + 8 * acc, ((i >> 1) & 1) ^ 1u, kLimitNs, cta_abort)) {
        *cta_abort = 1;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem_base + acc * kRows;
      for (int s = s_begin; s < s_end; ++s) {
        const uint32_t id = (uint32_t)s & (kPerSlot - 1);
        const bool fetch = s == s_begin || id == 0;
        if (!wait_bar(bar_full + 8 * stage, phase, kLimitNs, cta_abort) ||
            (fetch && !wait_bar(bar_sf_full + 8 * slot, sf_phase, kLimitNs, cta_abort))) {
          *cta_abort = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        if (fetch) {
          buf = slot;
          if (leader) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              copy_scales<1>(tmem_base + L::kTmemScales + buf * 8 + 4 * h,
                             sf_desc + (uint32_t)((buf * kSlotBytes + h * kSfBytes) >> 4));
          }
          if (++slot == kSlots) {
            slot = 0;
            sf_phase ^= 1u;
          }
        }
        const uint32_t a = (uint32_t)desc0 + (uint32_t)(stage * (L::kStageBytes >> 4));
        const uint32_t b = a + (uint32_t)(kWeightBytes >> 4);
        const uint32_t sf = tmem_base + L::kTmemScales + buf * 8;
        if (leader) {
#pragma unroll
          for (uint32_t j = 0; j < kBlk / 32; ++j)
            mma_scaled<1>(d, desc_join(a + a_step * j, hi), desc_join(b + 2 * j, hi), idesc_step(idesc, id), sf, sf + 4,
                          (s != s_begin || j != 0) ? 1u : 0u);
          mma_commit<1>(bar_empty + 8 * stage);
          if (id == kPerSlot - 1 || s == s_end - 1) mma_commit<1>(bar_sf_empty + 8 * buf);
        }
        if (++stage == L::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok && leader) mma_commit<1>(bar_acc_full + 8 * acc);
    }
    if (leader) mma_commit<1>(bar_drain);
    if (!wait_bar(bar_drain, 0, kDrainNs, cta_abort)) *cta_abort = 1;
  } else if (warp == 2) {
    // ------------------------------------------------------------------- scales
    griddep_wait();
    constexpr int kWords = (kRows + 31) / 32;
    if constexpr (!kE8m0) {
      // a step's for each row, times the weight's
      struct Step {
        float w, tok[kWords];
      } sf[kScaleBatch];
      int i = 0, step = s_begin, slot = 0;
      uint32_t phase = 0;
      auto fetch = [&](Step* x) {
        if (i >= n_active || s_begin == s_end) return false;
        const Active a = active[i];
        const float* w = static_cast<const float*>(p.w_scale);
        x->w = load_f32(kKind == kFp8Forward ? w + ((long long)a.e * steps + step) * p.NB + tile
                                             : w + ((long long)a.e * kWorld * p.KB + tile) * p.NB + step);
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          const int row = a.row0 + lane + 32 * j;
          x->tok[j] = load_f32(static_cast<const float*>(p.tok_scale) + step * p.tok_stride + (row < p.M ? row : p.M - 1));
        }
        if (++step == s_end) {
          step = s_begin;
          ++i;
        }
        return true;
      };
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
            if (lane == 0) *cta_abort = 1;
            ok = false;
            continue;
          }
#pragma unroll
          for (int k = 0; k < kWords; ++k)
            if (lane + 32 * k < kRows)
              st_shared_u32(sbase + L::kScales + (slot * kRows + lane + 32 * k) * 4, __float_as_uint(sf[j].w * sf[j].tok[k]));
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_sf_full + 8 * slot);
          if (++slot == kSteps) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
    }
    const int slot0 = s_begin / kPerSlot, slot1 = (s_end - 1) / kPerSlot;
    int i = 0, c = slot0, slot = 0;
    uint32_t phase = 0;
    struct Scales {
      uint32_t byte, tok[kWords];
    } sf[kScaleBatch];
    auto fetch = [&](Scales* x) {
      if (i >= n_active || s_begin == s_end) return false;
      const Active a = active[i];
      int step = c * kPerSlot + (lane & 3);
      step = step < steps ? step : steps - 1;
      if constexpr (kKind == kFp8Forward)
        x->byte = load_u8(static_cast<const uint8_t*>(p.w_scale) + ((long long)a.e * steps + step) * p.NB + tile);
      else
        x->byte = load_u8(static_cast<const uint8_t*>(p.w_scale) + ((long long)a.e * kWorld * p.KB + tile) * p.NB + step);
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        const int row = a.row0 + lane + 32 * j;
        x->tok[j] = load_u32(static_cast<const uint32_t*>(p.tok_scale) + c * p.tok_stride + (row < p.M ? row : p.M - 1));
      }
      if (++c > slot1) {
        c = slot0;
        ++i;
      }
      return true;
    };
    bool ok = kE8m0, more = true;
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
          if (lane == 0) *cta_abort = 1;
          ok = false;
          continue;
        }
        uint32_t word = 0, w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          word |= __shfl_sync(0xffffffffu, sf[j].byte, k) << (8 * k);
          w[k] = k < kWords ? sf[j].tok[k < kWords ? k : 0] : 0u;
        }
        const uint32_t dst = sbase + L::kScales + slot * kSlotBytes + lane * 16;
        st_shared_v4(dst, word, word, word, word);
        st_shared_v4(dst + kSfBytes, w[0], w[1], w[2], w[3]);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sf_full + 8 * slot);
        if (++slot == kSlots) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp >= 4) {
    // --------------------------------------------------------- sums to shared memory
    const int q = warp & 3;
    float* partial = reinterpret_cast<float*>(smem + L::kPartial) + q * 32 + lane;
    griddep_wait();
    if constexpr (!kE8m0) {
      // a step's products of codes, scaled, to sums in registers: a lane's column (for dA: row) of the weights
      int acc = 0, slot = 0;
      uint32_t acc_phase = 0, phase = 0;
      bool ok = true;
      for (int i = 0; ok && i < n_active; ++i) {
        const Active a = active[i];
        float sums[kRows];
#pragma unroll
        for (int c = 0; c < kRows; ++c) sums[c] = 0.f;
        for (int s = s_begin; s < s_end; ++s) {
          int got = 0;
          if (lane == 0)
            got = wait_bar(bar_sf_full + 8 * slot, phase, kLimitNs, cta_abort) &&
                  wait_bar(bar_acc_full + 8 * acc, acc_phase, kLimitNs, cta_abort);
          got = __shfl_sync(0xffffffffu, got, 0);
          if (!got) {
            if (lane == 0) *cta_abort = 1;
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kRows / 16; ++c) {
            uint32_t v[16];
            tmem_ld_16_columns(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kRows + 16 * c), v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float4 f;
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                           : "r"(sbase + L::kScales + (slot * kRows + 16 * c + 4 * k) * 4));
              sums[16 * c + 4 * k] = fmaf(__uint_as_float(v[4 * k]), f.x, sums[16 * c + 4 * k]);
              sums[16 * c + 4 * k + 1] = fmaf(__uint_as_float(v[4 * k + 1]), f.y, sums[16 * c + 4 * k + 1]);
              sums[16 * c + 4 * k + 2] = fmaf(__uint_as_float(v[4 * k + 2]), f.z, sums[16 * c + 4 * k + 2]);
              sums[16 * c + 4 * k + 3] = fmaf(__uint_as_float(v[4 * k + 3]), f.w, sums[16 * c + 4 * k + 3]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar_acc_empty + 8 * acc);
            mbar_arrive(bar_sf_empty + 8 * slot);
          }
          if (++acc == kSums) {
            acc = 0;
            acc_phase ^= 1u;
          }
          if (++slot == kSteps) {
            slot = 0;
            phase ^= 1u;
          }
        }
#pragma unroll
        for (int c = 0; c < kRows; ++c)
          if (ok && c < a.rows && a.row0 + c < kRows) partial[(a.row0 + c) * 128] = sums[c];
      }
    }
    for (int i = 0; kE8m0 && i < n_active; ++i) {
      const Active a = active[i];
      const int acc = i & 1;
      int got = 0;
      if (lane == 0) got = wait_bar(bar_acc_full + 8 * acc, (i >> 1) & 1, kLimitNs, cta_abort) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) {
        if (lane == 0) *cta_abort = 1;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kRows / 16; ++c) {
        uint32_t v[16];
        tmem_ld_16_columns(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kRows + 16 * c), v);
        if (s_begin == s_end) {
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = 0;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (16 * c + k < a.rows && a.row0 + 16 * c + k < kRows)
            partial[(a.row0 + 16 * c + k) * 128] = __uint_as_float(v[k]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_acc_empty + 8 * acc);
    }
  } else {
    griddep_wait();
  }

  __syncwarp();
  griddep_wait();
  tc_fence_before();
  __syncthreads();
  // every CTA's sums are in its shared memory, its copies and MMAs have ended; releasing all memory here and
  // below took 24 x 8192 x 8192 from 16.8 to 17.7 us
  cluster_sync_shared();
  if (*cta_abort) settle();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<1>(tmem_base, L::kTmemColumns);
  }
  if (*cta_abort && threadIdx.x == 0) *p.status = 1;
  // This CTA adds up its share of the tile's outputs, two columns for a thread, 16 pairs
  // of columns in turn for each CTA.
  const uint32_t partial = sbase + L::kPartial;
  const int rows = n_active ? active[n_active - 1].row0 + active[n_active - 1].rows : 0;
  const int items = (p.place ? p.tokens : rows) * (kBlk / 2);
  for (int x = cta * 16 + threadIdx.x / 16 * (16 * p.split) + threadIdx.x % 16; x < items; x += kThreads * p.split) {
    const int t = x / (kBlk / 2), n = 2 * (x % (kBlk / 2)), col = block * kBlk + n;
    if (col >= p.width) continue;
    float2 sum = make_float2(0.f, 0.f);
    for (int j = 0; j < p.top_k; ++j) {
      const int row = p.place ? p.place[t * p.top_k + j] : t;
      if ((unsigned)row >= (unsigned)p.M) continue;
      float2 y = make_float2(0.f, 0.f);
#pragma unroll 8
      for (int c = 0; c < p.split; ++c) {
        float2 v;
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                     : "=f"(v.x), "=f"(v.y)
                     : "r"(mapa_shared(partial + (uint32_t)(row * 128 + n) * 4, c))
                     : "memory");
        y.x += v.x;
        y.y += v.y;
      }
      if (p.y) *reinterpret_cast<float2*>(p.y + (long long)row * p.width + col) = y;
      if (p.place) {
        const float w = p.weights[t * p.top_k + j];
        sum.x = fmaf(w, y.x, sum.x);
        sum.y = fmaf(w, y.y, sum.y);
      } else {
        sum = y;
      }
    }
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + ((long long)plane * p.M + t) * p.width + col) =
        pack_bf16x2(sum.x, sum.y);
  }
  cluster_sync_shared();  // every CTA's shared memory has been read
}

template <int kKind, int kRows, bool kE8m0>
int launch(const Params& p, int tiles, cudaStream_t st) {
  using L = Layout<kRows>;
  static SmemAllowed allowed;
  if (!allowed.set(fp8_few_kernel<kKind, kRows, kE8m0>, L::kAlloc)) return GEMM_RS_ERR_CUDA;
  return launch_cluster(fp8_few_kernel<kKind, kRows, kE8m0>, tiles * p.split, p.split, kThreads, L::kAlloc, st, p);
}

template <int kKind, bool kE8m0>
int launch_rows(const Params& p, int rows, int tiles, cudaStream_t st) {
  return rows == 16   ? launch<kKind, 16, kE8m0>(p, tiles, st)
         : rows == 32 ? launch<kKind, 32, kE8m0>(p, tiles, st)
         : rows == 64 ? launch<kKind, 64, kE8m0>(p, tiles, st)
                      : launch<kKind, 128, kE8m0>(p, tiles, st);
}
template <bool kE8m0>
int launch_kind(bool forward, const Params& p, int rows, int tiles, cudaStream_t st) {
  return forward ? launch_rows<kFp8Forward, kE8m0>(p, rows, tiles, st) : launch_rows<kFp8InputGrad, kE8m0>(p, rows, tiles, st);
}

// Of the accumulator, for M rows.
int rows_of(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// Parts of the contraction: as many as run at once.  Where one CTA fits an SM, clusters of 8 leave a part
// of the SMs unused: 16 of them do not run at once (100 x 2048 x 4096 19.8 us, in clusters of 4 12.1).
int split_of(int rows, int tiles, int steps, int sms) {
  const int slots = rows == 128 ? sms : 2 * sms;
  int split = rows == 128 && tiles * 8 > sms * 3 / 4 ? 4 : 8;
  while (split > 1 && (tiles * split > slots || split > steps)) split /= 2;
  return split;
}

struct Grid {
  int tiles, steps, split;
};
Grid grid_of(Fp8Kind kind, int64_t M, int64_t N, int64_t Kr, int sms) {
  const int KB = (int)blocks_of(Kr), NB = (int)blocks_of(N);
  Grid g = {kind == kFp8Forward ? NB : kWorld * KB, kind == kFp8Forward ? kWorld * KB : NB, 1};
  g.split = split_of(rows_of(M), g.tiles, g.steps, sms);
  return g;
}

}  // namespace

// Estimated times, in units of 10 ns, fitted to 150 shapes of 1 to 128 rows, 152 to 28672 columns and 1 to 16
// experts with powers of two; the choice is within 15% of the faster one.  With fp32 scales both take a little
// longer: of 148 shapes the choice is the faster one or within 7% of it in 145, within 20% in all.  Here a CTA goes through its part of
// every expert in turn, there experts are side by side and a tile is 256 rows whatever it holds.
// 128 x 28672 x 8192 forward 81 against 55 us, 128 x 8192 x 28672 61 against 73, one row 40 against 76;
// 32 rows of 16 experts, 1024 x 8192, 63 against 33.
bool grs::fp8_few_serves(Fp8Kind kind, const Fp8Rows& rows, int64_t N, int64_t Kr, bool with_weight_grad, int sms) {
  if (rows.M > kFewRows) return false;
  const int64_t E = rows.offsets ? rows.experts : 1;
  // up to 32 M weights one launch for both gradients is faster (128 x 2048 x 4096 42 -> 17.5 us), above it the
  // weights are better streamed once (64 x 8192 x 8192 51 against 58)
  if (with_weight_grad && E * N * Kr * kWorld <= 1ll << 25) return false;
  const Grid g = grid_of(kind, rows.M, N, Kr, sms);
  const int n = rows_of(rows.M);
  const int64_t active = E < rows.M ? E : rows.M;
  const int64_t step = n == 16 ? 28 : n == 32 ? 33 : n == 64 ? 42 : 45, expert = n == 16 ? 40 : n == 32 ? 60 : n == 64 ? 120 : 750;
  const int64_t slots = n == 128 ? sms : 2 * sms, waves = ((int64_t)g.tiles * g.split + slots - 1) / slots;
  const int64_t few = waves * active * ((g.steps + g.split - 1) / g.split * step + expert);
  const int64_t wide = kind == kFp8Forward ? (N + 255) / 256 : kWorld * ((Kr + 255) / 256), pairs = sms / 2;
  const int64_t tiles = 250 + (active * wide + pairs - 1) / pairs * (g.steps * 29 + 250);
  const int64_t weighting = rows.offsets && kind == kFp8Forward ? 400 : 0;  // in a launch of its own there
  return few <= tiles + weighting;
}

int grs::fp8_few(const Fp8Few& d, cudaStream_t st) {
  const int64_t M = d.rows.M, N = d.N, Kr = d.Kr, E = d.rows.experts;
  int sms = 0;
  const int rc = current_device_sms(&sms);
  if (rc) return rc;
  const bool fwd = d.kind == kFp8Forward;
  Params p;
  memset(&p, 0, sizeof(p));
  p.tok_scale = d.a_scale;
  p.w_scale = d.b_scale;
  p.offsets = d.rows.offsets;
  p.out = d.out;
  p.weights = d.weights;
  p.place = d.place;
  p.y = d.y;
  p.status = d.status;
  p.tok_stride = row_scale_pitch(M);
  p.M = (int)M;
  p.width = (int)(fwd ? N : Kr);
  p.experts = (int)E;
  p.KB = (int)blocks_of(Kr);
  p.NB = (int)blocks_of(N);
  p.tokens = (int)d.tokens;
  p.top_k = d.place ? d.rows.top_k : 1;
  const Grid g = grid_of(d.kind, M, N, Kr, sms);
  const int tiles = g.tiles, rows = rows_of(M);
  p.split = g.split;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!(fwd ? encode_map(&p.tok, u8, 1, d.a, Kr, M, kWorld, kBlk, rows, fp8_pitch(Kr))
            : encode_map(&p.tok, u8, 1, d.a, N, M, 1, kBlk, rows, fp8_pitch(N))) ||
      !encode_map(&p.w, u8, 1, d.b, kBlk, Kr, kWorld * E * blocks_of(N), kBlk, kBlk, kBlk))
    return GEMM_RS_ERR_CUDA;
  return d.scale == kFp8F32 ? launch_kind<false>(fwd, p, rows, tiles, st) : launch_kind<true>(fwd, p, rows, tiles, st);
}
