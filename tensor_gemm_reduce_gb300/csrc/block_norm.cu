// block_norm.cu -- the norms after and before a block, fused with the block's
// gate and residual scale, forward and backward (gemm_rs_norm_* in
// include/gemm_rs_ops.h).
//
// Both passes read each row once and are bound by HBM: 8 bytes an element forward,
// 12 backward (14 and 16 with a gate value for each).  Measured on a GB300, whose
// copies reach 6.79 TB/s: forward 2048 x 8192 with 4 gate rows 25.6 us (5.2 TB/s),
// 8192 x 8192 85.1 us (6.3 TB/s), one row 3.5 us; backward 8192 x 8192 with the join
// of the sums over rows 125 us (6.4 TB/s), 1003 x 6152 with a gate value for each
// element 25.5 us (3.9 TB/s: 7 rows a block, of which the first and the last run
// beside nothing, and 3.5 us of join).
#include <cmath>

#include "ops_common.cuh"

using namespace grs;

namespace {

constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxSmem = 224 * 1024;  // of the SM's 228 KB
constexpr int kBackwardSmem = 200 * 1024;
// The backward pass cuts the rows into at most kBlocks x groups chunks, one
// block per SM of a GB300.  A constant, so that the workspace size and the
// order of the sums do not depend on the device.
constexpr int kBlocks = 152;

// Where the backward pass has the gate: one row (or none) is held in registers
// like the weights; a row for some rows each (kSequence) or for each row
// (kElement) goes through the ring with the row's other inputs.
enum GateMode : int { kSingle = 0, kSequence = 1, kElement = 2 };

// In the backward pass three and four vectors a thread leave too few registers for
// the weights, and spilled ones go to L2 where the ring takes most of L1: w_pre lies
// in shared memory (w_post too, where shared memory holds both), and w_post stays
// packed where the gate is not multiplied into it.  us, M x D: 4096 x 12288 with one
// gate row 137.7 -> 101.8, with 4 170 -> 143, with 4096 164 -> 146; 2048 x 9912 75 ->
// 57; 8192 x 4160 with 8 gate rows 133 -> 110.
__host__ __device__ constexpr bool pre_in_shared(int v, int mode) { return v == 3 || (v == 4 && mode != kSequence); }
__host__ __device__ constexpr bool post_in_shared(int v, int mode) { return v == 3 && mode == kSequence; }
__host__ __device__ constexpr bool post_packed(int v, int mode) { return v >= 3 && mode != kSingle; }

// A row belongs to a group of `warps` warps, thread t of the group holding its
// 16-byte vectors t, t + 32 warps, ... (`v` of them at most); a block has
// `groups` such groups, each with rows of its own.  Every thread copies the
// vectors that it will use into a ring of `stages` rows in shared memory with
// cp.async, so rows arrive while earlier ones are worked on, without registers
// for them and without a barrier: a thread waits for its own copies only.
struct Shape {
  int v, warps, groups, stages, smem;
};
// backward: the pass's GateMode, or -1 for the forward pass.
Shape shape_of(int nv, int arrays, long long rows, int blocks, int budget, int extra_per_vector, int backward = -1) {
  Shape s = {0, 0, 0, 0, 0};
  // Two vectors a thread unless that leaves more than a quarter of the warps out.
  int best = 0;
  for (int v : {2, 3, 1, 4}) {
    if (nv <= 32) v = 1;
    const int warps = (nv + 32 * v - 1) / (32 * v);
    if (warps > kMaxWarps) continue;
    const int groups = kMaxWarps / warps;
    const int used = groups * warps;
    if (used > best) {
      best = used;
      s.v = v;
      s.warps = warps;
      s.groups = groups;
      if (used >= kMaxWarps * 3 / 4) break;
    }
  }
  // few rows: spread them over the blocks first
  const long long need = (rows + blocks - 1) / blocks;
  if (s.groups > need) s.groups = need < 1 ? 1 : (int)need;
  const int row = s.groups * nv * 16;
  int extra = s.groups * nv * extra_per_vector;
  if (backward >= 0 && pre_in_shared(s.v, backward)) {
    const int weights = post_in_shared(s.v, backward) ? 2 * row : row;
    extra += weights;
    if (s.v == 3) budget = budget + weights < kMaxSmem ? budget + weights : kMaxSmem;
  }
  s.stages = (budget - extra) / (arrays * row);
  // Two are enough: a third row in flight gained nothing on 8192 rows of 8192
  // and queued in front of the first row on 1003 (16.5 against 15.2 us).
  if (s.stages > 2) s.stages = 2;
  if (s.stages < 1) s.stages = 1;
  s.smem = s.stages * arrays * row + extra;
  return s;
}

struct NormParams {
  uint32_t M;               // M * nv stays below 2^31: vector indexes are 32-bit
  int D, nv;                // nv = D / 8 vectors of 16 bytes in a row
  int warps, groups, stages;
  uint32_t rows_per_gate;   // M / gate_rows
  float scale, eps, inv_d;
  float least, least_eps;   // D 2^-124, and that less D eps
  const uint4 *x, *y, *gate, *w_post, *w_pre;
  uint4 *r, *h;
  float* stats;
  // backward
  const uint4 *dr, *dh;
  uint4 *dx, *dy, *dgate, *dw_post, *dw_pre;
  // Rows of a group: chunk_rows consecutive ones (step = 1) where a gate row
  // serves several of them, else rows `step` = the number of groups apart, so
  // that all blocks work on one region of memory at a time (8192 x 8192: 101 ->
  // 96 us forward, 133 -> 127 us backward).
  uint32_t chunk_rows, step;
  int chunks, blocks;
  float *part_post, *part_pre, *part_gate;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most `stages` - 1 of this thread's copy groups are pending.
__device__ __forceinline__ void cp_async_wait(int stages) {
  if (stages == 2)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Two fp32 values in a register pair: one instruction for both (the kernels are
// bound by instruction issue as much as by HBM).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 floats(F2 a) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(a.v));
  return f;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 both(float a) { return f2(a, a); }
__device__ __forceinline__ float sum(F2 a) {
  const float2 f = floats(a);
  return f.x + f.y;
}
__device__ __forceinline__ F2 from_bf16x2(uint32_t w) { return f2(bf16lo_to_f32(w), bf16hi_to_f32(w)); }
__device__ __forceinline__ uint32_t to_bf16x2(F2 a) {
  const float2 f = floats(a);
  return pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ void unpack8(const uint4& v, F2 (&f)[4]) {
  f[0] = from_bf16x2(v.x);
  f[1] = from_bf16x2(v.y);
  f[2] = from_bf16x2(v.z);
  f[3] = from_bf16x2(v.w);
}
__device__ __forceinline__ uint4 pack8(const F2 (&f)[4]) {
  return make_uint4(to_bf16x2(f[0]), to_bf16x2(f[1]), to_bf16x2(f[2]), to_bf16x2(f[3]));
}
__device__ __forceinline__ void store8(float* p, const F2 (&f)[4]) {
  float4* q = reinterpret_cast<float4*>(p);
  const float2 a = floats(f[0]), b = floats(f[1]), c = floats(f[2]), d = floats(f[3]);
  q[0] = make_float4(a.x, a.y, b.x, b.y);
  q[1] = make_float4(c.x, c.y, d.x, d.y);
}

// Sums of four values over a group, in each of its threads.  The first two
// exchanges halve the values that a lane carries (lane bits 4 and 3 select one
// of the four), so a warp takes 6 shuffles instead of 20.  `part` has a place
// for each value and warp; a group alternates between two of them, so that one
// barrier a sum is enough.
__device__ __forceinline__ void group_sum4(float (&v)[4], float (&part)[4][kMaxWarps], int warps, int group) {
  const int lane = threadIdx.x & 31;
  const bool hi = lane & 16, odd = lane & 8;
  const float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
  const float b = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
  float s = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  // lanes 8 i .. 8 i + 7 hold the warp's sum of value i
  if (warps > 1) {
    if ((lane & 7) == 0) part[lane >> 3][threadIdx.x >> 5] = s;
    asm volatile("barrier.sync.aligned %0, %1;" ::"r"(group + 1), "r"(32 * warps) : "memory");
    // lane 8 i + j adds value i of warps j and j + 8
    const int j = lane & 7;
    const float* row = &part[lane >> 3][group * warps];
    s = (j < warps ? row[j] : 0.f) + (j + 8 < warps ? row[j + 8] : 0.f);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, s, 8 * i);
}

// Blocks of the forward kernel that share an SM: with up to two vectors a
// thread 64 registers are enough.
constexpr int forward_blocks(int v) { return v <= 2 ? 2 : 1; }

// With c = scale gate w_post y the row's residual is r = x + p c, so
//   sum r^2 = sum x^2 + 2 p sum x c + p^2 sum c^2
// and one sum of four values (y^2, x^2, x c, c^2) serves both norms.  sum r^2 is
// taken directly where it would not have its digits:
//   sum r^2 + D eps < (terms that are not negative) / 4 + D 2^-124 (1 + p^2)
// The first part is a branch that cancels most of x, where the rounding of the terms
// would show; the second are products below 2^-126, each off by 2^-150 and multiplied
// by up to 1 + p^2.  An overflowing term or p^2 leaves NaN or infinity in the
// comparison, which does not hold then either.
// The row stays in the ring until it is written and is unpacked twice: keeping
// it in registers spilled some of them, and with most of the SM's memory given
// to the ring every spill went to L2.
// A gate row that serves several consecutive rows of a group stays in registers
// with w_post; kGateRing: the gate's row arrives through the ring instead (without
// a gate w_post does, and the registers hold scale alone).
template <int V, bool kGateRing>
__global__ void __launch_bounds__(kMaxThreads, forward_blocks(V)) norm_forward_kernel(const NormParams p) {
  extern __shared__ uint4 ring[];
  __shared__ float part[2][4][kMaxWarps];
  constexpr int kArrays = kGateRing ? 3 : 2;
  const int group = (int)(threadIdx.x >> 5) / p.warps, T = 32 * p.warps;
  const int t = threadIdx.x - group * T;
  const uint32_t mine = smem_u32(ring) + 16u * (group * p.nv + t);
  const uint32_t plane = 16u * p.groups * p.nv;  // one array of a stage
  const uint32_t c = blockIdx.x * p.groups + group, step = p.step;
  const uint32_t m0 = step == 1 ? c * p.chunk_rows : c;
  const uint32_t m1 = step == 1 && m0 + p.chunk_rows < p.M ? m0 + p.chunk_rows : p.M;
  griddep_launch_dependents();  // the next launch's blocks take the places that free up, and wait
  griddep_wait();

  const uint4* factor = p.gate ? p.gate : p.w_post;
  auto fetch = [&](uint32_t row, int stage) {
    if (row < m1) {
      const uint32_t base = mine + (uint32_t)(stage * kArrays) * plane;
      const uint32_t at = row * p.nv + t, gat = (kGateRing && p.gate ? row / p.rows_per_gate * p.nv : 0) + t;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (t + v * T < p.nv) {
          cp_async16(base + 16u * v * T, p.y + (at + v * T));
          cp_async16(base + plane + 16u * v * T, p.x + (at + v * T));
          if (kGateRing) cp_async16(base + 2 * plane + 16u * v * T, factor + (gat + v * T));
        }
    }
    cp_async_commit();
  };
  for (int s = 0; s < p.stages; ++s) fetch(m0 + s * step, s);
  // this thread's vectors of w_pre, after the ring: 64 registers do not hold
  // them, and L1 has too little room beside the ring
  uint4* w_pre = ring + (size_t)(p.stages * kArrays) * p.groups * p.nv + group * p.nv + t;
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (t + v * T < p.nv) w_pre[v * T] = load_v4(p.w_pre + t + v * T);
  F2 gw[V][4];  // the branch's factors that are not in the ring
  auto branch_weights = [&](uint32_t gate_row) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (t + v * T < p.nv) {
        if (kGateRing && !p.gate) {
#pragma unroll
          for (int j = 0; j < 4; ++j) gw[v][j] = both(p.scale);
          continue;
        }
        unpack8(load_v4(p.w_post + t + v * T), gw[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) gw[v][j] = gw[v][j] * both(p.scale);
        if (!kGateRing && p.gate) {
          F2 g[4];
          unpack8(load_v4(p.gate + gate_row * p.nv + t + v * T), g);
#pragma unroll
          for (int j = 0; j < 4; ++j) gw[v][j] = gw[v][j] * g[j];
        }
      }
  };
  uint32_t gate_row = p.gate ? m0 / p.rows_per_gate : 0, gate_end = p.gate ? (gate_row + 1) * p.rows_per_gate : p.M;
  if (m0 < p.M) branch_weights(gate_row);

  int stage = 0;
  uint32_t it = 0;
#pragma unroll 1
  for (uint32_t m = m0; m < m1; m += step, ++it) {
    if (!kGateRing && m == gate_end) {
      branch_weights(++gate_row);
      gate_end += p.rows_per_gate;
    }
    cp_async_wait(p.stages);
    const uint32_t base = mine + (uint32_t)(stage * kArrays) * plane;
    // y, x and the branch c of one vector, from the ring
    auto load = [&](int v, F2 (&y)[4], F2 (&x)[4], F2 (&c)[4]) {
      unpack8(ld_shared_v4(base + 16u * v * T), y);
      unpack8(ld_shared_v4(base + plane + 16u * v * T), x);
      if (kGateRing) unpack8(ld_shared_v4(base + 2 * plane + 16u * v * T), c);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = kGateRing ? c[j] * gw[v][j] * y[j] : gw[v][j] * y[j];
    };
    F2 yy = both(0.f), xx = yy, xc = yy, cc = yy;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (t + v * T < p.nv) {
        F2 y[4], x[4], c[4];
        load(v, y, x, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          yy = fma2(y[j], y[j], yy);
          xx = fma2(x[j], x[j], xx);
          xc = fma2(x[j], c[j], xc);
          cc = fma2(c[j], c[j], cc);
        }
      }
    float s[4] = {sum(yy), sum(xx), sum(xc), sum(cc)};
    group_sum4(s, part[it & 1], p.warps, group);
    const float pn = 1.f / sqrtf(fmaf(s[0], p.inv_d, p.eps));
    const F2 pn2 = both(pn);
    const float terms = fmaf(pn * pn, s[3], s[1]);
    float rr = fmaf(2.f * pn, s[2], terms);
    // the same in every thread of the group
    if (!(fmaf(-0.25f, terms, rr) >= fmaf(pn * pn, p.least, p.least_eps))) {
      F2 acc = both(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (t + v * T < p.nv) {
          F2 y[4], x[4], c[4];
          load(v, y, x, c);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const F2 r = fma2(c[j], pn2, x[j]);
            acc = fma2(r, r, acc);
          }
        }
      float d[4] = {sum(acc), 0.f, 0.f, 0.f};
      if (p.warps > 1) asm volatile("barrier.sync.aligned %0, %1;" ::"r"(group + 1), "r"(32 * p.warps) : "memory");
      group_sum4(d, part[it & 1], p.warps, group);
      rr = d[0];
    }
    const float qn = 1.f / sqrtf(fmaf(rr, p.inv_d, p.eps));
    const F2 qn2 = both(qn);
    const uint32_t at = m * p.nv + t;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (t + v * T < p.nv) {
        F2 y[4], x[4], c[4];
        load(v, y, x, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = fma2(c[j], pn2, x[j]);
        p.r[at + v * T] = pack8(x);
        unpack8(w_pre[v * T], y);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = y[j] * (x[j] * qn2);
        p.h[at + v * T] = pack8(x);
      }
    fetch(m + p.stages * step, stage);  // every read of the slot is done
    if (++stage == p.stages) stage = 0;
    if (p.stats && t == 0) {
      p.stats[m] = pn;
      p.stats[p.M + m] = qn;
    }
  }
}

// Backward.  With yn = y p, c = scale gate yn w_post (the branch), rn = (x + c) q,
// a = dh w_pre and m1 = mean(a rn):
//   t  = dr + q (a - rn m1)                       dx = t
//   dy = p (scale gate t w_post - yn m2),         m2 = mean(scale gate t w_post yn)
//                                                    = mean(c (dr + q a)) - q m1 mean(c rn)
// so one sum of three values over the row serves both norms.
// Each group owns rows and its threads own columns, so the sums over rows stay
// in registers: the sum S of t yn over the rows of one
// gate row gives both dgate = scale w_post S and that gate row's share
// scale gate S of dw_post; the sum of dh rn is dw_pre.  kSequence adds the
// shares of dw_post in shared memory, at the end of each gate row; kElement
// has no S.  A gate row whose rows all lie in the chunk is written at once;
// one that crosses a chunk border leaves a partial sum in slot 2 c (its rows
// begin at the chunk's first row or before) or 2 c + 1.  At the end the
// block's groups are added and the block writes one row of partial sums.
// As in the forward pass the row is unpacked twice rather than kept.
template <int V, int kMode>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_backward_kernel(const NormParams p) {
  extern __shared__ uint4 ring[];
  __shared__ float part[2][4][kMaxWarps];
  constexpr int kArrays = kMode == kSingle ? 4 : 5;
  const int group = (int)(threadIdx.x >> 5) / p.warps, T = 32 * p.warps;
  const int t = threadIdx.x - group * T;
  const uint32_t mine = smem_u32(ring) + 16u * (group * p.nv + t);
  const uint32_t plane = 16u * p.groups * p.nv;
  // kSequence: this thread's columns of dw_post, after the ring
  float* post = reinterpret_cast<float*>(ring + (size_t)p.stages * kArrays * p.groups * p.nv) + 8 * (group * p.nv + t);
  const uint32_t c = blockIdx.x * p.groups + group;
  const uint32_t step = kMode == kSequence ? 1 : p.step;
  const uint32_t m0 = step == 1 ? (c * p.chunk_rows < p.M ? c * p.chunk_rows : p.M) : c;
  const uint32_t m1 = step == 1 && m0 + p.chunk_rows < p.M ? m0 + p.chunk_rows : p.M;
  griddep_launch_dependents();  // the next launch's blocks take the places that free up, and wait
  griddep_wait();

  auto fetch = [&](uint32_t row, int stage) {
    if (row < m1) {
      const uint32_t base = mine + (uint32_t)(stage * kArrays) * plane;
      const uint32_t at = row * p.nv + t;
      const uint32_t gat = kMode == kSequence ? row / p.rows_per_gate * p.nv + t : at;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (t + v * T < p.nv) {
          const uint32_t dst = base + 16u * v * T;
          cp_async16(dst, p.y + (at + v * T));
          cp_async16(dst + plane, p.x + (at + v * T));
          cp_async16(dst + 2 * plane, p.dr + (at + v * T));
          cp_async16(dst + 3 * plane, p.dh + (at + v * T));
          if (kMode != kSingle) cp_async16(dst + 4 * plane, p.gate + (gat + v * T));
        }
    }
    cp_async_commit();
  };
  for (int s = 0; s < p.stages; ++s) fetch(m0 + s * step, s);

  constexpr bool kPreShared = pre_in_shared(V, kMode), kPacked = post_packed(V, kMode);
  F2 gw[kPacked ? 1 : V][4];  // scale w_post, times the gate when there is one row of it
  constexpr bool kPostShared = post_in_shared(V, kMode);
  uint4 wp[kPacked && !kPostShared ? V : 1], wq[kPreShared ? 1 : V];
  // this thread's vectors of w_pre, after the ring and the columns of dw_post
  const uint32_t pre = mine + plane * (p.stages * kArrays + (kMode == kSequence ? 2 : 0));
  F2 S[V][4], Ppre[V][4];  // kElement: S is this thread's sum for dw_post
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = t + v * T;
#pragma unroll
    for (int j = 0; j < 4; ++j) S[v][j] = Ppre[v][j] = both(0.f);
    if (i < p.nv) {
      const uint4 post_w = load_v4(p.w_post + i), pre_w = load_v4(p.w_pre + i);
      if constexpr (kPreShared)
        ring[(pre - smem_u32(ring)) / 16 + v * T] = pre_w;
      else
        wq[v] = pre_w;
      if constexpr (kPostShared) {
        ring[(pre + plane - smem_u32(ring)) / 16 + v * T] = post_w;
      } else if constexpr (kPacked) {
        wp[v] = post_w;
      } else {
        unpack8(post_w, gw[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) gw[v][j] = gw[v][j] * both(p.scale);
        if (kMode == kSingle && p.gate) {
          F2 g[4];
          unpack8(load_v4(p.gate + i), g);
#pragma unroll
          for (int j = 0; j < 4; ++j) gw[v][j] = gw[v][j] * g[j];
        }
      }
      if (kMode == kSequence) store8(post + 8 * v * T, S[v]);
    }
  }

  auto w_pre = [&](int v) {
    if constexpr (kPreShared)
      return ld_shared_v4(pre + 16u * v * T);
    else
      return wq[v];
  };
  auto factors = [&](int v, F2 (&f)[4]) {
    if constexpr (kPostShared)
      unpack8(ld_shared_v4(pre + plane + 16u * v * T), f);
    else if constexpr (kPacked)
      unpack8(wp[v], f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kPacked)
        f[j] = f[j] * both(p.scale);
      else
        f[j] = gw[v][j];
    }
  };
  int stage = 0;
  // the rows' statistics, one row ahead
  float pn_next = m0 < m1 ? load_f32(p.stats + m0) : 0.f, qn_next = m0 < m1 ? load_f32(p.stats + p.M + m0) : 0.f;
  uint32_t it = 0;
#pragma unroll 1
  for (uint32_t m = m0; m < m1; m += step, ++it) {
    const float pn = pn_next, qn = qn_next;
    if (m + step < m1) {
      pn_next = load_f32(p.stats + m + step);
      qn_next = load_f32(p.stats + p.M + m + step);
    }
    cp_async_wait(p.stages);
    const uint32_t base = mine + (uint32_t)(stage * kArrays) * plane;
    F2 s0 = both(0.f), s1 = s0, s2 = s0;
    const F2 pn2 = both(pn), qn2 = both(qn);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (t + v * T < p.nv) {
        const uint32_t src = base + 16u * v * T;
        F2 y[4], x[4], z[4], dh[4], w[4], g[4], gv[4];
        factors(v, gv);
        unpack8(ld_shared_v4(src), y);
        unpack8(ld_shared_v4(src + plane), x);
        unpack8(ld_shared_v4(src + 2 * plane), z);
        unpack8(ld_shared_v4(src + 3 * plane), dh);
        unpack8(w_pre(v), w);
        if (kMode != kSingle) unpack8(ld_shared_v4(src + 4 * plane), g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const F2 br = (kMode != kSingle ? g[j] * gv[j] : gv[j]) * (y[j] * pn2);
          const F2 rn = (x[j] + br) * qn2;
          const F2 a = dh[j] * w[j];
          Ppre[v][j] = fma2(dh[j], rn, Ppre[v][j]);
          s0 = fma2(a, rn, s0);
          s1 = fma2(br, fma2(qn2, a, z[j]), s1);
          s2 = fma2(br, rn, s2);
        }
      }
    }
    float s[4] = {sum(s0), sum(s1), sum(s2), 0.f};
    group_sum4(s, part[it & 1], p.warps, group);
    const float k1 = qn * (s[0] * p.inv_d);                 // q m1
    const float k2 = fmaf(-k1, s[2], s[1]) * p.inv_d * pn;  // p m2
    const F2 nk1 = both(-k1), nk2 = both(-k2);
    const uint32_t gi = kMode == kSequence ? m / p.rows_per_gate : m;
    const bool last = kMode == kSequence && (m + 1 == m1 || m + 1 == (gi + 1) * p.rows_per_gate);
    const uint32_t at = m * p.nv + t;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (t + v * T < p.nv) {
        const uint32_t src = base + 16u * v * T;
        F2 yn[4], g[4], dx[4], dy[4], gv[4];
        factors(v, gv);
        {
          F2 x[4], dh[4], w[4];
          unpack8(ld_shared_v4(src), yn);
          unpack8(ld_shared_v4(src + plane), x);
          unpack8(ld_shared_v4(src + 2 * plane), dx);
          unpack8(ld_shared_v4(src + 3 * plane), dh);
          unpack8(w_pre(v), w);
          if (kMode != kSingle) unpack8(ld_shared_v4(src + 4 * plane), g);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            yn[j] = yn[j] * pn2;
            const F2 f = kMode != kSingle ? g[j] * gv[j] : gv[j];
            const F2 e = fma2(nk1, fma2(f, yn[j], x[j]), dh[j] * w[j]);  // a - rn m1
            dx[j] = fma2(qn2, e, dx[j]);
            dy[j] = fma2(dx[j] * f, pn2, nk2 * yn[j]);
          }
        }
        p.dx[at + v * T] = pack8(dx);
        p.dy[at + v * T] = pack8(dy);
        if (kMode == kElement) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const F2 ty = dx[j] * yn[j];
            S[v][j] = fma2(g[j], ty, S[v][j]);
            dx[j] = gv[j] * ty;
          }
          p.dgate[at + v * T] = pack8(dx);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) S[v][j] = fma2(dx[j], yn[j], S[v][j]);
        }
        if (kMode == kSequence && last) {  // end of a gate row's rows in this chunk
          const uint32_t first = gi * p.rows_per_gate;
          const int i = t + v * T;
          if (first >= m0 && first + p.rows_per_gate <= m1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) dx[j] = gv[j] * S[v][j];
            p.dgate[gi * p.nv + i] = pack8(dx);
          } else {
            store8(p.part_gate + (2ll * c + (first > m0 ? 1 : 0)) * p.D + 8 * i, S[v]);
          }
          float* mp = post + 8 * v * T;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dy[j] = fma2(g[j], S[v][j], f2(mp[2 * j], mp[2 * j + 1]));
            S[v][j] = both(0.f);
          }
          store8(mp, dy);
        }
      }
    }
    fetch(m + p.stages * step, stage);  // every read of the slot is done
    if (++stage == p.stages) stage = 0;
  }

  // add the block's groups; the ring is free once every thread is here
  if (kMode == kSequence)
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (t + v * T < p.nv)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[v][j] = f2(post[8 * v * T + 2 * j], post[8 * v * T + 2 * j + 1]);
  float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* out = (which ? p.part_pre : p.part_post) + (long long)blockIdx.x * p.D;
    if (p.groups > 1) __syncthreads();
    float* to = p.groups > 1 ? sums + group * p.D : out;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (t + v * T < p.nv) store8(to + 8 * (t + v * T), which ? Ppre[v] : S[v]);
    if (p.groups == 1) continue;
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
      float f = 0.f;
      for (int k = 0; k < p.groups; ++k) f += sums[k * p.D + d];
      out[d] = f;
    }
  }
}

// The chunks whose sums make up a gate row that crosses a chunk border: job j's
// gate row, or false if it has none.  Gate row j if there are fewer gate rows than
// chunks, else the one that crosses the border after chunk j as its first.
struct GateChunks {
  long long gi, first;  // the gate row, its first chunk
  int n;
  bool odd;  // the first chunk's slot (the later chunks' are even)
};
__device__ __forceinline__ bool gate_chunks(const NormParams& p, int j, int by_gate, GateChunks* g) {
  g->gi = by_gate ? j : (long long)(j + 1) * p.chunk_rows / p.rows_per_gate;
  const long long first = g->gi * p.rows_per_gate, last = first + p.rows_per_gate - 1;
  g->first = first / p.chunk_rows;
  if (last / p.chunk_rows == g->first || (!by_gate && g->first != j)) return false;
  g->n = (int)(last / p.chunk_rows - g->first) + 1;
  g->odd = first > g->first * p.chunk_rows;
  return true;
}

// Joins the blocks' sums, 128 columns a block: warp w adds rows w, w + 16, ...,
// four columns a lane and all of its rows' loads in flight at once, and the
// sixteen sums are added in order.  blockIdx.y: 0 dw_pre, 1 dw_post (and dgate
// when there is one gate row), from 2 on the gate rows that cross a chunk border.
// Those that at most kJoinWarps chunks share (warp_each) take a warp each, which
// adds the chunks' sums in order (127 gate rows that two chunks share, 8192
// columns: a block each 88 us, a warp 13.5).
constexpr int kJoinWarps = 16, kJoinCols = 128;
__global__ void __launch_bounds__(32 * kJoinWarps)
    norm_join_kernel(const NormParams p, int many_gates, int by_gate, int gate_jobs, int warp_each) {
  __shared__ float part[kJoinWarps][kJoinCols];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * kJoinCols + 4 * lane;
  const int job = blockIdx.y;
  griddep_launch_dependents();
  griddep_wait();
  GateChunks g;
  if (job >= 2 && warp_each) {
    const int j = (job - 2) * kJoinWarps + warp;
    if (j >= gate_jobs || col >= p.D || !gate_chunks(p, j, by_gate, &g)) return;
    const float* src = p.part_gate + 2 * g.first * p.D + col;
    F2 lo = both(0.f), hi = lo;
#pragma unroll 4
    for (int k = 0; k < g.n; ++k) {
      const uint4 v = load_v4_stream(src + 2ll * k * p.D + (g.odd && k == 0 ? p.D : 0));
      lo = lo + f2(__uint_as_float(v.x), __uint_as_float(v.y));
      hi = hi + f2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    const uint2 w = load_v2_stream(reinterpret_cast<const uint16_t*>(p.w_post) + col);
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.dgate) + g.gi * p.D + col) =
        make_uint2(to_bf16x2(both(p.scale) * from_bf16x2(w.x) * lo), to_bf16x2(both(p.scale) * from_bf16x2(w.y) * hi));
    return;
  }
  const float* src;
  int n = p.blocks;  // rows of src to add, `step` apart
  long long step = p.D, gi = 0;
  bool odd = false;
  if (job == 0) {
    src = p.part_pre;
  } else if (job == 1) {
    src = p.part_post;
  } else {
    if (!gate_chunks(p, job - 2, by_gate, &g)) return;
    gi = g.gi;
    n = g.n;
    src = p.part_gate + 2 * g.first * p.D;
    step = 2ll * p.D;
    odd = g.odd;
  }
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = (kBlocks + kJoinWarps - 1) / kJoinWarps;
  if (col < p.D)
    for (int k0 = warp; k0 < n; k0 += kJoinWarps * kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int k = k0 + kJoinWarps * i;
        if (k < n) v[i] = load_v4_stream(src + k * step + (odd && k == 0 ? p.D : 0) + col);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (k0 + kJoinWarps * i < n) {
          s.x += __uint_as_float(v[i].x);
          s.y += __uint_as_float(v[i].y);
          s.z += __uint_as_float(v[i].z);
          s.w += __uint_as_float(v[i].w);
        }
    }
  *reinterpret_cast<float4*>(&part[warp][4 * lane]) = s;
  __syncthreads();
  const int c = blockIdx.x * kJoinCols + (int)threadIdx.x;
  if (threadIdx.x >= kJoinCols || c >= p.D) return;
  float f = part[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) f += part[w][threadIdx.x];
  auto bf = [](const uint4* base, long long k) {
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[k] << 16);
  };
  auto put = [](uint4* base, long long k, float v) {
    reinterpret_cast<uint16_t*>(base)[k] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xffffu);
  };
  if (job == 0) {
    put(p.dw_pre, c, f);
  } else if (job == 1 && many_gates) {
    put(p.dw_post, c, p.scale * f);
  } else if (job == 1) {
    put(p.dw_post, c, p.gate ? p.scale * bf(p.gate, c) * f : p.scale * f);
    if (p.gate) put(p.dgate, c, p.scale * bf(p.w_post, c) * f);
  } else {
    put(p.dgate, gi * p.D + c, p.scale * bf(p.w_post, c) * f);
  }
}

int check(const gemm_rs_norm_desc* d) {
  if (!d || d->gate_rows < 0 || !(d->eps >= 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->scale))
    return GEMM_RS_ERR_INVALID_ARG;
  if (d->M < 0 || d->D <= 0 || d->D % 8 || d->D > GEMM_RS_NORM_MAX_D || d->M > (1ll << 34) / d->D)
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  if (d->gate_rows > 0 && (d->M % d->gate_rows || (d->M > 0 && d->gate_rows > d->M)))
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  return GEMM_RS_OK;
}

GateMode mode_of(const gemm_rs_norm_desc* d) {
  return d->gate_rows <= 1 ? kSingle : d->gate_rows == d->M ? kElement : kSequence;
}

// How the backward pass cuts the rows: a function of the sizes alone.
struct Split {
  Shape shape;
  long long chunk_rows;
  int chunks, blocks;
};
Split split_of(const gemm_rs_norm_desc* d) {
  Split s;
  const GateMode mode = mode_of(d);
  s.shape = shape_of((int)(d->D / 8), mode == kSingle ? 4 : 5, d->M, kBlocks, kBackwardSmem, mode == kSequence ? 32 : 0,
                     mode);
  const long long lanes = (long long)kBlocks * s.shape.groups;
  s.chunk_rows = (d->M + lanes - 1) / lanes;
  if (s.chunk_rows < 1) s.chunk_rows = 1;
  s.chunks = (int)((d->M + s.chunk_rows - 1) / s.chunk_rows);
  s.blocks = (s.chunks + s.shape.groups - 1) / s.shape.groups;
  return s;
}

NormParams params_of(const gemm_rs_norm_desc* d) {
  NormParams p = {};
  p.M = (uint32_t)d->M;
  p.D = (int)d->D;
  p.nv = (int)(d->D / 8);
  p.rows_per_gate = d->gate_rows > 0 && d->M > 0 ? (uint32_t)(d->M / d->gate_rows) : 1;
  p.scale = d->scale;
  p.eps = d->eps;
  p.inv_d = 1.f / (float)d->D;
  p.least = 0x1p-124f * (float)d->D;
  p.least_eps = p.least - d->eps * (float)d->D;
  return p;
}

void set_shape(NormParams* p, const Shape& s) {
  p->warps = s.warps;
  p->groups = s.groups;
  p->stages = s.stages;
}

template <auto Kernel>
int launch(const NormParams& p, int grid, int threads, int smem, cudaStream_t st) {
  static SmemAllowed allowed;
  if (!allowed.set(Kernel, kMaxSmem)) return GEMM_RS_ERR_CUDA;
  return launch_overlapped(Kernel, dim3((unsigned)grid), threads, (size_t)smem, st, p);
}

template <int V>
int launch_forward(const NormParams& p, bool gate_ring, int grid, int smem, cudaStream_t st) {
  const int threads = 32 * p.warps * p.groups;
  return gate_ring ? launch<norm_forward_kernel<V, true>>(p, grid, threads, smem, st)
                    : launch<norm_forward_kernel<V, false>>(p, grid, threads, smem, st);
}
template <int V>
int launch_backward(const NormParams& p, GateMode mode, int smem, cudaStream_t st) {
  const int threads = 32 * p.warps * p.groups;
  if (mode == kSingle) return launch<norm_backward_kernel<V, kSingle>>(p, p.blocks, threads, smem, st);
  if (mode == kSequence) return launch<norm_backward_kernel<V, kSequence>>(p, p.blocks, threads, smem, st);
  return launch<norm_backward_kernel<V, kElement>>(p, p.blocks, threads, smem, st);
}

const uint4* in(const void* p) { return static_cast<const uint4*>(p); }
uint4* outp(void* p) { return static_cast<uint4*>(p); }

}  // namespace

extern "C" int gemm_rs_norm_forward(const gemm_rs_norm_desc* d, const void* x, const void* y,
                                    const void* gate, const void* w_post, const void* w_pre, void* r,
                                    void* h, void* stats, void* stream) {
  int rc = check(d);
  if (rc) return rc;
  if ((d->gate_rows > 0) != (gate != nullptr)) return GEMM_RS_ERR_INVALID_ARG;
  if (d->M == 0) return GEMM_RS_OK;
  if (!x || !y || !w_post || !w_pre || !r || !h) return GEMM_RS_ERR_INVALID_ARG;
  for (const void* q : {x, y, gate, w_post, w_pre, (const void*)r, (const void*)h, (const void*)stats})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  NormParams p = params_of(d);
  p.x = in(x); p.y = in(y); p.gate = in(gate); p.w_post = in(w_post); p.w_pre = in(w_pre);
  p.r = outp(r); p.h = outp(h); p.stats = static_cast<float*>(stats);
  // Where the gate's row comes from.  In registers it costs a stall of its group
  // wherever the next gate row begins, and consecutive rows for each group; through
  // the ring every row asks L2 for it, which all SMs do for the same lines.  That
  // pays where gate rows serve under 8 rows, and where rows are whole 128-byte
  // lines, not short, and there are several gate rows (2048 x 8192 with 4 27.2 ->
  // 25.2 us, with 128 28.1 -> 25.3; 65536 x 1024 with 4 99.2 -> 92.5; but 20000 x 1000
  // 31.9 -> 63.9, 131072 x 512 97.4 -> 102.8), or one or none but more traffic than L2
  // holds (8192 x 8192 94.2 -> 83.3; 2048 x 8192 24.4 -> 25.1): the ring's copies then
  // pace the reads against the writes.
  const bool lines = p.nv % 8 == 0 && p.nv >= 128;
  const bool gate_ring = d->gate_rows > 1 ? lines || p.rows_per_gate < 8 : lines && d->M * p.nv >= (1 << 22);
  const int arrays = gate_ring ? 3 : 2;
  Shape s = shape_of(p.nv, arrays, d->M, 2 * sms, kMaxSmem / 2, 16);
  const int per_sm = forward_blocks(s.v);
  if (per_sm == 1) s = shape_of(p.nv, arrays, d->M, sms, kMaxSmem, 16);
  set_shape(&p, s);
  const long long lanes = (long long)per_sm * sms * s.groups;
  p.chunk_rows = (uint32_t)((d->M + lanes - 1) / lanes);
  const long long chunks = (d->M + p.chunk_rows - 1) / p.chunk_rows;
  const int grid = (int)((chunks + s.groups - 1) / s.groups);
  p.step = d->gate_rows > 1 && !gate_ring ? 1 : (uint32_t)(grid * s.groups);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (s.v) {
    case 1: return launch_forward<1>(p, gate_ring, grid, s.smem, st);
    case 2: return launch_forward<2>(p, gate_ring, grid, s.smem, st);
    case 3: return launch_forward<3>(p, gate_ring, grid, s.smem, st);
    default: return launch_forward<4>(p, gate_ring, grid, s.smem, st);
  }
}

extern "C" int gemm_rs_norm_workspace(const gemm_rs_norm_desc* d, size_t* bytes) {
  const int rc = check(d);
  if (rc) return rc;
  if (!bytes) return GEMM_RS_ERR_INVALID_ARG;
  // the blocks' sums for dw_pre and dw_post, and two gate slots a chunk
  const Split sp = split_of(d);
  const size_t rows = 2 * (size_t)sp.blocks + (mode_of(d) == kSequence ? 2 * (size_t)sp.chunks : 0);
  *bytes = (rows > 0 ? rows : 1) * (size_t)d->D * sizeof(float);
  return GEMM_RS_OK;
}

extern "C" int gemm_rs_norm_backward(const gemm_rs_norm_desc* d, const void* dr, const void* dh,
                                     const void* x, const void* y, const void* gate,
                                     const void* w_post, const void* w_pre, const void* stats,
                                     void* dx, void* dy, void* dgate, void* dw_post, void* dw_pre,
                                     void* workspace, void* stream) {
  int rc = check(d);
  if (rc) return rc;
  if ((d->gate_rows > 0) != (gate != nullptr) || (d->gate_rows > 0) != (dgate != nullptr))
    return GEMM_RS_ERR_INVALID_ARG;
  if (!w_post || !w_pre || !dw_post || !dw_pre) return GEMM_RS_ERR_INVALID_ARG;
  if (d->M > 0 && (!dr || !dh || !x || !y || !stats || !dx || !dy)) return GEMM_RS_ERR_INVALID_ARG;
  if (!workspace) return GEMM_RS_ERR_WORKSPACE;
  for (const void* q : {dr, dh, x, y, gate, w_post, w_pre, stats, (const void*)dx, (const void*)dy,
                        (const void*)dgate, (const void*)dw_post, (const void*)dw_pre,
                        (const void*)workspace})
    if (misaligned16(q)) return GEMM_RS_ERR_MISALIGNED;
  int sms = 0;
  rc = current_device_sms(&sms);
  if (rc) return rc;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->M == 0) {
    if (cudaMemsetAsync(dw_post, 0, d->D * 2, st) != cudaSuccess ||
        cudaMemsetAsync(dw_pre, 0, d->D * 2, st) != cudaSuccess ||
        (dgate && cudaMemsetAsync(dgate, 0, d->gate_rows * d->D * 2, st) != cudaSuccess)) {
      cudaGetLastError();
      return GEMM_RS_ERR_CUDA;
    }
    return GEMM_RS_OK;
  }
  NormParams p = params_of(d);
  const Split sp = split_of(d);
  p.x = in(x); p.y = in(y); p.gate = in(gate); p.w_post = in(w_post); p.w_pre = in(w_pre);
  p.dr = in(dr); p.dh = in(dh);
  p.stats = static_cast<float*>(const_cast<void*>(stats));
  p.dx = outp(dx); p.dy = outp(dy); p.dgate = outp(dgate); p.dw_post = outp(dw_post); p.dw_pre = outp(dw_pre);
  p.chunk_rows = (uint32_t)sp.chunk_rows;
  p.chunks = sp.chunks;
  p.blocks = sp.blocks;
  p.step = mode_of(d) == kSequence ? 1 : (uint32_t)(sp.blocks * sp.shape.groups);
  set_shape(&p, sp.shape);
  const GateMode mode = mode_of(d);
  const long long plane = (long long)sp.blocks * d->D;
  p.part_pre = static_cast<float*>(workspace);
  p.part_post = p.part_pre + plane;
  p.part_gate = p.part_post + plane;
  switch (sp.shape.v) {
    case 1: rc = launch_backward<1>(p, mode, sp.shape.smem, st); break;
    case 2: rc = launch_backward<2>(p, mode, sp.shape.smem, st); break;
    case 3: rc = launch_backward<3>(p, mode, sp.shape.smem, st); break;
    default: rc = launch_backward<4>(p, mode, sp.shape.smem, st); break;
  }
  if (rc) return rc;
  const int many_gates = mode != kSingle, by_gate = d->gate_rows < sp.chunks;
  const int crossing = (int)(mode != kSequence ? 0 : by_gate ? d->gate_rows : sp.chunks - 1);
  const int warp_each = p.rows_per_gate / sp.chunk_rows + 2 <= kJoinWarps;  // chunks of a gate row, at most
  return launch_overlapped(norm_join_kernel,
                           dim3((unsigned)((p.D + kJoinCols - 1) / kJoinCols),
                                (unsigned)(2 + (warp_each ? (crossing + kJoinWarps - 1) / kJoinWarps : crossing))),
                           32 * kJoinWarps, 0, st, p, many_gates, by_gate, crossing, warp_each);
}
