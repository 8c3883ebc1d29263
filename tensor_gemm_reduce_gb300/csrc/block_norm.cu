// block_norm.cu -- the norms after and before a block, fused with the block's
// gate and residual scale, forward and backward (gemm_rs_norm_* in
// include/gemm_rs_ops.h).
#include <cmath>

#include "ops_common.cuh"

using namespace grs;

namespace {

constexpr int kMaxThreads = 512;
// Row chunks of the backward pass: one per SM of a GB300.  A constant, so that
// the workspace size and the order of the sums do not depend on the device.
constexpr int kChunks = 152;

struct NormParams {
  long long M;
  int D, nv;            // nv = D / 8 vectors of 16 bytes in a row
  long long rows_per_gate;  // M / gate_rows
  float scale, eps, inv_d;
  const uint4 *x, *y, *gate, *w_post, *w_pre;
  uint4 *r, *h;
  float* stats;
  // backward
  const uint4 *dr, *dh;
  uint4 *dx, *dy, *dgate, *dw_post, *dw_pre;
  long long chunk_rows;
  int chunks;
  float *part_s, *part_pre, *part_post, *part_gate;
};

// Threads take whole 16-byte vectors of a row: thread t vectors t, t + T, ...
// (V of them at most).  T is the least number of warps that covers the row
// with V vectors each.
int vectors_per_thread(int nv) { return (nv + kMaxThreads - 1) / kMaxThreads; }
int threads_for(int nv, int v) { return ((nv + v - 1) / v + 31) / 32 * 32; }

// One row at a time: both sums are block-wide, the row stays in registers.
template <int V>
__global__ void __launch_bounds__(kMaxThreads) norm_forward_kernel(const NormParams p) {
  __shared__ float part[2][32];
  const int t = threadIdx.x, T = blockDim.x;
  for (long long m = blockIdx.x; m < p.M; m += gridDim.x) {
    const uint4* xr = p.x + m * p.nv;
    const uint4* yr = p.y + m * p.nv;
    const uint4* gr = p.gate ? p.gate + (m / p.rows_per_gate) * p.nv : nullptr;
    float r[V][8], y[V][8];
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = t + v * T;
      const bool in = i < p.nv;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      unpack8(in ? yr[i] : zero, y[v]);
      unpack8(in ? xr[i] : zero, r[v]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(y[v][j], y[v][j], s[0]);
    }
    block_sum<1>(s, part[0]);
    const float pn = 1.f / sqrtf(fmaf(s[0], p.inv_d, p.eps));
    s[0] = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = t + v * T;
      if (i < p.nv) {
        float w[8], g[8];
        unpack8(__ldg(p.w_post + i), w);
        if (gr) unpack8(__ldg(gr + i), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = y[v][j] * pn * w[j];
          r[v][j] = fmaf(gr ? p.scale * g[j] : p.scale, u, r[v][j]);
          s[0] = fmaf(r[v][j], r[v][j], s[0]);
        }
      }
    }
    block_sum<1>(s, part[1]);
    const float qn = 1.f / sqrtf(fmaf(s[0], p.inv_d, p.eps));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = t + v * T;
      if (i < p.nv) {
        float w[8], h[8];
        unpack8(__ldg(p.w_pre + i), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = r[v][j] * qn * w[j];
        p.r[m * p.nv + i] = pack8(r[v]);
        p.h[m * p.nv + i] = pack8(h);
      }
    }
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
// so one block-wide sum of three values serves both norms.
// Each block owns chunk_rows consecutive rows and its threads own columns, so
// the sums over rows stay in registers: S = sum of t yn over the rows of one
// gate row, which gives both dgate = scale w_post S and that gate row's share
// scale gate S of dw_post; and sum of dh rn = dw_pre.  kMultiGate: several
// gate rows, so dw_post has an accumulator of its own.  A gate row whose rows
// all lie in the chunk is written at once; one that crosses a chunk border
// leaves a partial sum in slot 2 c (its rows begin at the chunk's first row or
// before) or 2 c + 1.
template <int V, bool kMultiGate>
__global__ void __launch_bounds__(kMaxThreads) norm_backward_kernel(const NormParams p) {
  __shared__ float part[2][96];
  const int t = threadIdx.x, T = blockDim.x, c = blockIdx.x;
  const long long m0 = c * p.chunk_rows;
  const long long m1 = m0 + p.chunk_rows < p.M ? m0 + p.chunk_rows : p.M;
  float S[V][8], Ppre[V][8], Ppost[kMultiGate ? V : 1][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      S[v][j] = Ppre[v][j] = 0.f;
      if (kMultiGate) Ppost[v][j] = 0.f;
    }
  for (long long m = m0; m < m1; ++m) {
    const float pn = p.stats[m], qn = p.stats[p.M + m];
    const long long gi = p.gate ? m / p.rows_per_gate : 0;
    const uint4* gr = p.gate ? p.gate + gi * p.nv : nullptr;
    float yn[V][8], rn[V][8], z[V][8];  // z = dr + q a
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = t + v * T;
      if (i < p.nv) {
        float x[8], w[8], g[8], dh[8], dr[8], wq[8];
        unpack8(p.y[m * p.nv + i], yn[v]);
        unpack8(p.x[m * p.nv + i], x);
        unpack8(p.dr[m * p.nv + i], dr);
        unpack8(p.dh[m * p.nv + i], dh);
        unpack8(__ldg(p.w_post + i), w);
        unpack8(__ldg(p.w_pre + i), wq);
        if (gr) unpack8(__ldg(gr + i), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          yn[v][j] *= pn;
          const float br = (gr ? p.scale * g[j] : p.scale) * (yn[v][j] * w[j]);
          rn[v][j] = (x[j] + br) * qn;
          const float a = dh[j] * wq[j];
          z[v][j] = fmaf(qn, a, dr[j]);
          Ppre[v][j] = fmaf(dh[j], rn[v][j], Ppre[v][j]);
          s[0] = fmaf(a, rn[v][j], s[0]);
          s[1] = fmaf(br, z[v][j], s[1]);
          s[2] = fmaf(br, rn[v][j], s[2]);
        }
      }
    }
    block_sum<3>(s, part[m & 1]);
    const float k1 = qn * (s[0] * p.inv_d);                 // q m1
    const float k2 = fmaf(-k1, s[2], s[1]) * p.inv_d * pn;  // p m2
    const bool last = !kMultiGate || m + 1 == m1 || (m + 1) % p.rows_per_gate == 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = t + v * T;
      if (i < p.nv) {
        float w[8], g[8], dx[8], dy[8];
        unpack8(__ldg(p.w_post + i), w);
        if (gr) unpack8(__ldg(gr + i), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float tt = fmaf(-k1, rn[v][j], z[v][j]);
          const float gs = gr ? p.scale * g[j] : p.scale;
          dx[j] = tt;
          S[v][j] = fmaf(tt, yn[v][j], S[v][j]);
          dy[j] = fmaf(pn * (gs * tt), w[j], -k2 * yn[v][j]);
        }
        p.dx[m * p.nv + i] = pack8(dx);
        p.dy[m * p.nv + i] = pack8(dy);
        if (kMultiGate && last) {  // end of a gate row's rows in this chunk
          const long long first = gi * p.rows_per_gate;
          if (first >= m0 && first + p.rows_per_gate <= m1) {
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = p.scale * w[j] * S[v][j];
            p.dgate[gi * p.nv + i] = pack8(o);
          } else {
            float* slot = p.part_gate + (2 * c + (first > m0 ? 1 : 0)) * (long long)p.D + 8 * i;
#pragma unroll
            for (int j = 0; j < 8; ++j) slot[j] = S[v][j];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            Ppost[v][j] = fmaf(p.scale * g[j], S[v][j], Ppost[v][j]);
            S[v][j] = 0.f;
          }
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = t + v * T;
    if (i < p.nv)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const long long at = (long long)c * p.D + 8 * i + j;
        p.part_pre[at] = Ppre[v][j];
        if (kMultiGate)
          p.part_post[at] = Ppost[v][j];
        else
          p.part_s[at] = S[v][j];
      }
  }
}

// Joins the chunks' sums, 32 columns a block: warp w adds chunks w, w + 8, ...
// and the eight sums are added in order.  blockIdx.y: 0 dw_pre, 1 dw_post (and
// dgate when there is one gate row), 2 + b the gate row that crosses the border
// between chunks b and b + 1 first (each crossing row has one first border).
__global__ void __launch_bounds__(256) norm_join_kernel(const NormParams p, int multi) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  const bool in = col < p.D;
  const int job = blockIdx.y;
  const float* src;
  int n = p.chunks;                       // rows of src to add, `step` apart
  long long step = p.D, gi = 0;
  if (job == 0) {
    src = p.part_pre;
  } else if (job == 1) {
    src = multi ? p.part_post : p.part_s;
  } else {
    const int b = job - 2;
    const long long border = (long long)(b + 1) * p.chunk_rows;
    gi = border / p.rows_per_gate;
    const long long first = gi * p.rows_per_gate;
    if (first == border || first / p.chunk_rows != b) return;
    const long long last = first + p.rows_per_gate - 1;
    n = (int)(last / p.chunk_rows) - b + 1;
    src = p.part_gate + 2ll * b * p.D;
    step = 2ll * p.D;
    // chunk b's slot is the odd one when the gate row begins after its first row
    if (first > b * p.chunk_rows) src += p.D;
  }
  float s = 0.f;
  if (in)
    for (int k = warp; k < n; k += 8) {
      long long at = k * step;
      if (job >= 2 && k > 0 && src != p.part_gate + 2ll * (job - 2) * p.D) at -= p.D;
      s += src[at + col];
    }
  part[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || !in) return;
  s = part[0][lane];
#pragma unroll
  for (int w = 1; w < 8; ++w) s += part[w][lane];
  auto bf = [](const uint4* base, long long k) {
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[k] << 16);
  };
  auto put = [](uint4* base, long long k, float f) {
    reinterpret_cast<uint16_t*>(base)[k] = (uint16_t)(pack_bf16x2(f, 0.f) & 0xffffu);
  };
  if (job == 0) {
    put(p.dw_pre, col, s);
  } else if (job == 1 && multi) {
    put(p.dw_post, col, s);
  } else if (job == 1) {
    put(p.dw_post, col, p.gate ? p.scale * bf(p.gate, col) * s : p.scale * s);
    if (p.gate) put(p.dgate, col, p.scale * bf(p.w_post, col) * s);
  } else {
    put(p.dgate, gi * p.D + col, p.scale * bf(p.w_post, col) * s);
  }
}

int check(const gemm_rs_norm_desc* d) {
  if (!d || d->gate_rows < 0 || !(d->eps >= 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->scale))
    return GEMM_RS_ERR_INVALID_ARG;
  if (d->M < 0 || d->M > (1ll << 40) || d->D <= 0 || d->D % 8 || d->D > GEMM_RS_NORM_MAX_D)
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  if (d->gate_rows > 0 && (d->M % d->gate_rows || (d->M > 0 && d->gate_rows > d->M)))
    return GEMM_RS_ERR_UNSUPPORTED_SHAPE;
  return GEMM_RS_OK;
}

struct Split {
  long long chunk_rows;
  int chunks;
};
Split split_of(const gemm_rs_norm_desc* d) {
  Split s;
  s.chunk_rows = (d->M + kChunks - 1) / kChunks;
  if (s.chunk_rows < 1) s.chunk_rows = 1;
  s.chunks = (int)((d->M + s.chunk_rows - 1) / s.chunk_rows);
  return s;
}

NormParams params_of(const gemm_rs_norm_desc* d) {
  NormParams p = {};
  p.M = d->M;
  p.D = (int)d->D;
  p.nv = (int)(d->D / 8);
  p.rows_per_gate = d->gate_rows > 0 && d->M > 0 ? d->M / d->gate_rows : 1;
  p.scale = d->scale;
  p.eps = d->eps;
  p.inv_d = 1.f / (float)d->D;
  return p;
}

template <int V>
void launch_forward(const NormParams& p, int grid, int threads, cudaStream_t st) {
  norm_forward_kernel<V><<<grid, threads, 0, st>>>(p);
}
template <int V>
void launch_backward(const NormParams& p, bool multi, int threads, cudaStream_t st) {
  if (multi)
    norm_backward_kernel<V, true><<<p.chunks, threads, 0, st>>>(p);
  else
    norm_backward_kernel<V, false><<<p.chunks, threads, 0, st>>>(p);
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
  const int v = vectors_per_thread(p.nv), threads = threads_for(p.nv, v);
  const int grid = (int)(p.M < 4ll * sms ? p.M : 4ll * sms);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (v) {
    case 1: launch_forward<1>(p, grid, threads, st); break;
    case 2: launch_forward<2>(p, grid, threads, st); break;
    case 3: launch_forward<3>(p, grid, threads, st); break;
    default: launch_forward<4>(p, grid, threads, st); break;
  }
  return launch_status();
}

extern "C" int gemm_rs_norm_workspace(const gemm_rs_norm_desc* d, size_t* bytes) {
  const int rc = check(d);
  if (rc) return rc;
  if (!bytes) return GEMM_RS_ERR_INVALID_ARG;
  // part_pre, part_s or part_post, and two gate slots a chunk
  const size_t rows = (size_t)split_of(d).chunks * (d->gate_rows > 1 ? 4 : 2);
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
  p.chunk_rows = sp.chunk_rows;
  p.chunks = sp.chunks;
  const bool multi = d->gate_rows > 1;
  float* ws = static_cast<float*>(workspace);
  const long long plane = (long long)sp.chunks * d->D;
  p.part_pre = ws;
  (multi ? p.part_post : p.part_s) = ws + plane;
  p.part_gate = ws + 2 * plane;
  const int v = vectors_per_thread(p.nv), threads = threads_for(p.nv, v);
  switch (v) {
    case 1: launch_backward<1>(p, multi, threads, st); break;
    case 2: launch_backward<2>(p, multi, threads, st); break;
    case 3: launch_backward<3>(p, multi, threads, st); break;
    default: launch_backward<4>(p, multi, threads, st); break;
  }
  rc = launch_status();
  if (rc) return rc;
  const dim3 grid((unsigned)((p.D + 31) / 32), (unsigned)(2 + (multi ? sp.chunks - 1 : 0)));
  norm_join_kernel<<<grid, 256, 0, st>>>(p, multi ? 1 : 0);
  return launch_status();
}
