// The norms before and after a block, fused with the block's gate and the residual scale, and
// their gradients.  With rms(v) = rstd v, rstd = 1 / sqrt(mean(v^2) + eps), w' = w + weight_offset:
//   before  n   = rms(x) w'
//   after   out = a x + b g rms(y) w'     (x the residual stream, y the block's output, g the gate:
//                                          none, per channel, per token or per element)
//           n'  = rms(out) w_next'        optionally, the next block's norm of the stored stream
// Gradients (xh = rstd x):  dx of a norm = rstd (d - xh mean(d xh)) with d = dn w',  dw = sum_t dn xh.
// Rows are read once and stay in registers between the row sums and their use, so every call moves
// the bytes of its inputs and outputs once and is bound by HBM; weights and gates of a channel stay
// in registers over the rows that a thread takes.  A group of threads takes a row (one or two units
// of eight elements per thread), a CTA several groups, and a group's next row is loaded before the
// current one's sums, whose barriers it would otherwise wait behind.  Sums are fp32 in a fixed
// order: a row's by shuffles and one array per group, a column's in registers over the group's
// rows, then over the CTA's groups, written per CTA and summed by a second kernel (no atomics).
#include <algorithm>

#include "row_units.cuh"

namespace moe {
namespace {

struct NormArgs {
  int64_t T;
  int units;                   // H / 8
  float inv_h, eps, w_off, a, b;
  int gate_kind;
  const void *x, *y, *dn, *dout, *dres;
  const float *w, *w_next;
  const void* gate;
  const float *rstd_in, *rstd_next_in;
  void *out, *n, *dx, *dy, *dgate;
  float *rstd, *rstd_next;
  float* part;                 // [sums][grid][H] column sums of each CTA
};

// This thread's place: rows are taken by groups of blockDim.x threads, threadIdx.y is the group.
// Units of a row: threadIdx.x, threadIdx.x + blockDim.x.
struct Place {
  int64_t row, stride;
  __device__ __forceinline__ Place()
      : row(static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y), stride(static_cast<int64_t>(gridDim.x) * blockDim.y) {}
};

// Sums of N values over the group, the same bits in every thread of it.  `slot` alternates between
// calls, so one barrier per call is enough.
constexpr int kMaxWarps = 32;
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int& slot) {
  __shared__ __align__(16) float s_sum[2][N][kMaxWarps];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int first = threadIdx.y * warps, warp = first + (threadIdx.x >> 5);   // groups of more than one warp have 2 or a multiple of 4
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s_sum[slot][i][warp] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float* p = &s_sum[slot][i][first];
    float t = 0.0f;
    if (warps == 2) {
      t = p[0] + p[1];
    } else {
      for (int w = 0; w < warps; w += 4) {
        const float4 q = *reinterpret_cast<const float4*>(p + w);
        t += (q.x + q.y) + (q.z + q.w);
      }
    }
    v[i] = t;
  }
  slot ^= 1;
}

__device__ __forceinline__ void load_vec(const float* p, int u, float add, float (&f)[8]) {
  Unit8<float> q;
  q.load(p, u);
  q.get(f);
#pragma unroll
  for (int c = 0; c < 8; ++c) f[c] += add;
}

#define UNIT(i) (static_cast<int>(threadIdx.x) + (i) * static_cast<int>(blockDim.x))
#define EACH_UNIT(i) _Pragma("unroll") for (int i = 0; i < U; ++i) if (UNIT(i) < a.units)
#define EACH(c) _Pragma("unroll") for (int c = 0; c < 8; ++c)

template <typename R, int U, int kMaxThreads, int kPerSm>
__global__ void __launch_bounds__(kMaxThreads, kPerSm) norm_before_kernel(NormArgs a) {
  float w[U][8];
  Unit8<R> qx[U];
  int slot = 0;
  const Place at;
  pdl_wait();
  if (at.row < a.T) EACH_UNIT(i) qx[i].load(a.x, at.row * a.units + UNIT(i));
  EACH_UNIT(i) load_vec(a.w, UNIT(i), a.w_off, w[i]);
  for (int64_t t = at.row; t < a.T; t += at.stride) {
    float x[U][8], sum[1] = {0.0f};
    EACH_UNIT(i) {
      qx[i].get(x[i]);
      if (t + at.stride < a.T) qx[i].load(a.x, (t + at.stride) * a.units + UNIT(i));
      EACH(c) sum[0] = fmaf(x[i][c], x[i][c], sum[0]);
    }
    group_sum(sum, slot);
    const float rstd = 1.0f / sqrtf(sum[0] * a.inv_h + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[t] = rstd;
    EACH_UNIT(i) {
      EACH(c) x[i][c] = x[i][c] * rstd * w[i][c];
      Unit8<uint16_t> q;
      q.set(x[i]);
      q.store(a.n, t * a.units + UNIT(i));
    }
  }
}

// One gate value per element of unit u of row t.
__device__ __forceinline__ void gate_of(const NormArgs& a, int64_t t, int u, const float (&gc)[8], float gt, float (&g)[8]) {
  if (a.gate_kind == MOE_GATE_ELEMENT) {
    Unit8<uint16_t> q;
    q.load(a.gate, t * a.units + u);
    q.get(g);
  } else {
    EACH(c) g[c] = a.gate_kind == MOE_GATE_CHANNEL ? gc[c] : gt;
  }
}

template <typename R, typename Y, int U, int kMaxThreads, int kPerSm, bool kNext>
__global__ void __launch_bounds__(kMaxThreads, kPerSm) norm_after_kernel(NormArgs a) {
  float w[U][8], gc[U][8], wn[U][8];
  Unit8<Y> qy[U];
  Unit8<R> qx[U];
  int slot = 0;
  const Place at;
  auto load_row = [&](int64_t t) {
    EACH_UNIT(i) {
      qy[i].load(a.y, t * a.units + UNIT(i));
      qx[i].load(a.x, t * a.units + UNIT(i));
    }
  };
  pdl_wait();
  if (at.row < a.T) load_row(at.row);
  EACH_UNIT(i) {
    load_vec(a.w, UNIT(i), a.w_off, w[i]);
    if (kNext) load_vec(a.w_next, UNIT(i), a.w_off, wn[i]);
    if (a.gate_kind == MOE_GATE_CHANNEL) load_vec(static_cast<const float*>(a.gate), UNIT(i), 0.0f, gc[i]);
  }
  for (int64_t t = at.row; t < a.T; t += at.stride) {
    float y[U][8], sum[1] = {0.0f};
    Unit8<R> x[U];
    EACH_UNIT(i) {
      qy[i].get(y[i]);
      x[i] = qx[i];
      EACH(c) sum[0] = fmaf(y[i][c], y[i][c], sum[0]);
    }
    if (t + at.stride < a.T) load_row(t + at.stride);
    group_sum(sum, slot);
    const float rstd = 1.0f / sqrtf(sum[0] * a.inv_h + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[t] = rstd;
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? __ldg(static_cast<const float*>(a.gate) + t) : 1.0f;
    sum[0] = 0.0f;
    EACH_UNIT(i) {
      float xv[8], g[8];
      x[i].get(xv);
      gate_of(a, t, UNIT(i), gc[i], gt, g);
      EACH(c) y[i][c] = a.a * xv[c] + a.b * g[c] * (y[i][c] * rstd * w[i][c]);
      Unit8<R> q;
      q.set(y[i]);
      q.store(a.out, t * a.units + UNIT(i));
      if (kNext) {
        q.get(y[i]);   // the stored stream, as a separate norm would read it
        EACH(c) sum[0] = fmaf(y[i][c], y[i][c], sum[0]);
      }
    }
    if (kNext) {
      group_sum(sum, slot);
      const float rn = 1.0f / sqrtf(sum[0] * a.inv_h + a.eps);
      if (threadIdx.x == 0 && a.rstd_next) a.rstd_next[t] = rn;
      EACH_UNIT(i) {
        EACH(c) y[i][c] = y[i][c] * rn * wn[i][c];
        Unit8<uint16_t> q;
        q.set(y[i]);
        q.store(a.n, t * a.units + UNIT(i));
      }
    }
  }
}

// Adds the groups' column sums in group order (through shared memory) and writes the CTA's row.
template <int U>
__device__ __forceinline__ void write_part(const NormArgs& a, int which, float (&s)[U][8], float* s_cols) {
  float4* mine = reinterpret_cast<float4*>(s_cols) + ((threadIdx.y - 1) * blockDim.x + threadIdx.x) * 2;
  if (blockDim.y > 1) {                 // one unit per thread then
    __syncthreads();
    if (threadIdx.y > 0) {
      mine[0] = make_float4(s[0][0], s[0][1], s[0][2], s[0][3]);
      mine[1] = make_float4(s[0][4], s[0][5], s[0][6], s[0][7]);
    }
    __syncthreads();
  }
  if (threadIdx.y > 0) return;
  for (int g = 1; g < static_cast<int>(blockDim.y); ++g) {
    const float4* q = reinterpret_cast<const float4*>(s_cols) + ((g - 1) * blockDim.x + threadIdx.x) * 2;
    const float4 lo = q[0], hi = q[1];
    s[0][0] += lo.x; s[0][1] += lo.y; s[0][2] += lo.z; s[0][3] += lo.w;
    s[0][4] += hi.x; s[0][5] += hi.y; s[0][6] += hi.z; s[0][7] += hi.w;
  }
  float* row = a.part + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * a.units * 8;
  EACH_UNIT(i) {
    Unit8<float> q;
    q.set(s[i]);
    q.store(row, UNIT(i));
  }
}

constexpr int kGradThreads = 512;       // threads of a gradient's CTA, groups of fewer than that together

template <typename R, int U, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_before_grad_kernel(NormArgs a) {
  __shared__ __align__(16) float s_cols[kGradThreads * 8];
  float w[U][8], dw[U][8];
  Unit8<R> qx[U], qr[U];
  Unit8<uint16_t> qd[U];
  float q_rstd = 0.0f;
  int slot = 0;
  const Place at;
  auto load_row = [&](int64_t t) {
    EACH_UNIT(i) {
      qx[i].load(a.x, t * a.units + UNIT(i));
      qd[i].load(a.dn, t * a.units + UNIT(i));
      if (a.dres) qr[i].load(a.dres, t * a.units + UNIT(i));
    }
    q_rstd = __ldg(a.rstd_in + t);
  };
  pdl_wait();
  if (at.row < a.T) load_row(at.row);
  EACH_UNIT(i) {
    load_vec(a.w, UNIT(i), a.w_off, w[i]);
    EACH(c) dw[i][c] = 0.0f;
  }
  for (int64_t t = at.row; t < a.T; t += at.stride) {
    const float rstd = q_rstd;
    float xh[U][8], d[U][8], dot[1] = {0.0f};
    Unit8<R> res[U];
    EACH_UNIT(i) {
      qx[i].get(xh[i]);
      qd[i].get(d[i]);
      res[i] = qr[i];
      EACH(c) {
        xh[i][c] *= rstd;
        dw[i][c] = fmaf(d[i][c], xh[i][c], dw[i][c]);
        d[i][c] *= w[i][c];
        dot[0] = fmaf(d[i][c], xh[i][c], dot[0]);
      }
    }
    if (t + at.stride < a.T) load_row(t + at.stride);
    group_sum(dot, slot);
    const float m = dot[0] * a.inv_h;
    EACH_UNIT(i) {
      float r[8];
      if (a.dres) res[i].get(r);
      else EACH(c) r[c] = 0.0f;
      EACH(c) r[c] += rstd * (d[i][c] - xh[i][c] * m);
      Unit8<R> q;
      q.set(r);
      q.store(a.dx, t * a.units + UNIT(i));
    }
  }
  write_part<U>(a, 0, dw, s_cols);
}

// Gradient of `after`: with d = dout (+ the gradient that comes through the next norm, whose input
// is the stored out),  dx = a d,  dgate = b d rms(y) w',  and the norm's gradient of b d g.
template <typename R, typename Y, int U, int kMaxThreads, bool kNext>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_after_grad_kernel(NormArgs a) {
  __shared__ __align__(16) float s_cols[kGradThreads * 8];
  float dw[U][8], dwn[U][8], dg[U][8];
  Unit8<R> qd[U], qo[U];
  Unit8<Y> qy[U];
  Unit8<uint16_t> qn[U];
  float q_rstd = 0.0f, q_rn = 0.0f;
  int slot = 0;
  const Place at;
  auto load_row = [&](int64_t t) {
    EACH_UNIT(i) {
      const int64_t u = t * a.units + UNIT(i);
      qd[i].load(a.dout, u);
      qy[i].load(a.y, u);
      if (kNext) {
        qo[i].load(a.x, u);
        qn[i].load(a.dn, u);
      }
    }
    q_rstd = __ldg(a.rstd_in + t);
    if (kNext) q_rn = __ldg(a.rstd_next_in + t);
  };
  pdl_wait();
  if (at.row < a.T) load_row(at.row);
  EACH_UNIT(i) {
    EACH(c) {
      dw[i][c] = 0.0f;
      dwn[i][c] = 0.0f;
      dg[i][c] = 0.0f;
    }
  }
  for (int64_t t = at.row; t < a.T; t += at.stride) {
    const float rstd = q_rstd, rn = q_rn;
    float d[U][8], yh[U][8], oh[U][8], e[U][8], dot[1] = {0.0f};
    EACH_UNIT(i) {
      qd[i].get(d[i]);
      qy[i].get(yh[i]);
      if (kNext) {
        float wn[8];
        load_vec(a.w_next, UNIT(i), a.w_off, wn);
        qo[i].get(oh[i]);
        qn[i].get(e[i]);
        EACH(c) {
          oh[i][c] *= rn;
          dwn[i][c] = fmaf(e[i][c], oh[i][c], dwn[i][c]);
          e[i][c] *= wn[c];
          dot[0] = fmaf(e[i][c], oh[i][c], dot[0]);
        }
      }
    }
    if (t + at.stride < a.T) load_row(t + at.stride);
    if (kNext) {
      group_sum(dot, slot);
      const float m = dot[0] * a.inv_h;
      EACH_UNIT(i) EACH(c) d[i][c] += rn * (e[i][c] - oh[i][c] * m);
    }
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? __ldg(static_cast<const float*>(a.gate) + t) : 1.0f;
    float sums[2] = {0.0f, 0.0f};
    EACH_UNIT(i) {
      float r[8], g[8], w[8];
      EACH(c) r[c] = a.a * d[i][c];
      Unit8<R> q;
      q.set(r);
      q.store(a.dx, t * a.units + UNIT(i));
      load_vec(a.w, UNIT(i), a.w_off, w);
      float gc[8];
      if (a.gate_kind == MOE_GATE_CHANNEL) load_vec(static_cast<const float*>(a.gate), UNIT(i), 0.0f, gc);
      gate_of(a, t, UNIT(i), gc, gt, g);
      EACH(c) {
        yh[i][c] *= rstd;
        d[i][c] *= a.b;
        r[c] = d[i][c] * (yh[i][c] * w[c]);   // the gate's gradient
        sums[1] += r[c];
        dg[i][c] += r[c];
        d[i][c] *= g[c];
        dw[i][c] = fmaf(d[i][c], yh[i][c], dw[i][c]);
        d[i][c] *= w[c];
        sums[0] = fmaf(d[i][c], yh[i][c], sums[0]);
      }
      if (a.gate_kind == MOE_GATE_ELEMENT) {
        Unit8<uint16_t> qg;
        qg.set(r);
        qg.store(a.dgate, t * a.units + UNIT(i));
      }
    }
    group_sum(sums, slot);
    if (a.gate_kind == MOE_GATE_TOKEN && threadIdx.x == 0) static_cast<float*>(a.dgate)[t] = sums[1];
    const float m = sums[0] * a.inv_h;
    EACH_UNIT(i) {
      EACH(c) d[i][c] = rstd * (d[i][c] - yh[i][c] * m);
      Unit8<Y> q;
      q.set(d[i]);
      q.store(a.dy, t * a.units + UNIT(i));
    }
  }
  write_part<U>(a, 0, dw, s_cols);
  if (kNext) write_part<U>(a, 1, dwn, s_cols);
  if (a.gate_kind == MOE_GATE_CHANNEL) write_part<U>(a, 2, dg, s_cols);
}

// Column sums: part [3][rows][H] -> one vector each (NULL: skipped).  32 columns per CTA, 32
// threads per column, each over every 32nd row; then one sum over the 32 in a fixed order.
__global__ void __launch_bounds__(1024) norm_columns_kernel(const float* __restrict__ part, int rows, int H, float* o0,
                                                            float* o1, float* o2) {
  __shared__ float s_sum[32][33];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  pdl_wait();
  if (!out) return;
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float v = 0.0f;
  if (col < H)
    for (int i = r; i < rows; i += 32) v += part[(static_cast<int64_t>(blockIdx.y) * rows + i) * H + col];
  s_sum[c][r] = v;
  __syncthreads();
  v = s_sum[r][c];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (c == 0 && blockIdx.x * 32 + r < H) out[blockIdx.x * 32 + r] = v;
}

constexpr int kOneUnit = 512;    // rows of up to this many units: one unit per thread, else two
constexpr int kForwardThreads = 256;
constexpr int kMaxSms = 160;     // the workspace holds the column sums of this many CTAs

// Threads of a row: 32, 64 or a multiple of 128.
int row_threads(int units) {
  const int per = units <= kOneUnit ? units : (units + 1) / 2;
  return per <= 32 ? 32 : per <= 64 ? 64 : (per + 127) / 128 * 128;
}

// A launch of as many CTAs as are resident (`per_sm`), with a row per group at least.
struct NormLaunch {
  dim3 grid, block;
};
NormLaunch launch_of(int64_t T, int units, int threads, int per_sm, int n_sm) {
  const int x = row_threads(units), y = std::max(1, threads / x);
  const int64_t most = static_cast<int64_t>(n_sm) * std::max(1, per_sm * threads / (x * y));
  NormLaunch l;
  l.block = dim3(x, y);
  l.grid = dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min((T + y - 1) / y, most))));
  return l;
}
NormLaunch forward_launch(int64_t T, int units, int n_sm) { return launch_of(T, units, kForwardThreads, 4, n_sm); }
NormLaunch grad_launch(int64_t T, int units, int n_sm) {
  return launch_of(T, units, kGradThreads, 1, std::min(n_sm, kMaxSms));
}

NormArgs args_of(const moe_norm_t& s) {
  NormArgs a = {};
  a.T = s.T;
  a.units = s.H / 8;
  a.inv_h = 1.0f / static_cast<float>(s.H);
  a.eps = s.eps;
  a.w_off = s.weight_offset;
  a.a = s.residual_scale;
  a.b = s.branch_scale;
  a.gate_kind = s.gate;
  return a;
}

// Launch bounds: up to 256 threads four CTAs per SM (64 registers), else one CTA; two units per
// thread in up to 512 threads (128 registers), and in 1024 (64, some spilled) above 8192 columns.
#define PICK_UNITS(small, one, two, more) \
  (s.H / 8 <= 256 ? small : s.H / 8 <= kOneUnit ? one : s.H / 8 <= 2 * kOneUnit ? two : more)
#define PICK_BEFORE(K, R) PICK_UNITS((K<R, 1, 256, 4>), (K<R, 1, 512, 1>), (K<R, 2, 512, 1>), (K<R, 2, 1024, 1>))
#define PICK_GRAD(K, R) PICK_UNITS((K<R, 1, 512>), (K<R, 1, 512>), (K<R, 2, 512>), (K<R, 2, 1024>))
#define PICK_AFTER(K, R, Y, next) \
  PICK_UNITS((K<R, Y, 1, 256, 4, next>), (K<R, Y, 1, 512, 1, next>), (K<R, Y, 2, 512, 1, next>), (K<R, Y, 2, 1024, 1, next>))
#define PICK_AFTER_GRAD(K, R, Y, next) \
  PICK_UNITS((K<R, Y, 1, 512, next>), (K<R, Y, 1, 512, next>), (K<R, Y, 2, 512, next>), (K<R, Y, 2, 1024, next>))
#define PICK_NEXT(PICK, K, R, Y) (next ? PICK(K, R, Y, true) : PICK(K, R, Y, false))
#define PICK_TYPES(PICK, K)                                                                                          \
  (s.residual_fp32 ? (s.branch_fp32 ? PICK_NEXT(PICK, K, float, float) : PICK_NEXT(PICK, K, float, uint16_t))        \
                   : (s.branch_fp32 ? PICK_NEXT(PICK, K, uint16_t, float) : PICK_NEXT(PICK, K, uint16_t, uint16_t)))

}  // namespace

// CTAs that write column sums, at most (the size of the workspace).
int64_t norm_max_parts(int64_t T, int H) { return grad_launch(T, H / 8, kMaxSms).grid.x; }

cudaError_t launch_norm_before(const moe_norm_t& s, const void* x, const float* w, void* n, float* rstd, cudaStream_t st) {
  int n_sm = 0;
  cudaError_t e = current_sm_count(&n_sm);
  if (e != cudaSuccess) return e;
  NormArgs a = args_of(s);
  a.x = x;
  a.w = w;
  a.n = n;
  a.rstd = rstd;
  auto kern = s.residual_fp32 ? PICK_BEFORE(norm_before_kernel, float) : PICK_BEFORE(norm_before_kernel, uint16_t);
  const NormLaunch l = forward_launch(s.T, a.units, n_sm);
  return launch_pdl(true, kern, l.grid, l.block, 0, st, a);
}

cudaError_t launch_norm_after(const moe_norm_t& s, const void* y, const void* x, const float* w, const void* gate,
                              const float* w_next, void* out, void* n, float* rstd, float* rstd_next, cudaStream_t st) {
  int n_sm = 0;
  cudaError_t e = current_sm_count(&n_sm);
  if (e != cudaSuccess) return e;
  NormArgs a = args_of(s);
  a.y = y;
  a.x = x;
  a.w = w;
  a.gate = gate;
  a.w_next = w_next;
  a.out = out;
  a.n = n;
  a.rstd = rstd;
  a.rstd_next = rstd_next;
  const bool next = w_next != nullptr;
  auto kern = PICK_TYPES(PICK_AFTER, norm_after_kernel);
  const NormLaunch l = forward_launch(s.T, a.units, n_sm);
  return launch_pdl(true, kern, l.grid, l.block, 0, st, a);
}

cudaError_t launch_norm_before_grad(const moe_norm_t& s, const void* dn, const void* x, const float* w, const float* rstd,
                                    const void* dres, void* dx, float* dw, float* part, cudaStream_t st) {
  int n_sm = 0;
  cudaError_t e = current_sm_count(&n_sm);
  if (e != cudaSuccess) return e;
  NormArgs a = args_of(s);
  a.dn = dn;
  a.x = x;
  a.w = w;
  a.rstd_in = rstd;
  a.dres = dres;
  a.dx = dx;
  a.part = part;
  const NormLaunch l = grad_launch(s.T, a.units, n_sm);
  const int grid = static_cast<int>(l.grid.x);
  auto kern = s.residual_fp32 ? PICK_GRAD(norm_before_grad_kernel, float) : PICK_GRAD(norm_before_grad_kernel, uint16_t);
  e = launch_pdl(true, kern, l.grid, l.block, 0, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(true, norm_columns_kernel, dim3((s.H + 31) / 32, 1), dim3(1024), 0, st,
                    static_cast<const float*>(part), grid, s.H, dw, static_cast<float*>(nullptr),
                    static_cast<float*>(nullptr));
}

cudaError_t launch_norm_after_grad(const moe_norm_t& s, const void* dout, const void* dn, const void* y, const void* out,
                                   const float* w, const void* gate, const float* w_next, const float* rstd,
                                   const float* rstd_next, void* dy, void* dx, float* dw, void* dgate, float* dw_next,
                                   float* part, cudaStream_t st) {
  int n_sm = 0;
  cudaError_t e = current_sm_count(&n_sm);
  if (e != cudaSuccess) return e;
  NormArgs a = args_of(s);
  a.dout = dout;
  a.dn = dn;
  a.y = y;
  a.x = out;
  a.w = w;
  a.gate = gate;
  a.w_next = w_next;
  a.rstd_in = rstd;
  a.rstd_next_in = rstd_next;
  a.dy = dy;
  a.dx = dx;
  a.dgate = dgate;
  a.part = part;
  const NormLaunch l = grad_launch(s.T, a.units, n_sm);
  const int grid = static_cast<int>(l.grid.x);
  const bool next = w_next != nullptr;
  auto kern = PICK_TYPES(PICK_AFTER_GRAD, norm_after_grad_kernel);
  e = launch_pdl(true, kern, l.grid, l.block, 0, st, a);
  if (e != cudaSuccess) return e;
  float* dgc = s.gate == MOE_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr;
  return launch_pdl(true, norm_columns_kernel, dim3((s.H + 31) / 32, dgc ? 3 : dw_next ? 2 : 1), dim3(1024), 0, st,
                    static_cast<const float*>(part), grid, s.H, dw, dw_next, dgc);
}

}  // namespace moe
