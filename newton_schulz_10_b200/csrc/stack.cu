// Row kernels of the stack update: momentum (with Nesterov's target), the
// Frobenius norms, the operand cast and the weight update of stacks of
// matrices with strides and 16-bit or fp32 weights and gradients.
//
// All four are bound by HBM. A warp (rows up to 2048) or a block (longer
// rows) walks a row with four elements a lane and several loads in flight;
// the sums of squares are fp64 in a fixed order, so results are
// bit-reproducible. Types of W, G and the copy are read from the table (the
// branch is uniform over the row), so one kernel serves every combination.
#include <type_traits>

#include "common.cuh"
#include "rowio.cuh"
#include "stack.cuh"

namespace muon {

namespace {

constexpr int BLOCK = 256;
constexpr int UNROLL = 4;

struct Row {
  int mat, b, r;  // stack of the launch, matrix of the stack, row of the matrix
};

__device__ __forceinline__ Row find_row(const StackLaunch& L, int task) {
  int lo = 0, hi = L.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.m[mid].row_begin <= task) lo = mid; else hi = mid - 1;
  }
  const int local = task - L.m[lo].row_begin, rows = L.m[lo].rows;
  return Row{lo, local / rows, local % rows};
}

template <int WG>
__device__ __forceinline__ double group_sum(double v, double* scratch) {
  if (WG == 32) return warp_sum(v);
  return block_sum(v, scratch);
}

template <int WG, typename T, bool CAST>
__global__ void __launch_bounds__(BLOCK) stack_momentum(const __grid_constant__ StackLaunch L) {
  __shared__ double scratch[32];
  grid_dependency_wait();
  grid_dependents_launch();
  // the launches that may report come after this one
  if (L.clear && blockIdx.x == 0 && threadIdx.x == 0) *L.status = MUON_OK;
  const int task = blockIdx.x * (BLOCK / WG) + threadIdx.x / WG;
  const int l = threadIdx.x % WG;
  const bool active = task < L.total_rows;
  double ss = 0.0;
  if (active) {
    const Row w = find_row(L, task);
    const StackMat& m = L.m[w.mat];
    float* M = m.M + w.b * m.m_stride + w.r * m.m_ld;
    const void* G = m.G ? row_at(m.G, m.g_type, w.b * m.g_stride + w.r * m.g_ld) : nullptr;
    T* X = CAST ? static_cast<T*>(m.X) + ((int64_t)w.b * m.rows + w.r) * m.ldx : nullptr;
    const float mu = L.mu;
    if (m.vec) {
      const int n4 = m.cols >> 2;
      for (int c0 = l; c0 < n4; c0 += UNROLL * WG) {
        float4 x[UNROLL], g[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          const int c = c0 + u * WG;
          if (c < n4) {
            x[u] = *reinterpret_cast<const float4*>(M + 4 * c);
            if (G) g[u] = load4(G, m.g_type, 4 * c);
          }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          const int c = c0 + u * WG;
          if (c >= n4) break;
          float4 y = x[u];
          if (G) {
            y.x = fmaf(mu, y.x, g[u].x); y.y = fmaf(mu, y.y, g[u].y);
            y.z = fmaf(mu, y.z, g[u].z); y.w = fmaf(mu, y.w, g[u].w);
            *reinterpret_cast<float4*>(M + 4 * c) = y;
            y.x = target(y.x, g[u].x, mu, L.nesterov); y.y = target(y.y, g[u].y, mu, L.nesterov);
            y.z = target(y.z, g[u].z, mu, L.nesterov); y.w = target(y.w, g[u].w, mu, L.nesterov);
          }
          if (CAST) store4(X, TypeOf<T>::value, 4 * c, y);
          const double a = y.x, b = y.y, cc = y.z, d = y.w;
          ss += a * a + b * b + cc * cc + d * d;
        }
      }
    } else {
      for (int c = l; c < m.cols; c += WG) {
        float y = M[c];
        if (G) {
          const float g = load1(G, m.g_type, c);
          y = fmaf(mu, y, g);
          M[c] = y;
          y = target(y, g, mu, L.nesterov);
        }
        if (CAST) store1(X, TypeOf<T>::value, c, y);
        ss += (double)y * (double)y;
      }
    }
  }
  ss = group_sum<WG>(ss, scratch);
  if (active && l == 0) L.rsum[task] = ss;
}

// 1 / (norm + eps) from the sum of squares. A matrix of zeros gets scale 0
// (its update is 0, also with eps = 0); the scale of a norm below 1 / FLT_MAX
// is FLT_MAX.
__device__ __forceinline__ float scale_of(double t, float eps) {
  const double inv = t > 0.0 ? 1.0 / (sqrt(t) + (double)eps) : 0.0;
  return inv > 3.4028234663852886e38 ? 3.4028234663852886e38f : (float)inv;
}
// Sum of a matrix's row sums by a warp, in a fixed order.
__device__ __forceinline__ double sum_rows(const double* r, int rows, int lane) {
  double t = 0.0;
  for (int k = lane; k < rows; k += 32) t += r[k];
  return warp_sum(t);
}

// One warp per matrix.
__global__ void __launch_bounds__(BLOCK) stack_norm(const __grid_constant__ StackLaunch L) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int i = blockIdx.x * (BLOCK / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= L.total_mats) return;
  int lo = 0, hi = L.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.m[mid].mat_begin <= i) lo = mid; else hi = mid - 1;
  }
  const StackMat& m = L.m[lo];
  const double t = sum_rows(L.rsum + m.row_begin + (int64_t)(i - m.mat_begin) * m.rows, m.rows, lane);
  if (lane == 0) {
    if (!isfinite(t)) report(L.status, MUON_ERR_NONFINITE);
    const float s = scale_of(t, L.eps);
    L.scale[i] = s;
    L.xscale[i] = L.folded ? s : 1.f / m.kappa;
  }
}

// X <- scale * target * kappa: the gradient is read again for Nesterov's
// target (2 or 4 bytes an element against 8 for writing the target in fp32
// and reading it back). With L.sums each warp adds its matrix's row sums
// itself: where there are few rows (stack_impl) that is less than a launch.
template <int WG, typename T, int PL>
__global__ void __launch_bounds__(BLOCK) stack_cast(const __grid_constant__ StackLaunch L) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int task = blockIdx.x * (BLOCK / WG) + threadIdx.x / WG;
  const int l = threadIdx.x % WG;
  if (task >= L.total_rows) return;
  const Row w = find_row(L, task);
  const StackMat& m = L.m[w.mat];
  const float* M = m.M + w.b * m.m_stride + w.r * m.m_ld;
  const void* G = m.G && L.nesterov ? row_at(m.G, m.g_type, w.b * m.g_stride + w.r * m.g_ld) : nullptr;
  T* X = static_cast<T*>(m.X) + ((int64_t)w.b * PL * m.rows + w.r) * m.ldx;
  T* Y = X + (int64_t)m.rows * m.ldx;  // the low plane
  float sc;
  if (L.sums) {
    const double t = sum_rows(L.rsum + m.row_begin + (int64_t)w.b * m.rows, m.rows, threadIdx.x & 31);
    if (!isfinite(t) && w.r == 0 && l == 0) report(L.status, MUON_ERR_NONFINITE);
    sc = scale_of(t, L.eps);
  } else {
    sc = L.scale[m.mat_begin + w.b];
  }
  const float kappa = m.kappa, mu = L.mu;
  if (m.vec) {
    const int n4 = m.cols >> 2;
#pragma unroll UNROLL
    for (int c = l; c < n4; c += WG) {
      float4 y = *reinterpret_cast<const float4*>(M + 4 * c);
      if (G) {
        const float4 g = load4(G, m.g_type, 4 * c);
        y.x = fmaf(mu, y.x, g.x); y.y = fmaf(mu, y.y, g.y); y.z = fmaf(mu, y.z, g.z); y.w = fmaf(mu, y.w, g.w);
      }
      y.x = y.x * sc * kappa; y.y = y.y * sc * kappa; y.z = y.z * sc * kappa; y.w = y.w * sc * kappa;
      store4(X, TypeOf<T>::value, 4 * c, y);
      if (PL == 2) {
        const float4 h = unpack4((const __half*)nullptr, pack4<__half>(y));
        store4(Y, MUON_F16, 4 * c, make_float4(y.x - h.x, y.y - h.y, y.z - h.z, y.w - h.w));
      }
    }
  } else {
    for (int c = l; c < m.cols; c += WG) {
      float y = M[c];
      if (G) y = fmaf(mu, y, load1(G, m.g_type, c));
      y = y * sc * kappa;
      store1(X, TypeOf<T>::value, c, y);
      if (PL == 2) store1(Y, MUON_F16, c, y - __half2float(__float2half_rn(y)));
    }
  }
}

// W <- keep W - step O, rounded once to W's type (and once, from the same
// fp32 value, to the copy's). A non-finite O is reported.
template <int WG, typename T, int PL>
__global__ void __launch_bounds__(BLOCK) stack_update(const __grid_constant__ StackLaunch L) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int task = blockIdx.x * (BLOCK / WG) + threadIdx.x / WG;
  const int l = threadIdx.x % WG;
  if (task >= L.total_rows) return;
  const Row w = find_row(L, task);
  const StackMat& m = L.m[w.mat];
  const T* X = static_cast<const T*>(m.X) + ((int64_t)w.b * PL * m.rows + w.r) * m.ldx;
  const T* Y = X + (int64_t)m.rows * m.ldx;
  void* W = row_at(m.W, m.w_type, w.b * m.w_stride + w.r * m.w_ld);
  void* C = m.copy ? row_at(m.copy, m.c_type, w.b * m.c_stride + w.r * m.c_ld) : nullptr;
  const float step = PL == 2 ? L.step / m.kappa : L.step, keep = L.keep;
  bool bad = false;
  if (m.vec) {
    const int n4 = m.cols >> 2;
#pragma unroll UNROLL
    for (int c = l; c < n4; c += WG) {
      float4 o = load4(X, TypeOf<T>::value, 4 * c);
      if (PL == 2) {
        const float4 y = load4(Y, MUON_F16, 4 * c);
        o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
      }
      bad |= !(isfinite(o.x) && isfinite(o.y) && isfinite(o.z) && isfinite(o.w));
      float4 v = load4(W, m.w_type, 4 * c);
      v.x = fmaf(-step, o.x, keep * v.x); v.y = fmaf(-step, o.y, keep * v.y);
      v.z = fmaf(-step, o.z, keep * v.z); v.w = fmaf(-step, o.w, keep * v.w);
      store4(W, m.w_type, 4 * c, v);
      if (C) store4(C, m.c_type, 4 * c, v);
    }
  } else {
    for (int c = l; c < m.cols; c += WG) {
      float o = load1(X, TypeOf<T>::value, c);
      if (PL == 2) o += load1(Y, MUON_F16, c);
      bad |= !isfinite(o);
      const float v = fmaf(-step, o, keep * load1(W, m.w_type, c));
      store1(W, m.w_type, c, v);
      if (C) store1(C, m.c_type, c, v);
    }
  }
  if (bad) report(L.status, MUON_ERR_NONFINITE);
}

// Rows longer than this are walked by a whole block.
constexpr int kWarpCols = 2048;

bool long_rows(const StackLaunch& L) {
  for (int i = 0; i < L.count; ++i)
    if (L.m[i].cols > kWarpCols) return true;
  return false;
}

template <typename F>
muon_status launch(F* kernel, int blocks, const StackLaunch& L, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(BLOCK);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  counters().launches += 1;
  return cudaLaunchKernelEx(&cfg, kernel, L) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

int row_blocks(const StackLaunch& L, bool wide) { return wide ? L.total_rows : (L.total_rows + BLOCK / 32 - 1) / (BLOCK / 32); }

template <typename T>
muon_status momentum_typed(const StackLaunch& L, bool cast, cudaStream_t s) {
  const bool wide = long_rows(L);
  if (cast) return launch(wide ? stack_momentum<BLOCK, T, true> : stack_momentum<32, T, true>, row_blocks(L, wide), L, s);
  return launch(wide ? stack_momentum<BLOCK, T, false> : stack_momentum<32, T, false>, row_blocks(L, wide), L, s);
}

}  // namespace

muon_status launch_stack_momentum(const StackLaunch& L, Op t, bool cast, cudaStream_t s) {
  if (cast && t == Op::BF16) return momentum_typed<__nv_bfloat16>(L, true, s);
  return momentum_typed<float>(L, cast, s);
}

muon_status launch_stack_norm(const StackLaunch& L, cudaStream_t s) {
  return launch(stack_norm, (L.total_mats + BLOCK / 32 - 1) / (BLOCK / 32), L, s);
}

#define MUON_STACK_FORMS(kernel)                                                                              \
  const bool wide = long_rows(L);                                                                             \
  const int blocks = row_blocks(L, wide);                                                                     \
  if (planes == 2) return launch(wide ? kernel<BLOCK, __half, 2> : kernel<32, __half, 2>, blocks, L, s);      \
  if (t == Op::BF16) return launch(wide ? kernel<BLOCK, __nv_bfloat16, 1> : kernel<32, __nv_bfloat16, 1>, blocks, L, s); \
  if (t == Op::F16) return launch(wide ? kernel<BLOCK, __half, 1> : kernel<32, __half, 1>, blocks, L, s);     \
  return launch(wide ? kernel<BLOCK, float, 1> : kernel<32, float, 1>, blocks, L, s);

muon_status launch_stack_cast(const StackLaunch& L, Op t, int planes, cudaStream_t s) { MUON_STACK_FORMS(stack_cast) }

muon_status launch_stack_update(const StackLaunch& L, Op t, int planes, cudaStream_t s) { MUON_STACK_FORMS(stack_update) }

}  // namespace muon
