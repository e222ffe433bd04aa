// The whole update of a stack of small matrices in one launch: momentum,
// norm, Newton-Schulz chain and weight update with the matrix resident on
// chip. For matrices whose shorter side n is at most 128 and whose longer
// side m at most 2048.
//
// The chain of a small matrix is bound by latency: 15 dependent products of a
// few microseconds each, every one paying a launch, its setup, a pipeline
// fill and a drain. Here a cluster of C CTAs (1 to 16) holds one matrix:
// CTA r keeps columns [r mc, (r+1) mc) of the wide view X (n x m) in shared
// memory, mc = 64 g <= 512, as operands of tcgen05.mma; per step
//   A  = sum over the cluster of X_r X_r^T   (M = 128, N = n, K = mc)
//   B' = a I + b A + c A A                   (every CTA, K = n)
//   X_r <- B' X_r                            (N = mc, K = n)
// where the sum goes through distributed shared memory by bulk copies: CTA r
// receives its np / C rows of every partial result, adds them in rank order
// and copies its rows of the operand to every CTA. Both arrive on mbarriers,
// so the loop has no cluster barrier; that copies may land is implied by what
// has arrived (below), and a sender waits until its copies have read their
// source before it writes there. Element-wise remote stores took 1500 to 5900 cycles a
// step where these take a few hundred. Folding a X into B' saves reading X back
// in the epilogue.
//
// A and B' always keep two planes (hi + lo of the operand type): they never
// leave the chip, and with one plane the rounding of their diagonals would be
// the largest error of the chain (a 513 x 33 bf16 matrix, whose singular
// values are all alike: 2.6e-2 with one plane). X has one plane in bf16 and
// fp16 and two in two-plane fp16.
//
// Both products that read X use the same copy of it: 64-column groups of
// 128-byte rows with 128-byte swizzle are K-major for X X^T and MN-major for
// B' X. Rows n.. of the M side may hold anything (they only reach accumulator
// lanes that are never read), but the K side of B' X reads rows up to np, n
// rounded up to 16, which are zero.
//
// Until the norm is known, and for the last step's result, an element's fp32
// value is kept split over the two planes' places (its high and low 16 bits),
// so neither needs memory of its own.
//
// A product of two-plane operands is hi hi + hi lo + lo hi, as in the
// Newton-Schulz GEMM; X is stored times kappa and A, B' times rho, powers of
// two.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "resident_model.h"
#include "rowio.cuh"
#include "stack.cuh"

namespace muon {

namespace res {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int TMEM_COLS = 512;

struct Params {
  StackMat m;
  int n, np, long_side, tall;  // wide view: n x long_side
  int g, C;
  float mu, step, keep, eps;
  int nesterov, T;
  float kappa;
  float alpha;            // rho / kappa^2: the stored A from X X^T
  float back, last;       // 1 / rho, and 1 / (rho kappa) for the last step's result
  float lin[MUON_MAX_T], quad[MUON_MAX_T], diag[MUON_MAX_T];  // b, c / rho, rho a: the stored B'
  int* status;
  unsigned long long timeout_ns;
};

// Copy of `bytes` of this CTA's shared memory to a CTA of the cluster (its own
// included), whose barrier counts the bytes.
__device__ __forceinline__ void copy_cluster(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// Arrive on a barrier of another CTA, ordered after this thread's earlier accesses.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void st_cluster_f64(uint32_t a, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(v) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* a) { asm volatile("prefetch.global.L2 [%0];" ::"l"(a)); }

__device__ __forceinline__ void tmem_ld_32x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Byte offset of 16-byte chunk ch (8 columns) of row r in a 64-column group.
__device__ __forceinline__ uint32_t at(int r, int ch) { return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4)); }

// Eight values to operand chunks: the high plane at hi, the low one at lo.
template <typename T, int PL>
__device__ __forceinline__ void put8(uint8_t* hi, uint8_t* lo, const float* v) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = Elem<T>::pack2(v[2 * i], v[2 * i + 1]);
    if (PL == 2) {
      const float2 f = Elem<T>::unpack2(h[i]);
      l[i] = Elem<T>::pack2(v[2 * i] - f.x, v[2 * i + 1] - f.y);
    }
  }
  *reinterpret_cast<uint4*>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
  if (PL == 2) *reinterpret_cast<uint4*>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
}
template <typename T, int PL>
__device__ __forceinline__ void get8(const uint8_t* hi, const uint8_t* lo, float* v) {
  const uint4 h = *reinterpret_cast<const uint4*>(hi);
  const uint32_t hh[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Elem<T>::unpack2(hh[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
  if (PL == 2) {
    const uint4 l = *reinterpret_cast<const uint4*>(lo);
    const uint32_t ll[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Elem<T>::unpack2(ll[i]);
      v[2 * i] += f.x;
      v[2 * i + 1] += f.y;
    }
  }
}
// Eight fp32 values as their high and low halves in the two planes' places.
__device__ __forceinline__ void put8_raw(uint8_t* hi, uint8_t* lo, const float* v) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
    h[i] = __byte_perm(a, b, 0x7632);
    l[i] = __byte_perm(a, b, 0x5410);
  }
  *reinterpret_cast<uint4*>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void get8_raw(const uint8_t* hi, const uint8_t* lo, float* v) {
  const uint4 h = *reinterpret_cast<const uint4*>(hi), l = *reinterpret_cast<const uint4*>(lo);
  const uint32_t hh[4] = {h.x, h.y, h.z, h.w}, ll[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(__byte_perm(ll[i], hh[i], 0x5410));
    v[2 * i + 1] = __uint_as_float(__byte_perm(ll[i], hh[i], 0x7632));
  }
}

template <typename T, int PL>
__global__ void __launch_bounds__(THREADS, 1) stack_resident(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int g = p.g, C = p.C, group = group_bytes(p.np);
  uint8_t* const X = smem;                     // high plane: g groups; low plane behind
  uint8_t* const Xl = X + g * group;
  uint8_t* const A = X + 2 * g * group;        // high plane; low plane behind
  const int a_plane = (p.np + 63) / 64 * group;
  uint8_t* const Al = A + a_plane;
  uint8_t* const R = Al + a_plane;  // cluster: partial sums of this CTA's rows, [C][np / C][np] fp32
  double* slots = reinterpret_cast<double*>(R + (C > 1 ? p.np * p.np * 4 : 0));  // one partial norm per CTA of the cluster
  double* scratch = slots + MAX_C;
  uint64_t* bar = reinterpret_cast<uint64_t*>(scratch + 32);  // products done
  uint64_t* sums = bar + 1;   // partial sums arrived, and every CTA's own have been sent
  uint64_t* rows = bar + 2;   // rows of A arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = C > 1 ? (int)cluster_rank() : 0;
  const int mat = (int)blockIdx.x / C;
  auto sync_all = [&]() {
    if (C > 1) cluster_sync(); else __syncthreads();
  };

  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(sums, (uint32_t)C + 1);
    mbar_init(rows, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  // zeros where the matrix has no element
  for (int i = tid; i < 2 * g * group / 16; i += THREADS) reinterpret_cast<uint4*>(X)[i] = make_uint4(0u, 0u, 0u, 0u);
  tc_fence_before();
  sync_all();  // also: every CTA of the cluster has started, so its shared memory may be written
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();

  // ------------------------------------------------------------------
  // momentum and the update's target, in fp32 halves
  // ------------------------------------------------------------------
  const StackMat& m = p.m;
  const int mc = 64 * g;
  const int first = rank * mc;  // this CTA's columns of the wide view
  const int width = max(0, min(mc, p.long_side - first));
  float* const M = m.M + (int64_t)mat * m.m_stride;
  const void* const G = m.G ? row_at(m.G, m.g_type, (int64_t)mat * m.g_stride) : nullptr;
  void* const W = row_at(m.W, m.w_type, (int64_t)mat * m.w_stride);
  void* const K = m.copy ? row_at(m.copy, m.c_type, (int64_t)mat * m.c_stride) : nullptr;
  // stored rows of this CTA and the contiguous run in each of them
  const int srows = p.tall ? width : p.n, srow0 = p.tall ? first : 0;
  const int scols = p.tall ? p.n : width, scol0 = p.tall ? 0 : first;
  // byte offset (within a plane) of stored element (r, c) of this CTA
  auto spot = [&](int r, int c) -> uint32_t {
    const int i = p.tall ? c : r, j = p.tall ? r : c;
    return (uint32_t)((j >> 6) * group) + at(i, (j & 63) >> 3) + (j & 7) * 2;
  };
  auto put_raw = [&](int r, int c, float v) {
    const uint32_t o = spot(r, c), u = __float_as_uint(v);
    *reinterpret_cast<uint16_t*>(X + o) = (uint16_t)(u >> 16);
    *reinterpret_cast<uint16_t*>(Xl + o) = (uint16_t)u;
  };
  auto get_raw = [&](int r, int c) -> float {
    const uint32_t o = spot(r, c);
    return __uint_as_float(((uint32_t)*reinterpret_cast<const uint16_t*>(X + o) << 16) |
                           *reinterpret_cast<const uint16_t*>(Xl + o));
  };
  double ss = 0.0;
  if (m.vec) {
    constexpr int U = 8;  // rows in flight per warp
    for (int r0 = warp; r0 < srows; r0 += WARPS * U) {
      for (int c = 4 * lane; c < scols; c += 128) {
        float4 y[U], gr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * WARPS;
          if (r < srows) {
            y[u] = *reinterpret_cast<const float4*>(M + (srow0 + r) * m.m_ld + scol0 + c);
            if (G) gr[u] = load4(row_at(G, m.g_type, (srow0 + r) * m.g_ld + scol0), m.g_type, c);
            // W is read at the end: into L2 meanwhile
            prefetch_l2(row_at(W, m.w_type, (srow0 + r) * m.w_ld + scol0 + c));
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * WARPS;
          if (r >= srows) break;
          float4 v = y[u];
          if (G) {
            v.x = fmaf(p.mu, v.x, gr[u].x); v.y = fmaf(p.mu, v.y, gr[u].y);
            v.z = fmaf(p.mu, v.z, gr[u].z); v.w = fmaf(p.mu, v.w, gr[u].w);
            *reinterpret_cast<float4*>(M + (srow0 + r) * m.m_ld + scol0 + c) = v;
            v.x = target(v.x, gr[u].x, p.mu, p.nesterov); v.y = target(v.y, gr[u].y, p.mu, p.nesterov);
            v.z = target(v.z, gr[u].z, p.mu, p.nesterov); v.w = target(v.w, gr[u].w, p.mu, p.nesterov);
          }
          if (p.tall) {
            put_raw(r, c, v.x); put_raw(r, c + 1, v.y); put_raw(r, c + 2, v.z); put_raw(r, c + 3, v.w);
          } else {
            const uint32_t a = __float_as_uint(v.x), b = __float_as_uint(v.y), d = __float_as_uint(v.z),
                           e = __float_as_uint(v.w);
            const uint32_t o = spot(r, c);
            *reinterpret_cast<uint2*>(X + o) = make_uint2(__byte_perm(a, b, 0x7632), __byte_perm(d, e, 0x7632));
            *reinterpret_cast<uint2*>(Xl + o) = make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(d, e, 0x5410));
          }
          const double a = v.x, b = v.y, d = v.z, e = v.w;
          ss += a * a + b * b + d * d + e * e;
        }
      }
    }
  } else {
    constexpr int U = 8;
    for (int r0 = warp; r0 < srows; r0 += WARPS * U)
      for (int c = lane; c < scols; c += 32) {
        float y[U], gr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * WARPS;
          if (r < srows) {
            y[u] = M[(srow0 + r) * m.m_ld + scol0 + c];
            if (G) gr[u] = load1(row_at(G, m.g_type, (srow0 + r) * m.g_ld + scol0), m.g_type, c);
            if (lane % 8 == 0) prefetch_l2(row_at(W, m.w_type, (srow0 + r) * m.w_ld + scol0 + c));
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * WARPS;
          if (r >= srows) break;
          float v = y[u];
          if (G) {
            v = fmaf(p.mu, v, gr[u]);
            M[(srow0 + r) * m.m_ld + scol0 + c] = v;
            v = target(v, gr[u], p.mu, p.nesterov);
          }
          put_raw(r, c, v);
          ss += (double)v * (double)v;
        }
      }
  }
  double total = block_sum(ss, scratch);
  if (C > 1) {
    if (tid < C) st_cluster_f64(mapa_shared(smem_u32(slots + rank), (uint32_t)tid), total);
    cluster_sync();
    total = 0.0;
    for (int r = 0; r < C; ++r) total += slots[r];  // in rank order: the same sum in every CTA
  }
  if (!isfinite(total) && tid == 0 && rank == 0) report(p.status, MUON_ERR_NONFINITE);
  const double inv = total > 0.0 ? 1.0 / (sqrt(total) + (double)p.eps) : 0.0;
  const float sc = inv > 3.4028234663852886e38 ? 3.4028234663852886e38f : (float)inv;
  __syncthreads();  // every element is in place
  for (int i = tid; i < g * group / 16; i += THREADS) {
    uint8_t* h = X + i * 16;
    float v[8];
    get8_raw(h, h + g * group, v);
#pragma unroll
    for (int x = 0; x < 8; ++x) v[x] = v[x] * sc * p.kappa;
    put8<T, PL>(h, h + g * group, v);
  }

  // ------------------------------------------------------------------
  // the chain
  // ------------------------------------------------------------------
  constexpr int fmt = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
  // Descriptors hold 14 bits of the address; in a cluster the bits above the
  // shared-memory window carry the CTA's rank and must not reach the other fields.
  const uint32_t a_a = smem_u32(A);
  const uint32_t x_d = smem_u32(X) & 0x3FFFFu, a_d = a_a & 0x3FFFFu;
  const uint32_t x_low = PL == 2 ? (uint32_t)(g * group) >> 4 : 0u, a_low = (uint32_t)a_plane >> 4;
  const uint64_t k_major = smem_desc_sw128(0, 16, 1024);       // 8-row groups 1 KB apart
  const uint64_t mn_major = smem_desc_sw128(0, group, 1024);   // 64-column atoms a group apart
  const uint32_t idesc_n = idesc_f16(fmt, 0, 0, 128, p.np), idesc_x = idesc_f16(fmt, 0, 1, 128, min(mc, 256)),
                 idesc_x2 = idesc_f16(fmt, 0, 1, 128, mc > 256 ? mc - 256 : 64);  // N is at most 256
  uint32_t parity = 0;
  // after the operands are written: order them before the products, which
  // warp 0 issues, and wait for their completion. A wait that runs out
  // reports it and then still waits, with the drain's bound, so that nothing
  // reads, overwrites or frees what a product in flight uses; the cluster's
  // barriers need every CTA, so the chain goes on.
  auto wait_for = [&](uint64_t* b, uint32_t par) {
    if (!mbar_wait_bounded(b, par, abort_flag, p.timeout_ns, p.status)) drain_wait(b, par, p.status);
  };
  auto products = [&](auto issue) {
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
      tc_fence_after();
      const uint32_t on = elect_one();
      issue(on);
      umma_commit_if(on, bar);
    }
    wait_for(bar, parity);
    parity ^= 1;
    __syncwarp();
    tc_fence_after();
  };
  // hi hi, + hi lo where the N side has two planes, + lo hi where the M side has
  auto mma = [&](uint32_t on, uint32_t d, uint64_t ad, uint64_t bd, uint32_t low_a, uint32_t low_b, uint32_t idesc, bool acc) {
    umma_f16_if(on, d, ad, bd, idesc, acc);
    if (low_b) umma_f16_if(on, d, ad, bd + low_b, idesc, 1);
    if (low_a) umma_f16_if(on, d, ad + low_a, bd, idesc, 1);
  };
  const int q = warp & 3, half = warp >> 2;
  const int row = q * 32 + lane;                 // this thread's accumulator lane
  const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
  const bool rows_here = q * 32 < p.np;          // warp-uniform
  const int swz = p.np % 32 == 0 ? 7 : 3;        // 16-byte chunks of the fp32 sums, swizzled by the row
  const int rows_per = p.np / C;                 // rows of A that this CTA sums (np is a multiple of 16)
  // This thread's columns of A's accumulator, 16 from half * 16, half * 16 +
  // 32, ...: all loads in flight before the one wait. Returns their count.
  auto load_chunks = [&](float (&v)[4][16]) -> int {
    int n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (half * 16 + 32 * k < p.np) {  // warp-uniform
        tmem_ld_32x16(tl + half * 16 + 32 * k, reinterpret_cast<uint32_t(&)[16]>(v[k]));
        n = k + 1;
      }
    tmem_wait_ld();
    return n;
  };

  for (int t = 0; t < p.T; ++t) {
    const float lin = p.lin[t], quad = p.quad[t], diag = p.diag[t], alpha = p.alpha;
    const uint32_t odd = (uint32_t)t & 1u;  // phase of the exchange's barriers
    // A = X X^T over this CTA's columns
    products([&](uint32_t on) {
      for (int j = 0; j < g; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t d = k_major | (uint64_t)((x_d + j * group + k * 32) >> 4);
          mma(on, tmem, d, d, x_low, x_low, idesc_n, j != 0 || k != 0);
        }
    });
    if (rows_here) {
      float v[4][16];
      const int chunks = load_chunks(v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k >= chunks) break;
        const int c0 = half * 16 + 32 * k;
        if (row >= p.np) continue;
        if (C == 1) {
          const uint32_t o = (uint32_t)((c0 >> 6) * group);
#pragma unroll
          for (int x = 0; x < 16; ++x) v[k][x] *= alpha;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t w = o + at(row, ((c0 & 63) >> 3) + s);
            put8<T, 2>(A + w, Al + w, v[k] + 8 * s);
          }
        } else {
          // partial sums in fp32 where A's planes go: B' of the last step has
          // been read, and the peers send rows of A only once this CTA's
          // partial sums have left
#pragma unroll
          for (int s = 0; s < 4; ++s)
            *reinterpret_cast<float4*>(A + row * p.np * 4 + ((((c0 >> 2) + s) ^ (row & swz)) << 4)) =
                make_float4(v[k][4 * s], v[k][4 * s + 1], v[k][4 * s + 2], v[k][4 * s + 3]);
        }
      }
    }
    if (C > 1) {
      const uint32_t part = (uint32_t)(rows_per * p.np * 4);
      fence_async_smem();
      tc_fence_before();
      __syncthreads();
      if (warp == 0) {
        if (lane == 0) {
          mbar_arrive_expect_tx(sums, part * C);
          mbar_arrive_expect_tx(rows, (uint32_t)(2 * a_plane));
        }
        __syncwarp();
        if (lane < C) {
          // rows lane * rows_per .. to that CTA, in its slot for this one. It
          // has added what came in the last step: rows of A from it followed.
          copy_cluster(mapa_shared(smem_u32(R) + rank * part, (uint32_t)lane), a_a + lane * part, part,
                       mapa_shared(smem_u32(sums), (uint32_t)lane));
          bulk_commit();
          bulk_wait_read0();
        }
        __syncwarp();  // all of this CTA's copies have been read: its A may be overwritten
        if (lane < C) arrive_cluster(mapa_shared(smem_u32(sums), (uint32_t)lane));
      }
      wait_for(sums, odd);
      // the sums of this CTA's rows, eight columns a thread, at their place
      const int cpr = p.np >> 3;
      for (int j = tid; j < rows_per * cpr; j += THREADS) {
        const int lr = j / cpr, c0 = 8 * (j - lr * cpr);
        float v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = 0.f;
#pragma unroll 4
        for (int k = 0; k < C; ++k) {
          const uint8_t* src = R + (k * rows_per + lr) * p.np * 4;
          const int x0 = (rank * rows_per + lr) & swz, ch = c0 >> 2;
          const float4 x = *reinterpret_cast<const float4*>(src + ((ch ^ x0) << 4));
          const float4 y = *reinterpret_cast<const float4*>(src + (((ch + 1) ^ x0) << 4));
          v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
          v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] *= alpha;
        const uint32_t w = (uint32_t)((c0 >> 6) * group) + at(rank * rows_per + lr, (c0 & 63) >> 3);
        put8<T, 2>(A + w, Al + w, v);
      }
      fence_async_smem();
      __syncthreads();
      // and to the peers: every CTA's partial sums have left its A
      const int pieces = 2 * a_plane / group;  // groups of both planes, contiguous
      for (int i = tid; i < pieces * C; i += THREADS) {
        const int to = i / pieces;
        if (to == rank) continue;
        const uint32_t o = a_a + (i - to * pieces) * group + rank * rows_per * 128;
        copy_cluster(mapa_shared(o, (uint32_t)to), o, (uint32_t)(rows_per * 128), mapa_shared(smem_u32(rows), (uint32_t)to));
      }
      bulk_commit();
      if (tid == 0) mbar_complete_tx(rows, (uint32_t)(pieces * rows_per * 128));  // its own are there
      wait_for(rows, odd);
      // What has arrived says nothing of what this thread has sent: B' takes the
      // place of these rows once every copy has read them (the barrier ahead of
      // the next product makes that every thread's).
      bulk_wait_read0();
    }
    // B' = a I + b A + c A A, in A's place (every thread rewrites what it read)
    products([&](uint32_t on) {
      for (int k = 0; k < p.np / 16; ++k) {
        const uint64_t d = k_major | (uint64_t)((a_d + (k >> 2) * group + (k & 3) * 32) >> 4);
        mma(on, tmem, d, d, a_low, a_low, idesc_n, k != 0);
      }
    });
    if (rows_here) {
      float y[4][16];
      const int chunks = load_chunks(y);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k >= chunks || row >= p.np) break;
        const int c0 = half * 16 + 32 * k;
        const uint32_t o = (uint32_t)((c0 >> 6) * group);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t w = o + at(row, ((c0 & 63) >> 3) + s);
          float v[8];
          get8<T, 2>(A + w, Al + w, v);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            v[x] = fmaf(quad, y[k][8 * s + x], lin * v[x]);
            if (c0 + 8 * s + x == row) v[x] += diag;
          }
          put8<T, 2>(A + w, Al + w, v);
        }
      }
    }
    // X <- B' X
    products([&](uint32_t on) {
      for (int k = 0; k < p.np / 16; ++k) {
        const uint64_t ad = k_major | (uint64_t)((a_d + (k >> 2) * group + (k & 3) * 32) >> 4);
        const uint64_t bd = mn_major | (uint64_t)((x_d + k * 2048) >> 4);
        mma(on, tmem, ad, bd, a_low, x_low, idesc_x, k != 0);
        if (mc > 256) mma(on, tmem + 256, ad, bd + (uint32_t)(4 * group >> 4), a_low, x_low, idesc_x2, k != 0);
      }
    });
    const bool last = t + 1 == p.T;
    const float back = last ? p.last : p.back;
    if (rows_here)
      for (int c0 = half * 32; c0 < mc; c0 += 64) {  // one group an iteration
        uint32_t r[32];
        tmem_ld_32x32(tl + c0, r);
        tmem_wait_ld();
        if (row < p.np) {
          const uint32_t o = (uint32_t)((c0 >> 6) * group);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            float v[8];
            const uint32_t w = o + at(row, ((c0 & 63) >> 3) + s);
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = back * __uint_as_float(r[8 * s + x]);
            if (last) put8_raw(X + w, Xl + w, v);
            else put8<T, PL>(X + w, Xl + w, v);
          }
        }
      }
  }
  tc_fence_before();
  sync_all();  // the result is in place; no peer writes here any more

  // ------------------------------------------------------------------
  // W <- keep W - step O
  // ------------------------------------------------------------------
  bool bad = false;
  if (m.vec) {
    constexpr int U = 8;
    for (int r0 = warp; r0 < srows; r0 += WARPS * U) {
      for (int c = 4 * lane; c < scols; c += 128) {
        float4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * WARPS;
          if (r < srows) w[u] = load4(row_at(W, m.w_type, (srow0 + r) * m.w_ld + scol0), m.w_type, c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * WARPS;
          if (r >= srows) break;
          float4 o;
          if (p.tall) {
            o = make_float4(get_raw(r, c), get_raw(r, c + 1), get_raw(r, c + 2), get_raw(r, c + 3));
          } else {
            const uint32_t s = spot(r, c);
            const uint2 h = *reinterpret_cast<const uint2*>(X + s), l = *reinterpret_cast<const uint2*>(Xl + s);
            o = make_float4(__uint_as_float(__byte_perm(l.x, h.x, 0x5410)), __uint_as_float(__byte_perm(l.x, h.x, 0x7632)),
                            __uint_as_float(__byte_perm(l.y, h.y, 0x5410)), __uint_as_float(__byte_perm(l.y, h.y, 0x7632)));
          }
          bad |= !(isfinite(o.x) && isfinite(o.y) && isfinite(o.z) && isfinite(o.w));
          float4 v = w[u];
          v.x = fmaf(-p.step, o.x, p.keep * v.x); v.y = fmaf(-p.step, o.y, p.keep * v.y);
          v.z = fmaf(-p.step, o.z, p.keep * v.z); v.w = fmaf(-p.step, o.w, p.keep * v.w);
          store4(row_at(W, m.w_type, (srow0 + r) * m.w_ld + scol0), m.w_type, c, v);
          if (K) store4(row_at(K, m.c_type, (srow0 + r) * m.c_ld + scol0), m.c_type, c, v);
        }
      }
    }
  } else {
    constexpr int U = 8;
    for (int r0 = warp; r0 < srows; r0 += WARPS * U)
      for (int c = lane; c < scols; c += 32) {
        float w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * WARPS;
          if (r < srows) w[u] = load1(row_at(W, m.w_type, (srow0 + r) * m.w_ld + scol0), m.w_type, c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = r0 + u * WARPS;
          if (r >= srows) break;
          const float o = get_raw(r, c);
          bad |= !isfinite(o);
          const float v = fmaf(-p.step, o, p.keep * w[u]);
          store1(row_at(W, m.w_type, (srow0 + r) * m.w_ld + scol0), m.w_type, c, v);
          if (K) store1(row_at(K, m.c_type, (srow0 + r) * m.c_ld + scol0), m.c_type, c, v);
        }
      }
  }
  if (bad) report(p.status, MUON_ERR_NONFINITE);
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

}  // namespace res

namespace {

// The kernel's attributes, once per device.
template <typename T, int PL>
muon_status set_up() {
  static std::mutex mu;
  static bool ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return MUON_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(res::stack_resident<T, PL>, cudaFuncAttributeMaxDynamicSharedMemorySize, res::SMEM_MAX) != cudaSuccess ||
        cudaFuncSetAttribute(res::stack_resident<T, PL>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
      cudaGetLastError();
      return MUON_ERR_CUDA;
    }
    ready[dev] = true;
  }
  return MUON_OK;
}

template <typename T, int PL>
muon_status launch_resident(const res::Params& p, cudaStream_t s) {
  const muon_status up = set_up<T, PL>();
  if (up != MUON_OK) return up;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.m.count * p.C));
  cfg.blockDim = dim3(res::THREADS);
  cfg.dynamicSmemBytes = res::smem_bytes(p.g, p.np, p.C);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.C > 1 ? 2 : 1;
  counters().launches += 1;
  return cudaLaunchKernelEx(&cfg, res::stack_resident<T, PL>, p) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

}  // namespace

namespace {

// Clusters of C CTAs (one per SM) that can run at once on the current device;
// 0 where such a cluster cannot be scheduled.
int cluster_capacity(int C) {
  static std::mutex mu;
  static int cap[64][5];  // 0: not asked yet, -1: none
  if (C == 1) return num_sms();
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || set_up<__half, 2>() != MUON_OK) {
    cudaGetLastError();
    return 0;
  }
  int k = 0;
  while ((1 << k) < C) ++k;
  std::lock_guard<std::mutex> lock(mu);
  int& n = cap[dev][k];
  if (n == 0) {
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3((unsigned)(num_sms() / C * C));
    q.blockDim = dim3(res::THREADS);
    q.dynamicSmemBytes = res::SMEM_MAX;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = (unsigned)C;
    a[0].val.clusterDim.y = 1;
    a[0].val.clusterDim.z = 1;
    q.attrs = a;
    q.numAttrs = 1;
    int c = 0;
    const bool ok = num_sms() >= C && cudaOccupancyMaxActiveClusters(&c, res::stack_resident<__half, 2>, &q) == cudaSuccess && c > 0;
    cudaGetLastError();
    n = ok ? std::min(c, num_sms() / C) : -1;
  }
  return std::max(n, 0);
}

}  // namespace

bool resident_fits(int64_t rows, int64_t cols, int64_t count, int T, int planes, int* C_out) {
  return res::choose_cluster(rows, cols, count, T, planes, cluster_capacity, C_out);
}

muon_status launch_stack_resident(const StackLaunch& L, const muon_ns_params& ns, Op t, int planes, float kappa, float rho,
                                  uint64_t timeout_ns, cudaStream_t s) {
  res::Params p{};
  p.m = L.m[0];
  p.tall = p.m.rows > p.m.cols;
  p.n = p.tall ? p.m.cols : p.m.rows;
  p.long_side = p.tall ? p.m.rows : p.m.cols;
  p.np = (p.n + 15) / 16 * 16;
  resident_fits(p.m.rows, p.m.cols, p.m.count, ns.T, planes, &p.C);
  if (p.C < 1) return MUON_ERR_INVALID_ARG;
  p.g = ((p.long_side + 63) / 64 + p.C - 1) / p.C;
  p.mu = L.mu;
  p.step = L.step;
  p.keep = L.keep;
  p.eps = L.eps;
  p.nesterov = L.nesterov;
  p.T = ns.T;
  p.kappa = kappa;
  p.alpha = rho / kappa / kappa;
  p.back = 1.f / rho;
  p.last = 1.f / rho / kappa;
  for (int i = 0; i < ns.T; ++i) {
    p.lin[i] = ns.coeffs[i][1];
    p.quad[i] = ns.coeffs[i][2] / rho;
    p.diag[i] = ns.coeffs[i][0] * rho;
  }
  p.status = L.status;
  p.timeout_ns = timeout_ns;
  if (planes == 2) return launch_resident<__half, 2>(p, s);
  return t == Op::BF16 ? launch_resident<__nv_bfloat16, 1>(p, s) : launch_resident<__half, 1>(p, s);
}

}  // namespace muon
