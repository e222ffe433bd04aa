// Matrix products grouped by expert with ragged sizes, on sm_100a.
//
// The rows of x (tokens x k) are sorted by expert; expert e owns rows
// offsets[e] .. offsets[e+1] (device int32, so the sizes never reach the
// host). With W_e the e-th n x k weight:
//   grouped_matmul     y[r,:]  = x[r,:] W_e^T          (ROWS, W read K-major)
//   grouped_matmul_dx  dx[r,:] = dy[r,:] W_e           (ROWS, W read MN-major)
//   grouped_matmul_dw  dW_e    = alpha dy_e^T x_e + beta dW_e   (DW)
//
// One persistent, warp-specialised launch over every expert's tiles (the
// roles and the CTA-pair mainloop are those of the Newton-Schulz GEMM): a
// cluster of two CTAs owns a tile of 256 x NT, tcgen05.mma cta_group::2 with
// M = 256, operands by TMA with 128-byte swizzle, two fp32 accumulators of
// 256 TMEM columns so that the epilogue of one tile overlaps the mainloop of
// the next.
//
// ROWS computes the transposed product: the expert's weights are the M side
// (always full tiles) and its tokens the N side, because the instruction
// takes any N that is a multiple of 32: a ragged group wastes at most 31
// columns instead of up to 255 rows, and a decoding batch of a few tokens
// streams each weight once through a narrow tile. NT, the widest token tile
// of a launch, is 32, 64, 128 or 256; a narrow one leaves room for more
// stages. Rows of neighbouring experts that a box reads past the end of a
// group only reach accumulator columns that are never stored.
//
// DW has the tokens on the K side, where a neighbour's rows would enter the
// sums (and a NaN among them would spoil them): a small launch first writes,
// per expert, copies of the two operands' tensor maps whose row count ends
// with the expert's last row, so that the copies themselves fill zeros behind
// it. An expert without rows gets beta dW_e (0 when beta is 0).
// When there are fewer tiles than CTA pairs, each expert's rows are cut into
// parts, one work unit each, whose fp32 sums go to the workspace (at most one
// per CTA pair); a second launch adds them in order.
//
// The issuing roles are whole warps (common.cuh: a tenth less time for 32768
// rows of 2048 into 64 x 4096, both forms in turn on one GPU; in a loop, at the
// power cap, that product takes 510 to 545 us). An operand is one copy per
// k-block (an MN-major one, 64 columns wide by its swizzle, through a map that
// has the 64-column blocks as a dimension of their own).
//
// Every wait is bounded as in the Newton-Schulz GEMM; offsets are clamped to
// 0..tokens before use, and a decreasing or out-of-range entry is reported as
// MUON_ERR_INVALID_ARG.
#include <algorithm>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace muon {

namespace grp {

constexpr int BM = 128, BK = 64;  // BM: rows of the M side per CTA
constexpr int TILE_M = 2 * BM;
constexpr int UMMA_K = 16;
constexpr int EPI_WARP0 = 4;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int TMEM_COLS = 512;
constexpr int ACC_COLS = 256;
constexpr int kMaxExperts = 1024;
// The tensor core truncates each addition to an fp32 accumulator, which
// shrinks a long sum a little with every instruction (measured: an fp32 dW of
// 1024 rows is 9.7e-7 off, in proportion to the rows). Sums into fp32 outputs
// are therefore cut every 768 rows (12 k-blocks) and the parts added with
// rounding to nearest, in order, by the same threads; a part's epilogue
// overlaps the next part's products.
constexpr int kPartBlocks = 12;

enum : int { ROWS = 0, DW = 1 };

template <typename O, int MODE, int NT>
struct Cfg {
  static constexpr int A_STAGE = BM * BK * 2;
  static constexpr int B_STAGE = (NT / 2) * BK * 2;
  static constexpr int TX_BYTES = 2 * (A_STAGE + B_STAGE);  // per stage, both CTAs
  static constexpr int STAGES = MODE == DW && sizeof(O) == 4 ? 5 : NT == 256 ? 6 : NT <= 64 ? 10 : 8;
  static constexpr int EPI_BLOCK = 32 * 32 * (int)sizeof(O);
  static constexpr int EPI_BUF = MODE == ROWS ? EPI_BLOCK : 2 * EPI_BLOCK;  // per warp; DW: two, in turn
  static constexpr int TABLE = MODE == ROWS ? (2 * kMaxExperts + 1 + 32) * 4 : 0;
  static constexpr int SMEM = 1024 + STAGES * (A_STAGE + B_STAGE) + EPI_WARPS * EPI_BUF + TABLE + (2 * STAGES + 5 + 2 * EPI_WARPS) * 8 + 64;
  static_assert(SMEM <= 232448, "exceeds the opt-in shared memory of one sm_100 CTA");
};

struct Params {
  CUtensorMap mapA;       // ROWS: W; DW: dy (the copies per expert are in `clipped`)
  CUtensorMap mapB;       // ROWS: x or dy; DW: x
  CUtensorMap* clipped;   // DW: [experts][2]
  CUtensorMap mapO;       // DW: where the kernel's results go (dW, or the parts' sums), in 32 x 32 blocks
  const int32_t* offsets;
  void* out;
  long long ldo, so;      // row stride; DW: expert stride
  int tokens, experts;
  int M, N, K;            // ROWS: M = features out, K = features in; DW: M = n, N = k
  unsigned mt_inverse;    // ROWS: 2^32 / (tiles of the M side), rounded up
  int a_mn;               // ROWS: W read MN-major
  int a_one, b_one;       // an MN-major operand's boxes are one copy (its width is a multiple of 64)
  int splits;             // DW: parts of an expert's rows (1: none, results go to out)
  float* partial;         // DW, splits > 1: 256 x 256 fp32 per (tile, part)
  float alpha, beta;      // DW
  int by_element;         // DW: rows end inside 16 bytes, which a bulk store would write whole
  int* status;
  unsigned long long timeout_ns;
};

struct Span {
  int begin, end;
};

// Rows of expert e, clamped to 0..tokens.
__device__ __forceinline__ Span span_of(const Params& p, int e) {
  int s = __ldg(p.offsets + e), t = __ldg(p.offsets + e + 1);
  s = s < 0 ? 0 : s > p.tokens ? p.tokens : s;
  t = t < s ? s : t > p.tokens ? p.tokens : t;
  return Span{s, t};
}

struct Tile {
  int e;
  int m0;        // first row of the pair's M side
  int n0;        // ROWS: first token; DW: first column of the pair's N side
  int nvalid;    // ROWS: tokens of this tile
  int n_mma;     // N of the instruction
  int t0;        // DW: first row of the K side
  int nkb;       // k-blocks
  bool whole;    // DW: the tile's only part
};

// Token tiles of a group of `cnt` rows, and their width: equal shares of a
// multiple of 32 tokens while there are few (two tiles of 160 rather than
// 256 and 44), full tiles for long groups (where rounding the shares up
// could leave a last tile without rows).
template <int NT>
__device__ __forceinline__ int token_tiles(int cnt) { return (cnt + NT - 1) / NT; }
template <int NT>
__device__ __forceinline__ int token_width(int cnt, int tiles) {
  const int share = tiles <= 1 ? cnt : tiles == 2 ? (cnt + 1) >> 1 : tiles == 3 ? (cnt + 2) / 3 : (cnt + 3) >> 2;
  return tiles > 4 ? NT : (share + 31) & ~31;
}

template <int MODE, int NT>
__device__ __forceinline__ Tile decode(const Params& p, const int* tile_begin, int tile, int mt, int ntl) {
  Tile t;
  if (MODE == ROWS) {
    // tile / mt by a multiplication with the inverse rounded up: one too large at most
    int tt = mt == 1 ? tile : (int)(((unsigned long long)(unsigned)tile * p.mt_inverse) >> 32);
    if (tt * mt > tile) --tt;
    t.m0 = (tile - tt * mt) * TILE_M;
    int lo = 0, hi = p.experts - 1;  // the last expert whose first token tile is <= tt
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tile_begin[mid] <= tt) lo = mid; else hi = mid - 1;
    }
    t.e = lo;
    const int* const first = tile_begin + kMaxExperts;  // the offsets, clamped
    const int begin = first[lo], end = max(begin, first[lo + 1]);
    const int cnt = end - begin, tiles = token_tiles<NT>(cnt);
    const int w = token_width<NT>(cnt, tiles);
    t.n0 = begin + (tt - tile_begin[lo]) * w;
    const int left = end - t.n0;
    t.nvalid = left < w ? left : w;
    t.n_mma = (t.nvalid + 31) & ~31;
    t.t0 = 0;
    t.nkb = (p.K + BK - 1) / BK;
    t.whole = true;
  } else {
    const int per = mt * ntl, u = tile / p.splits;
    t.e = u / per;
    const int r = u - t.e * per;
    t.m0 = (r / ntl) * TILE_M;
    t.n0 = (r % ntl) * NT;
    t.nvalid = 0;
    t.n_mma = NT;
    const Span s = span_of(p, t.e);
    t.t0 = s.begin;
    t.nkb = (s.end - s.begin + BK - 1) / BK;
    t.whole = p.splits == 1;
    if (!t.whole) {
      const int each = (t.nkb + p.splits - 1) / p.splits, first = (tile - u * p.splits) * each;
      t.t0 += first * BK;
      t.nkb = max(0, min(each, t.nkb - first));
    }
  }
  return t;
}

// Parts that a tile's sum is cut into (kPartBlocks).
template <int MODE, typename O>
__device__ __forceinline__ int parts_of(int nkb) {
  if (MODE == DW && std::is_same<O, float>::value && nkb > kPartBlocks) return (nkb + kPartBlocks - 1) / kPartBlocks;
  return 1;
}

// Sixteen bytes of row `lane` of a staged 32 x 32 block: chunk k, swizzled as
// the block's tensor map has it (128-byte rows of fp32, 64-byte of 16 bits).
template <typename O>
__device__ __forceinline__ uint32_t block_at(int lane, int k) {
  return sizeof(O) == 4 ? (uint32_t)(lane * 128 + ((k ^ (lane & 7)) << 4)) : (uint32_t)(lane * 64 + (((k ^ (lane >> 1)) & 3) << 4));
}

__device__ __forceinline__ void fence_map_acquire(const CUtensorMap* m) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// One thread per expert and operand: the operand's tensor map with its row
// count cut at the expert's last row.
__global__ void __launch_bounds__(128) clip_maps(const __grid_constant__ Params p) {
  grid_dependency_wait();
  grid_dependents_launch();  // the products' setup overlaps this launch; they wait for its end
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  const int e = i >> 1;
  if (e >= p.experts) return;
  const int raw0 = __ldg(p.offsets + e), raw1 = __ldg(p.offsets + e + 1);
  const Span s = span_of(p, e);
  if ((raw0 != s.begin || raw1 != s.end) && !(i & 1)) report(p.status, MUON_ERR_INVALID_ARG);
  if (s.end <= s.begin) return;  // no copy reads this expert's maps
  CUtensorMap* m = p.clipped + i;
  const uint4* src = reinterpret_cast<const uint4*>((i & 1) ? &p.mapB : &p.mapA);
#pragma unroll
  for (int k = 0; k < 8; ++k) reinterpret_cast<uint4*>(m)[k] = src[k];
  asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(__cvta_generic_to_global(m)),
               "r"(s.end)
               : "memory");
  asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
}

template <typename O>
__device__ __forceinline__ float out_to_f(O x);
template <>
__device__ __forceinline__ float out_to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float out_to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float out_to_f<__half>(__half x) { return __half2float(x); }
template <typename O>
__device__ __forceinline__ O f_to_out(float x);
template <>
__device__ __forceinline__ float f_to_out<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 f_to_out<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half f_to_out<__half>(float x) { return __float2half_rn(x); }

// Four consecutive elements of the output, aligned to 4 elements.
template <typename O>
__device__ __forceinline__ float4 load_out4(const O* p) {
  if constexpr (std::is_same<O, float>::value) {
    return *reinterpret_cast<const float4*>(p);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = Elem<O>::unpack2(u.x), b = Elem<O>::unpack2(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
}
template <typename O>
__device__ __forceinline__ void store_out4(O* p, float4 v) {
  if constexpr (std::is_same<O, float>::value) {
    *reinterpret_cast<float4*>(p) = v;
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(Elem<O>::pack2(v.x, v.y), Elem<O>::pack2(v.z, v.w));
  }
}

template <typename T, typename O, int MODE, int NT>
__global__ void __launch_bounds__(THREADS, 1) grouped_kernel(const __grid_constant__ Params p) {
  using Cf = Cfg<O, MODE, NT>;
  constexpr int STAGES = Cf::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * Cf::A_STAGE;
  uint8_t* sEpi = sB + STAGES * Cf::B_STAGE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sEpi + EPI_WARPS * Cf::EPI_BUF);
  uint64_t* full = bars;
  uint64_t* empty = bars + STAGES;
  uint64_t* tfull = bars + 2 * STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* olds = drain + 1;        // DW: blocks to add to have arrived, two per epilogue warp
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(olds + 2 * EPI_WARPS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued_cnt = reinterpret_cast<volatile int*>(tmem_slot + 2);
  // ROWS: first token tile of each expert, the experts' first rows (and the end), then scan scratch
  int* table = reinterpret_cast<int*>(tmem_slot + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();  // 0 = leader
  const int unit = (int)(blockIdx.x >> 1), units = (int)(gridDim.x >> 1);
  auto raise_peer = [&]() { st_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u), 1u); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], EPI_WARPS * 2);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 2 * EPI_WARPS; ++i) mbar_init(&olds[i], 1);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) issued_cnt[i] = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  if (MODE == ROWS && warp == 0 && lane == 0) {
    prefetch_tmap(&p.mapA);
    prefetch_tmap(&p.mapB);
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // barriers initialised in both CTAs
  tc_fence_after();
  // all of the above overlaps the previous launch's end
  grid_dependency_wait();
  grid_dependents_launch();
  const int mt = (p.M + TILE_M - 1) / TILE_M;
  const int ntl = MODE == DW ? (p.N + NT - 1) / NT : 1;
  int total;
  if (MODE == ROWS) {
    // Prefix sum of the experts' token tiles: each thread sums up to three
    // consecutive experts, then warps, then the block.
    constexpr int PER = (kMaxExperts + THREADS - 1) / THREADS;
    int* wsum = table + 2 * kMaxExperts + 1;
    const int e0 = threadIdx.x * PER;
    int c[PER], sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = 0;
      if (e0 + i < p.experts) {
        const Span s = span_of(p, e0 + i);
        bad |= s.begin != __ldg(p.offsets + e0 + i) || s.end != __ldg(p.offsets + e0 + i + 1);
        c[i] = token_tiles<NT>(s.end - s.begin);
        table[kMaxExperts + e0 + i] = s.begin;
        if (e0 + i + 1 == p.experts) table[kMaxExperts + p.experts] = s.end;
      }
      sum += c[i];
    }
    if (bad && blockIdx.x == 0) report(p.status, MUON_ERR_INVALID_ARG);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) wsum[warp] = incl;
    // Offsets that decrease could own more rows than there are, and the sum of
    // their tiles leave 32 bits: nothing is computed for a table that is wrong.
    const bool wrong = __syncthreads_or(bad);
    int base = incl - sum, all = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) base += wsum[w];
      all += wsum[w];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (e0 + i < p.experts) table[e0 + i] = base;
      base += c[i];
    }
    __syncthreads();
    total = wrong ? 0 : all * mt;
  } else {
    total = p.experts * mt * ntl * p.splits;
  }
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t budget = p.timeout_ns;

  if (warp == 0 || warp == 3) {
    // TMA producers: warp 0 the M side (and the leader's byte count), warp 3
    // the N side; both take part in every phase of every stage.
    const uint32_t on = elect_one();
    const bool issues_a = warp == 0;
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    int last_e = -1;
    bool ok = true;
    for (int tile = unit; tile < total && ok; tile += units) {
      const Tile t = decode<MODE, NT>(p, table, tile, mt, ntl);
      const int am0 = t.m0 + (int)rank * BM;
      const int bn0 = t.n0 + (int)rank * (t.n_mma / 2);
      const CUtensorMap* map = issues_a ? &p.mapA : &p.mapB;
      if (MODE == DW) {
        map = p.clipped + 2 * t.e + (issues_a ? 0 : 1);
        if (t.e != last_e && t.nkb > 0) {
          fence_map_acquire(map);
          last_e = t.e;
        }
      }
      for (int kb = 0; kb < t.nkb; ++kb) {
        if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, budget, p.status)) {
          if (on) raise_peer();
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (issues_a && rank == 0) mbar_arrive_expect_tx_if(on, &full[stage], Cf::TX_BYTES);
        uint8_t* a = sA + stage * Cf::A_STAGE;
        uint8_t* b = sB + stage * Cf::B_STAGE;
        const int k0 = kb * BK;
        if (MODE == ROWS) {
          if (!issues_a) {
            tma_load_3d_pair_if(on, b, map, k0, bn0, 0, &full[stage]);
          } else if (!p.a_mn) {
            tma_load_3d_pair_if(on, a, map, k0, am0, t.e, &full[stage]);
          } else if (p.a_one) {
            tma_load_4d_pair_if(on, a, map, 0, k0, am0 >> 6, t.e, &full[stage]);
          } else {
            tma_load_3d_pair_if(on, a, map, am0, k0, t.e, &full[stage]);
            tma_load_3d_pair_if(on, a + 8192, map, am0 + 64, k0, t.e, &full[stage]);
          }
        } else {
          uint8_t* d = issues_a ? a : b;
          const int c0 = issues_a ? am0 : bn0;
          if (issues_a ? p.a_one : p.b_one) {
            tma_load_3d_pair_if(on, d, map, 0, t.t0 + k0, c0 >> 6, &full[stage]);
          } else {
            tma_load_3d_pair_if(on, d, map, c0, t.t0 + k0, 0, &full[stage]);
            tma_load_3d_pair_if(on, d + 8192, map, c0 + 64, t.t0 + k0, 0, &full[stage]);
          }
        }
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    const uint32_t slot = smem_u32(const_cast<int*>(issued_cnt + 2 * rank + (issues_a ? 0 : 1)));
    if (on) st_cluster_u32(mapa_shared(slot, 0), (uint32_t)issued);
  } else if (warp == 1 && rank == 0) {
    // MMA issuer (the leader issues for the pair)
    const uint32_t on = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    const uint32_t a_base = smem_u32(sA), b_base = smem_u32(sB);
    constexpr int fmt = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    const int a_mn = MODE == DW ? 1 : p.a_mn;
    constexpr int b_mn = MODE == DW ? 1 : 0;
    // K-major: 8-row groups 1024 B apart, one K step = 32 B inside the swizzle
    // atom. MN-major: 64-element MN atoms 8 KB apart, 8-row K groups 1024 B
    // apart, one K step of 16 rows = 2048 B.
    const uint32_t a_kstep = a_mn ? 2048u : 32u, b_kstep = b_mn ? 2048u : 32u;
    const uint64_t a_hi = smem_desc_sw128(0, a_mn ? 8192u : 16u, 1024);
    const uint64_t b_hi = smem_desc_sw128(0, b_mn ? 8192u : 16u, 1024);
    bool ok = true;
    for (int tile = unit; tile < total && ok; tile += units) {
      const Tile t = decode<MODE, NT>(p, table, tile, mt, ntl);
      const uint32_t idesc = idesc_f16(fmt, a_mn, b_mn, TILE_M, t.n_mma);
      const int parts = parts_of<MODE, O>(t.nkb);
      for (int part = 0; part < parts && ok; ++part) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&tempty[acc], acc_phase ^ 1, abort_flag, budget, p.status));
        if (!ok) {
          if (on) raise_peer();
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * ACC_COLS;
        const int kb0 = part * kPartBlocks, kb1 = part + 1 < parts ? kb0 + kPartBlocks : t.nkb;
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[stage], phase, abort_flag, budget, p.status));
          if (!ok) {
            if (on) raise_peer();
            break;
          }
          const uint32_t a_lo = (a_base + stage * Cf::A_STAGE) >> 4, b_lo = (b_base + stage * Cf::B_STAGE) >> 4;
#pragma unroll
          for (int k = 0; k < BK / UMMA_K; ++k)
            umma_f16_pair_if(on, d_tmem, a_hi | (uint64_t)(a_lo + k * (a_kstep >> 4)),
                          b_hi | (uint64_t)(b_lo + k * (b_kstep >> 4)), idesc, kb != kb0 || k != 0);
          umma_commit_pair_if(on, &empty[stage], 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        umma_commit_pair_if(on, &tfull[acc], 0x3);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
    }
    umma_commit_pair_if(on, drain, 0x3);
    drain_wait(drain, 0, p.status);
  } else if (warp == 1) {
    drain_wait(drain, 0, p.status);  // the follower: no MMA reads its shared memory or writes its TMEM any more
  } else if (warp >= EPI_WARP0) {
    const int e = warp - EPI_WARP0;
    const int q = warp & 3;   // TMEM lane quarter
    const int half = e >> 2;  // which of the alternating 32-column chunks
    uint8_t* const sd = sEpi + e * Cf::EPI_BUF;
    const uint32_t sd_a = smem_u32(sd);
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t old_phase = 0;  // DW: bit b is the parity of this warp's buffer b
    uint32_t in_flight = 0;  // DW, lane 0: buffers whose block was asked for and not waited for
    // DW: the buffer that the last bulk store did not leave from. A block that
    // is not added to takes it, from tile to tile: one store may still read
    // its source then, and that is the other buffer.
    uint32_t next_buf = 0;
    bool go = true;
    for (int tile = unit; tile < total && go; tile += units) {
      const Tile t = decode<MODE, NT>(p, table, tile, mt, ntl);
      const int parts = parts_of<MODE, O>(t.nkb);
      for (int part = 0; part < parts; ++part) {
        const float beta = part == 0 ? p.beta : 1.f;
        const int r0 = t.m0 + (int)rank * BM + q * 32;  // first M-side row of this warp
        // DW: this warp's 32 x 32 blocks (four, 64 columns apart) go through two
        // buffers: what is added to arrives in one by a bulk copy while the
        // other is worked on, the result replaces it and leaves by a bulk
        // store. Rows and columns out of range are the copies' business.
        const int rows = p.M - r0, z = t.whole ? t.e : tile;
        const int row0 = t.whole ? r0 : r0 - t.m0, col0 = (t.whole ? t.n0 : 0) + half * 32;
        const int blocks = MODE != DW || rows <= 0 || (!t.whole && t.nkb == 0) ? 0 : min(NT / 64, (p.N - t.n0 - half * 32 + 63) / 64);
        const bool adds = MODE == DW && beta != 0.f;
        auto ask = [&](int n) {  // lane 0; the buffer's last store has been read
          mbar_arrive_expect_tx(&olds[2 * e + (n & 1)], Cf::EPI_BLOCK);
          tma_load_3d(sd + (n & 1) * Cf::EPI_BLOCK, &p.mapO, col0 + 64 * n, row0, z, &olds[2 * e + (n & 1)]);
          in_flight |= 1u << (n & 1);
        };
        if (adds && lane == 0) {
          if (part > 0) bulk_wait0(); else bulk_wait_read0();  // a later part adds to what the last one stored
          if (blocks > 0) ask(0);
          if (blocks > 1) ask(1);
        }
        const bool ok = mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, budget, p.status);
        go = __all_sync(0xffffffffu, ok);
        if (!go) {
          if (lane == 0) raise_peer();
          break;
        }
        tc_fence_after();
        const uint32_t trow = tmem_base + ((uint32_t)(q * 32) << 16) + acc * ACC_COLS;
        if (MODE == ROWS) {
          // block: lanes = features r0.., columns = tokens; stored transposed
          O* const out = reinterpret_cast<O*>(p.out);
          for (int c = half * 32; c < t.nvalid; c += 64) {
            if (r0 >= p.M) break;  // warp-uniform
            uint32_t f0[16], f1[16];
            tmem_ld_16x256_x4(trow + c, f0);
            tmem_ld_16x256_x4(trow + c + (16u << 16), f1);
            tmem_wait_ld();
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int x = 4 * i + 2 * k;
                pk[4 * k + i] = Elem<T>::pack2(__uint_as_float(f0[x]), __uint_as_float(f0[x + 1]));
                pk[8 + 4 * k + i] = Elem<T>::pack2(__uint_as_float(f1[x]), __uint_as_float(f1[x + 1]));
              }
            __syncwarp();  // the previous chunk has been read
#pragma unroll
            for (int k = 0; k < 4; ++k)
              stsm_x4_trans(sd_a + sw64(lane, 16 * (k >> 1) + 8 * (k & 1)), pk[4 * k], pk[4 * k + 1], pk[4 * k + 2],
                            pk[4 * k + 3]);
            __syncwarp();
            // rows of 32 features: four lanes a row, 16 bytes a lane
            const int f = r0 + (lane & 3) * 8;
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint4*>(sd + sw64(8 * j + (lane >> 2), (lane & 3) * 8));
            O* d = out + (long long)(t.n0 + c + (lane >> 2)) * p.ldo + f;
            const int left = t.nvalid - c - (lane >> 2);  // tokens from this lane's first row on
            if (f + 8 <= p.M) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (8 * j < left) *reinterpret_cast<uint4*>(d + 8 * j * p.ldo) = v[j];
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const O* h = reinterpret_cast<const O*>(&v[j]);
#pragma unroll
                for (int x = 0; x < 8; ++x)
                  if (8 * j < left && f + x < p.M) d[8 * j * p.ldo + x] = h[x];
              }
            }
          }
        } else {
          // block: lanes = rows of dW_e (or of a part's 256 x 256), columns = its columns
          for (int n = 0; n < blocks; ++n) {
            const uint32_t b = adds ? (uint32_t)(n & 1) : next_buf;  // blocks to add to arrive in turn from buffer 0
            uint8_t* const buf = sd + b * Cf::EPI_BLOCK;
            next_buf = b ^ 1u;
            uint32_t raw[32];
            if (t.nkb > 0) {
              tmem_ld_32x32(trow + half * 32 + 64 * n, raw);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int x = 0; x < 32; ++x) raw[x] = 0u;
            }
            float v[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = p.alpha * __uint_as_float(raw[x]);
            constexpr int V = 16 / sizeof(O);
            if (adds) {
              const bool here = mbar_wait_bounded(&olds[2 * e + b], (old_phase >> b) & 1, abort_flag, budget, p.status);
              go = __all_sync(0xffffffffu, here);
              if (!go) {
                if (lane == 0) raise_peer();
                break;
              }
              old_phase ^= 1u << b;
              in_flight &= ~(1u << b);
#pragma unroll
              for (int k = 0; k < 32 / V; ++k) {
                const uint4 u = *reinterpret_cast<const uint4*>(buf + block_at<O>(lane, k));
                const O* o = reinterpret_cast<const O*>(&u);
#pragma unroll
                for (int x = 0; x < V; ++x) v[V * k + x] = fmaf(beta, out_to_f<O>(o[x]), v[V * k + x]);
              }
            } else {
              if (lane == 0) bulk_wait_read1();  // the store before last has read this buffer
              __syncwarp();
            }
#pragma unroll
            for (int k = 0; k < 32 / V; ++k) {
              uint4 u;
              O* o = reinterpret_cast<O*>(&u);
#pragma unroll
              for (int x = 0; x < V; ++x) o[x] = f_to_out<O>(v[V * k + x]);
              *reinterpret_cast<uint4*>(buf + block_at<O>(lane, k)) = u;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (adds && n > 0 && n + 1 < blocks) {
                bulk_wait_read0();  // the other buffer's store
                ask(n + 1);
              }
              if (!p.by_element) {
                tma_store_3d(&p.mapO, smem_u32(buf), col0 + 64 * n, row0, z);
                bulk_commit();
              }
            }
            if (p.by_element) {
              O* const out = reinterpret_cast<O*>(p.out) + (long long)z * p.so + (long long)row0 * p.ldo + col0 + 64 * n;
              const int cols = p.N - col0 - 64 * n;
              for (int i = lane; i < 32 * (32 / V); i += 32) {
                const int r = i / (32 / V), k = i % (32 / V);
                if (r >= rows || V * k >= cols) continue;
                const uint4 u = *reinterpret_cast<const uint4*>(buf + block_at<O>(r, k));
                const O* o = reinterpret_cast<const O*>(&u);
                O* d = out + (long long)r * p.ldo + V * k;
                if (V * k + V <= cols) *reinterpret_cast<uint4*>(d) = u;
                else
                  for (int x = 0; V * k + x < cols; ++x) d[x] = o[x];
              }
              asm volatile("fence.proxy.async;" ::: "memory");  // a later part reads this by bulk copies
              __syncwarp();
            }
          }
          if (!go) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank != 0) mbar_arrive_remote(mapa_shared(smem_u32(&tempty[acc]), 0));
          else mbar_arrive(&tempty[acc]);
        }
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
    }
    if (MODE == DW && lane == 0)  // after an early stop: no copy still writes here
      for (int b = 0; b < 2; ++b)
        if ((in_flight >> b) & 1) drain_wait(&olds[2 * e + b], (old_phase >> b) & 1, p.status);
  }

  if (MODE == DW && warp >= EPI_WARP0 && lane == 0) bulk_wait0();  // every block is stored
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // no CTA leaves while its pair still signals it
  tc_fence_after();
  if (rank == 0 && threadIdx.x == 0 && *abort_flag) settle_pair_copies<Cf>(full, issued_cnt, p.status);
  __syncwarp();
  cluster_sync();
  if (warp == 2) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// dW = alpha sum of the parts + beta dW: four columns a thread, parts in order.
template <typename O>
__global__ void __launch_bounds__(256) add_parts(const __grid_constant__ Params p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int q = (p.N + 3) / 4;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)p.experts * p.M * q) return;
  const int c = (int)(i % q) * 4;
  const long long er = i / q;
  const int e = (int)(er / p.M), r = (int)(er % p.M);
  const Span s = span_of(p, e);
  const int nkb = (s.end - s.begin + BK - 1) / BK, each = (nkb + p.splits - 1) / p.splits;
  const int mt = (p.M + TILE_M - 1) / TILE_M, ntl = (p.N + 255) / 256;
  const long long tile = ((long long)e * mt + r / TILE_M) * ntl + c / 256;
  const float* src = p.partial + tile * p.splits * (TILE_M * 256) + (r % TILE_M) * 256 + c % 256;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k * each < nkb; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(src + (long long)k * (TILE_M * 256));
    v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
  }
  v.x *= p.alpha; v.y *= p.alpha; v.z *= p.alpha; v.w *= p.alpha;
  O* d = reinterpret_cast<O*>(p.out) + (long long)e * p.so + (long long)r * p.ldo + c;
  if (c + 4 <= p.N) {
    if (p.beta != 0.f) {
      const float4 o = load_out4<O>(d);
      v.x = fmaf(p.beta, o.x, v.x); v.y = fmaf(p.beta, o.y, v.y); v.z = fmaf(p.beta, o.z, v.z); v.w = fmaf(p.beta, o.w, v.w);
    }
    store_out4<O>(d, v);
  } else {
    const float* y = &v.x;
    for (int x = 0; c + x < p.N; ++x) d[x] = f_to_out<O>(p.beta != 0.f ? fmaf(p.beta, out_to_f<O>(d[x]), y[x]) : y[x]);
  }
}

}  // namespace grp

namespace {

constexpr int kMaxDevices = 64;

// Co-resident clusters of one form of the kernel on the current device.
template <typename T, typename O, int MODE, int NT>
int pair_units() {
  static std::mutex mu;
  static int per_device[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> lock(mu);
  int& units = per_device[dev];
  if (units == 0) {
    const void* fn = (const void*)grp::grouped_kernel<T, O, MODE, NT>;
    constexpr int smem = grp::Cfg<O, MODE, NT>::SMEM;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    int u = num_sms() / 2;
    cudaLaunchConfig_t q = {};
    q.gridDim = dim3(2 * u);
    q.blockDim = dim3(grp::THREADS);
    q.dynamicSmemBytes = smem;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = 2;
    a[0].val.clusterDim.y = 1;
    a[0].val.clusterDim.z = 1;
    q.attrs = a;
    q.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, fn, &q) == cudaSuccess && clusters > 0 && clusters < u) u = clusters;
    cudaGetLastError();
    units = u;
  }
  return units;
}

template <typename T, typename O, int MODE, int NT>
muon_status launch_grouped(const grp::Params& p, long long tiles, cudaStream_t s) {  // tiles: at most, to size the grid
  const int units = pair_units<T, O, MODE, NT>();
  if (units <= 0) return MUON_ERR_CUDA;
  const int use = tiles < units ? (int)tiles : units;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * use);
  cfg.blockDim = dim3(grp::THREADS);
  cfg.dynamicSmemBytes = grp::Cfg<O, MODE, NT>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  counters().launches += 1;
  return cudaLaunchKernelEx(&cfg, grp::grouped_kernel<T, O, MODE, NT>, p) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

template <typename T>
muon_status rows_typed(grp::Params& p, int nt, cudaStream_t s) {
  const long long mt = (p.M + grp::TILE_M - 1) / grp::TILE_M;
  const long long tiles = mt * ((p.tokens + nt - 1) / nt + p.experts);  // at least the tiles there are
  switch (nt) {
    case 32: return launch_grouped<T, T, grp::ROWS, 32>(p, tiles, s);
    case 64: return launch_grouped<T, T, grp::ROWS, 64>(p, tiles, s);
    case 128: return launch_grouped<T, T, grp::ROWS, 128>(p, tiles, s);
    default: return launch_grouped<T, T, grp::ROWS, 256>(p, tiles, s);
  }
}

// A small launch that may start while the one before it ends.
template <typename F>
muon_status launch_plain(F* kernel, long long blocks, int threads, const grp::Params& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  counters().launches += 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

// A part of an expert's rows pays for its fp32 sum's way through memory and
// the second launch from about 4 k-blocks (256 rows) on.
constexpr int kMinPartBlocks = 4;
constexpr int kMaxParts = 16;

template <typename T, typename O>
muon_status dw_typed(grp::Params& p, Op out, cudaStream_t s) {
  muon_status r = launch_plain(grp::clip_maps, (2 * p.experts + 127) / 128, 128, p, s);
  if (r != MUON_OK) return r;
  const long long mt = (p.M + grp::TILE_M - 1) / grp::TILE_M, nt = (p.N + 255) / 256, tiles = mt * nt * p.experts;
  const int units = pair_units<T, float, grp::DW, 256>();
  if (units <= 0) return MUON_ERR_CUDA;
  long long parts = units / tiles;
  parts = std::min(parts, (long long)p.tokens / p.experts / (64 * kMinPartBlocks));
  p.splits = (int)std::max(1ll, std::min(parts, (long long)kMaxParts));
  if (p.splits == 1) {
    p.by_element = p.N * (int)sizeof(O) % 16 != 0;
    if (!make_block_store_map(&p.mapO, out, p.out, p.N, p.M, p.experts, p.ldo, p.so)) return MUON_ERR_CUDA;
    return launch_grouped<T, O, grp::DW, 256>(p, tiles, s);
  }
  grp::Params q = p;
  if (!make_block_store_map(&q.mapO, Op::F32, p.partial, 256, grp::TILE_M, tiles * p.splits, 256, grp::TILE_M * 256)) return MUON_ERR_CUDA;
  q.alpha = 1.f;
  q.beta = 0.f;
  r = launch_grouped<T, float, grp::DW, 256>(q, tiles * p.splits, s);
  if (r != MUON_OK) return r;
  const long long quads = (long long)p.experts * p.M * ((p.N + 3) / 4);
  return launch_plain(grp::add_parts<O>, (quads + 255) / 256, 256, p, s);
}

}  // namespace

int grouped_max_experts() { return grp::kMaxExperts; }

bool grouped_fits(const GroupedDesc& g) {
  // the narrowest token tile and both tile counts of the widest direction
  const double mt = (double)((g.n > g.k ? g.n : g.k) / grp::TILE_M + 1);
  const double rows = mt * ((double)g.tokens / 32 + g.experts + 1);
  const double dw = (double)g.experts * (g.n / 256 + 1) * (g.k / 256 + 1);
  return rows < 2147483647.0 && dw < 2147483647.0;
}

// Token tile of a launch: the smallest width that holds twice the average
// group, so that most groups are one tile; wider tiles read each weight fewer
// times, narrower ones keep more stages of weights in flight. Halved while
// that leaves CTA pairs without a tile.
static int token_tile(int64_t tokens, int experts, int64_t mt) {
  const int64_t want = 2 * ((tokens + experts - 1) / experts);
  int nt = want <= 32 ? 32 : want <= 64 ? 64 : want <= 128 ? 128 : 256;
  while (nt > 32 && mt * ((tokens + nt - 1) / nt) * 2 <= num_sms() / 2) nt /= 2;
  return nt;
}

muon_status grouped_rows(const GroupedDesc& g, const void* x, const void* w, void* y, bool mn, uint64_t timeout_ns,
                         cudaStream_t s) {
  // mn: dx = dy W (x holds dy, y holds dx), else y = x W^T
  grp::Params p;
  memset(&p, 0, sizeof(p));
  p.M = (int)(mn ? g.k : g.n);
  p.K = (int)(mn ? g.n : g.k);
  const int64_t ldi = mn ? g.ldy : g.ldx;
  p.ldo = mn ? g.ldx : g.ldy;
  const int nt = token_tile(g.tokens, g.experts, (p.M + grp::TILE_M - 1) / grp::TILE_M);
  p.a_one = mn && g.k % 64 == 0;
  const bool made = p.a_one ? make_block_map(&p.mapA, g.type, w, g.k, g.n, g.experts, g.ldw, g.w_stride)
                            : make_tensor_map(&p.mapA, g.type, w, g.k, g.n, g.experts, g.ldw, g.w_stride, mn ? 64 : grp::BM);
  if (!made) return MUON_ERR_CUDA;
  if (!make_tensor_map(&p.mapB, g.type, x, p.K, g.tokens, 1, ldi, 0, nt / 2)) return MUON_ERR_CUDA;
  p.offsets = g.offsets;
  p.out = y;
  p.tokens = (int)g.tokens;
  p.experts = g.experts;
  p.a_mn = mn ? 1 : 0;
  const unsigned mt = (unsigned)((p.M + grp::TILE_M - 1) / grp::TILE_M);
  p.mt_inverse = (unsigned)((0x100000000ull + mt - 1) / mt);  // not used for mt = 1
  p.status = g.status;
  p.timeout_ns = timeout_ns;
  return g.type == Op::BF16 ? rows_typed<__nv_bfloat16>(p, nt, s) : rows_typed<__half>(p, nt, s);
}

// The maps of every expert, and one part's sum per CTA pair.
static size_t maps_bytes(int experts) { return ((size_t)experts * 2 * sizeof(CUtensorMap) + 1023) / 1024 * 1024; }
size_t grouped_ws(int experts) {
  return 1024 + maps_bytes(experts) + (size_t)(num_sms() / 2) * grp::TILE_M * 256 * sizeof(float);
}

muon_status grouped_dw(const GroupedDesc& g, const void* dy, const void* x, void* dw, Op out, float alpha, float beta,
                       void* ws, uint64_t timeout_ns, cudaStream_t s) {
  grp::Params p;
  memset(&p, 0, sizeof(p));
  p.M = (int)g.n;
  p.N = (int)g.k;
  if (g.tokens > 0) {  // without rows no copy reads the maps
    p.a_one = g.n % 64 == 0;
    p.b_one = g.k % 64 == 0;
    if (!(p.a_one ? make_block_map(&p.mapA, g.type, dy, g.n, g.tokens, 0, g.ldy, 0)
                  : make_tensor_map(&p.mapA, g.type, dy, g.n, g.tokens, 1, g.ldy, 0, 64)) ||
        !(p.b_one ? make_block_map(&p.mapB, g.type, x, g.k, g.tokens, 0, g.ldx, 0)
                  : make_tensor_map(&p.mapB, g.type, x, g.k, g.tokens, 1, g.ldx, 0, 64)))
      return MUON_ERR_CUDA;
  }
  const uintptr_t base = (reinterpret_cast<uintptr_t>(ws) + 1023) & ~uintptr_t(1023);
  p.clipped = reinterpret_cast<CUtensorMap*>(base);
  p.partial = reinterpret_cast<float*>(base + maps_bytes(g.experts));
  p.offsets = g.offsets;
  p.out = dw;
  p.ldo = g.ldw;
  p.so = g.w_stride;
  p.tokens = (int)g.tokens;
  p.experts = g.experts;
  p.alpha = alpha;
  p.beta = beta;
  p.status = g.status;
  p.timeout_ns = timeout_ns;
  if (g.type == Op::BF16)
    return out == Op::F32 ? dw_typed<__nv_bfloat16, float>(p, out, s) : dw_typed<__nv_bfloat16, __nv_bfloat16>(p, out, s);
  return out == Op::F32 ? dw_typed<__half, float>(p, out, s) : dw_typed<__half, __half>(p, out, s);
}

}  // namespace muon
