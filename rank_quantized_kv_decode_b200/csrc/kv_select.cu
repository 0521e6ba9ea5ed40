// Choice of pages for sparse attention over the plain key-value cache.
//
// Mathematics: a key inside the bounds lo <= k <= hi of its page has q.k <= sum_c max(q_c lo_c, q_c hi_c)
// = q+.hi + q-.lo (q split into its positive and negative channels); the score of a page is the largest
// such sum over the query heads of its KV head.  The choice is that of scores in fp64, where 16-bit
// factors have exact products and sums of 64 or 128 of them are exact or nearly so: it does not
// hang on the order of a summation, and equal pages score equally.
//
// Two steps give that choice at the cost of fp32.  (1) All scores in fp32 on mma.sync (16 pages and all
// heads of a KV head a round, 4 d / 16 products), with a bound e of their error.  (2) With v the n-th
// largest, the n-th largest exact score lies within e of v: pages above v + 2 e are in, pages below
// v - 2 e are out, and only those between are scored again in fp64 and ranked.  fp64 throughout
// took 65 us at 32 sequences x 512 pages x 8 KV heads (170 registers, one CTA per SM).
//
// Bound: HBM for large batches (the bounds are 4 d bytes per page and KV head, read once), latency
// for one sequence.  A cluster of CTAs shares one (sequence, KV head): each scores its share of the
// pages into the first CTA's shared memory, which then chooses.
#include <cooperative_groups.h>

#include "kv.cuh"

namespace starkv {
namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
// Error of an fp32 score over S = sum |q_c| |b_c|: d / 8 products of 16 terms accumulate, each losing at
// most 17 x 2^-24 of the running magnitude (<= S) where the unit cuts instead of rounding: 16 x 17 x
// 2^-24 < 2^-15.9 at d = 128.
constexpr float kScoreError = 1.f / 32768.f;
constexpr int kRankAll = 256;  // pages between that are ranked by comparing all pairs

template <bool BF>
__device__ __forceinline__ void mma_score(float (&c)[4], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1));
}

// The negative 16-bit halves of a word, and the rest.
__device__ __forceinline__ uint32_t negatives(uint32_t w) {
  const uint32_t s = (w >> 15) & 0x00010001u;
  return w & (s * 0xffffu);
}

// Larger magnitude of two pairs of 16-bit values (sign bit dropped: their order is that of the bits).
__device__ __forceinline__ uint32_t max_mag(uint32_t a, uint32_t w) { return __vmaxu2(a, w & 0x7fff7fffu); }

// A 16-bit value as a double times 2^-896 (bf16) or 2^-1008 (fp16), by moving its exponent and
// mantissa fields into place: exact, subnormals included.
template <int F>
__device__ __forceinline__ double field_double(uint32_t high16) {  // the value in the upper half
  const int w = static_cast<int>(high16);
  return F == STARKV_KV_F16 ? __hiloint2double((w >> 6) & 0x81ffffff, 0)
                            : __hiloint2double((w >> 3) & 0x8fffffff, 0);
}

// Order-preserving maps of floating values to unsigned integers, and back.
__device__ __forceinline__ unsigned long long order_key(double x) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
}

// Exact score of a page (whole warp): the sum scaled by a power of two, the same for all pages.
template <int F, int D>
__device__ double exact_score(const KvPool& P, const uint16_t* q, int G, const uint8_t* bounds, int lane) {
  constexpr int W = D / 64;  // words (channel pairs) of a lane
  double best = -__longlong_as_double(0x7ff0000000000000ll);
  const uint32_t* lo = reinterpret_cast<const uint32_t*>(bounds) + lane * W;
  uint32_t l[W], u[W];
#pragma unroll
  for (int i = 0; i < W; ++i) l[i] = lo[i], u[i] = lo[D / 2 + i];
  // undoes field_double's factor, up to a power of two that keeps the largest query finite
  const double up = __hiloint2double((1023 + (F == STARKV_KV_F16 ? 1000 : 880)) << 20, 0);
  for (int h = 0; h < G; ++h) {
    double a = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 x = kv_unpack<F>(reinterpret_cast<const uint32_t*>(q + h * D)[lane * W + i]);
      a = fma(x.x * up, field_double<F>((x.x < 0.f ? l[i] : u[i]) << 16), a);
      a = fma(x.y * up, field_double<F>((x.y < 0.f ? l[i] : u[i]) & 0xffff0000u), a);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    best = fmax(best, a);
  }
  return best;
}

template <int F, int D>
__global__ void __launch_bounds__(kSelThreads, 2) kv_select_kernel(const KvSelectParams p) {
  constexpr int NJ = D / 32;   // 16-byte loads per row and lane
  constexpr int RP = 16;       // pages of a warp's round
  extern __shared__ __align__(16) uint8_t smem[];
  const KvPool& P = p.pool;
  // in the cluster's first CTA: exact keys of the pages between, fp32 keys of all, the pages between
  unsigned long long* keys64 = reinterpret_cast<unsigned long long*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(keys64 + P.max_pages);
  uint16_t* list = reinterpret_cast<uint16_t*>(keys + P.max_pages);
  __shared__ uint32_t s_mag[8];      // largest magnitude of a bound, per CTA of the cluster
  __shared__ uint32_t s_cnt[2][2][kSelWarps];
  __shared__ uint32_t s_ext[2][kSelWarps];
  __shared__ float s_q1[kSelWarps];
  __shared__ int s_m, s_in;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x % p.cluster, unit = blockIdx.x / p.cluster;
  const int b = unit / P.Hkv, g = unit % P.Hkv, G = P.H / P.Hkv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, row = lane / 4, t = lane % 4;
  pdl_wait();
  pdl_launch_dependents();
  const int raw = p.seq_lens[b];
  const int len = min(max(raw, 0), P.max_pages * kPage);
  const int pages = (len + kPage - 1) / kPage;
  if (threadIdx.x == 0 && rank == 0 && g == 0 && raw != len) atomicOr(P.status, STARKV_DEV_BOUNDS);
  int* sel = p.sel + (long long)unit * p.n_sel;
  if (pages <= p.n_sel) {  // the same for the whole cluster
    if (rank == 0)
      for (int i = threadIdx.x; i < p.n_sel; i += kSelThreads) sel[i] = i < pages ? i : -1;
    return;
  }
  const int c0 = p.keep_first, nc = pages - p.keep_first - p.keep_last;  // candidates [c0, c0 + nc)
  const int want = p.n_sel - p.keep_first - p.keep_last;
  const uint16_t* q = p.q + ((long long)b * P.H + g * G) * D;
  if (want == 0) {
    if (rank == 0)
      for (int i = threadIdx.x; i < p.n_sel; i += kSelThreads)
        sel[i] = i < p.keep_first ? i : pages - p.n_sel + i;
    return;
  }

  // ---- fp32 scores
  {
    uint32_t* first = cluster.map_shared_rank(keys, 0);
    uint32_t mag = 0;
    for (int h0 = 0; h0 < G; h0 += 8) {
      // A fragments: row = head (a head beyond the last stands twice), the lane's channels 8 (t + 4 j) + 0..7
      uint32_t qp[NJ][4], qn[NJ][4];
      const uint16_t* src = q + min(h0 + row, G - 1) * D + 8 * t;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + 32 * j);
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qn[j][i] = negatives(a[i]);
          qp[j][i] = a[i] ^ qn[j][i];
        }
      }
      for (int i0 = (rank * kSelWarps + warp) * RP; i0 < nc; i0 += p.cluster * kSelWarps * RP) {
        uint4 lo[2][NJ], hi[2][NJ];
        bool have[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = i0 + 8 * k + row;
          const uint8_t* page = i < nc ? kv_page(P, b, c0 + i) : nullptr;
          have[k] = page != nullptr;
          if (!page && i < nc && t == 0) atomicOr(P.status, STARKV_DEV_BOUNDS);
          const uint4* x = reinterpret_cast<const uint4*>(page + (long long)g * 4 * D) + t;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            lo[k][j] = page ? x[4 * j] : make_uint4(0, 0, 0, 0);
            hi[k][j] = page ? x[4 * j + D / 8] : make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float c[4] = {}, z[4] = {};
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const uint4 x = lo[k][j], y = hi[k][j];
            mma_score<F == STARKV_KV_BF16>(c, qp[j][0], qp[j][1], y.x, y.y);
            mma_score<F == STARKV_KV_BF16>(z, qn[j][0], qn[j][1], x.x, x.y);
            mma_score<F == STARKV_KV_BF16>(c, qp[j][2], qp[j][3], y.z, y.w);
            mma_score<F == STARKV_KV_BF16>(z, qn[j][2], qn[j][3], x.z, x.w);
            mag = max_mag(max_mag(max_mag(max_mag(mag, x.x), x.y), x.z), x.w);
            mag = max_mag(max_mag(max_mag(max_mag(mag, y.x), y.y), y.z), y.w);
          }
          // the largest over the heads (rows): lanes t = 0..3 of row 0 hold pages 2t, 2t + 1
          float s0 = c[0] + z[0], s1 = c[1] + z[1];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            s0 = fmaxf(s0, __shfl_xor_sync(0xffffffffu, s0, o));
            s1 = fmaxf(s1, __shfl_xor_sync(0xffffffffu, s1, o));
          }
          const unsigned ok = __ballot_sync(0xffffffffu, have[k]);  // page r: lanes 4r .. 4r + 3
          if (row == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int pg = 2 * t + e, i = i0 + 8 * k + pg;
              if (i >= nc) continue;
              uint32_t key = ok >> (4 * pg) & 1 ? max(order_key(e ? s1 : s0), 1u) : 0u;  // 0: no page
              if (h0 > 0) key = max(key, first[i]);  // written by this thread for the heads before
              first[i] = key;
            }
          }
        }
      }
    }
    mag = max(mag & 0xffffu, mag >> 16);
    mag = __reduce_max_sync(0xffffffffu, mag);
    if (lane == 0) s_ext[0][warp] = mag;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) mag = max(mag, s_ext[0][w]);
      *cluster.map_shared_rank(&s_mag[rank], 0) = mag;
    }
  }
  cluster.sync();
  if (rank != 0) return;

  // ---- error bound: kScoreError times the largest sum |q_c| of a head times the largest |bound|
  {
    float q1 = 0.f;
    for (int h = warp; h < G; h += kSelWarps) {
      float a = 0.f;
      for (int c = lane; c < D / 2; c += 32) {
        const float2 x = kv_unpack<F>(reinterpret_cast<const uint32_t*>(q + h * D)[c]);
        a += fabsf(x.x) + fabsf(x.y);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
      q1 = fmaxf(q1, a);
    }
    if (lane == 0) s_q1[warp] = q1;
    if (threadIdx.x == 0) s_m = 0, s_in = 0;
  }
  // sums over the CTA, two buffers in turn: one barrier each
  int buf = 0;
  auto total2 = [&](uint32_t x, uint32_t y, uint32_t& sx, uint32_t& sy) {
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    if (lane == 0) s_cnt[buf][0][warp] = x, s_cnt[buf][1][warp] = y;
    __syncthreads();
    sx = sy = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) sx += s_cnt[buf][0][w], sy += s_cnt[buf][1][w];
    buf ^= 1;
  };

  // ---- v, the want-th largest fp32 key: two bits a round from the first that differs
  uint32_t vkey;
  {
    uint32_t mn = 0xffffffffu, mx = 0;
    for (int i = threadIdx.x; i < nc; i += kSelThreads) mn = min(mn, keys[i]), mx = max(mx, keys[i]);
    mn = __reduce_min_sync(0xffffffffu, mn), mx = __reduce_max_sync(0xffffffffu, mx);
    if (lane == 0) s_ext[0][warp] = mn, s_ext[1][warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) mn = min(mn, s_ext[0][w]), mx = max(mx, s_ext[1][w]);
    uint32_t thr = mx;
    int high = 31 - __clz(mn ^ mx);  // -1: all equal
    if (high >= 0) {
      high |= 1;  // whole pairs of bits
      thr = high < 31 ? mx & ~((2u << high) - 1) : 0u;
      bool done = false;
      for (int bit = high - 1; bit >= 0 && !done; bit -= 2) {
        const uint32_t t1 = thr | 1u << bit, t2 = thr | 2u << bit, t3 = thr | 3u << bit;
        uint32_t n12 = 0, n3 = 0;  // at most 16384 keys: two counts in a word
        for (int i = threadIdx.x; i < nc; i += kSelThreads) {
          const uint32_t k = keys[i];
          n12 += (k >= t1) + ((k >= t2) << 16);
          n3 += k >= t3;
        }
        uint32_t s12, s3;
        total2(n12, n3, s12, s3);
        const uint32_t s1 = s12 & 0xffffu, s2 = s12 >> 16, w = want;
        thr = s3 >= w ? t3 : s2 >= w ? t2 : s1 >= w ? t1 : thr;
        done = s1 == w || s2 == w || s3 == w;  // the chosen one has exactly `want` keys
      }
    }
    mn = 0xffffffffu;
    for (int i = threadIdx.x; i < nc; i += kSelThreads)
      if (keys[i] >= thr) mn = min(mn, keys[i]);
    mn = __reduce_min_sync(0xffffffffu, mn);
    __syncthreads();
    if (lane == 0) s_ext[0][warp] = mn;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) mn = min(mn, s_ext[0][w]);
    vkey = mn;
  }

  // ---- in, out or between
  {
    uint32_t mag = 0;
    for (int r = 0; r < p.cluster; ++r) mag = max(mag, s_mag[r]);
    float q1 = 0.f;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) q1 = fmaxf(q1, s_q1[w]);
    const float e2 = 2.f * kScoreError * q1 * kv_unpack<F>(mag).x;
    // a bad page has key 0, below every score; where v itself is one, they all tie
    const float v = vkey ? key_value(vkey) : 0.f;
    for (int i = threadIdx.x; i < nc; i += kSelThreads) {
      const uint32_t k = keys[i];
      const float s = key_value(k);
      const bool in = vkey == 0 ? k > 0 : (k > 0 && s > v + e2);
      const bool out = vkey == 0 ? false : (k == 0 || s < v - e2);
      keys[i] = in ? 0xffffffffu : 0u;
      if (in) atomicAdd(&s_in, 1);
      if (!in && !out) list[atomicAdd(&s_m, 1)] = static_cast<uint16_t>(i);
    }
  }
  __syncthreads();
  const int m = s_m, need = want - s_in;  // 1 <= need <= m
  for (int e = warp; e < m; e += kSelWarps) {
    const uint8_t* page = kv_page(P, b, c0 + list[e]);
    const double x = page ? exact_score<F, D>(P, q, G, page + (long long)g * 4 * D, lane) : 0.0;
    if (lane == 0) keys64[e] = page ? order_key(x) : 0ull;
  }
  __syncthreads();
  if (m <= kRankAll) {
    if ((int)threadIdx.x < m) {
      const unsigned long long k = keys64[threadIdx.x];
      const int i = list[threadIdx.x];
      int before = 0;
      for (int e = 0; e < m; ++e) before += keys64[e] > k || (keys64[e] == k && list[e] < i);
      if (before < need) keys[i] = 0xffffffffu;
    }
  } else {
    // many pages tie (or nearly): the need-th largest exact key, then the lowest pages at it
    unsigned long long thr = 0;
    uint32_t n, dummy;
    bool exact = false;
    for (int bit = 63; bit >= 0 && !exact; --bit) {
      const unsigned long long cand = thr | 1ull << bit;
      n = 0;
      for (int e = threadIdx.x; e < m; e += kSelThreads) n += keys64[e] >= cand;
      total2(n, 0, n, dummy);
      if ((int)n >= need) thr = cand;
      exact = (int)n == need;
    }
    n = 0;
    for (int e = threadIdx.x; e < m; e += kSelThreads) n += keys64[e] > thr;
    total2(n, 0, n, dummy);
    const int at = need - static_cast<int>(n);  // pages to take at thr
    int bound = 0;                              // those with an index below the largest bound that holds <= at
    for (int bit = 14; bit >= 0; --bit) {
      const int cand = bound | 1 << bit;
      n = 0;
      for (int e = threadIdx.x; e < m; e += kSelThreads) n += keys64[e] == thr && list[e] < cand;
      total2(n, 0, n, dummy);
      if ((int)n <= at) bound = cand;
    }
    for (int e = threadIdx.x; e < m; e += kSelThreads)
      if (keys64[e] > thr || (keys64[e] == thr && list[e] < bound)) keys[list[e]] = 0xffffffffu;
  }
  __syncthreads();

  // ---- the chosen pages in order: a thread takes a run of candidates
  const int per = (nc + kSelThreads - 1) / kSelThreads, i0 = min((int)threadIdx.x * per, nc), i1 = min(i0 + per, nc);
  int mine = 0;
  for (int i = i0; i < i1; ++i) mine += keys[i] != 0;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_cnt[buf][0][warp] = inc;
  __syncthreads();
  int at = c0 + inc - mine;
  for (int w = 0; w < warp; ++w) at += s_cnt[buf][0][w];
  for (int i = i0; i < i1; ++i)
    if (keys[i]) sel[at++] = c0 + i;
  for (int i = threadIdx.x; i < p.keep_first; i += kSelThreads) sel[i] = i;
  for (int i = threadIdx.x; i < p.keep_last; i += kSelThreads) sel[p.n_sel - p.keep_last + i] = pages - p.keep_last + i;
}

constexpr int select_smem(int max_pages) { return max_pages * (8 + 4 + 2); }

template <int F, int D>
cudaError_t select_launch(const KvSelectParams& p, cudaStream_t s) {
  auto kern = kv_select_kernel<F, D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       select_smem(STARKV_KV_MAX_SELECT_PAGES));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.pool.batch * p.pool.Hkv * p.cluster));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(select_smem(p.pool.max_pages));
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_kv_select(const KvSelectParams& p, cudaStream_t s) {
  const int d = p.pool.d;
  if (p.pool.fmt == STARKV_KV_F16)
    return d == 64 ? select_launch<STARKV_KV_F16, 64>(p, s) : select_launch<STARKV_KV_F16, 128>(p, s);
  return d == 64 ? select_launch<STARKV_KV_BF16, 64>(p, s) : select_launch<STARKV_KV_BF16, 128>(p, s);
}

}  // namespace starkv
