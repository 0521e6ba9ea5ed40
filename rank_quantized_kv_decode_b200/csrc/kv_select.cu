// Choice of pages for sparse attention over the plain key-value cache.
//
// Mathematics: a key inside the bounds lo <= k <= hi of its page has q.k <= sum_c max(q_c lo_c, q_c hi_c)
// = q+.hi + q-.lo (q split into its positive and negative channels); the score of a page is the largest
// such sum over the query heads of its KV head.  The choice is that of scores in fp64, where 16-bit
// factors have exact products and sums of 64 or 128 of them are exact or nearly so: it does not
// hang on the order of a summation, and equal pages score equally.
//
// Two steps give that choice at the cost of fp32.  (1) All scores in fp32 on mma.sync (16 pages and all
// heads of a KV head a round, 4 d / 16 products), with a bound e of their error.  (2) A histogram finds
// the bin [v0, v1] of the n-th largest; the n-th largest exact score lies in [v0 - e, v1 + e], so pages
// above v1 + 2 e are in, pages below v0 - 2 e are out, and only those between (a few) are scored again in
// fp64 and ranked.  fp64 throughout took 65 us at 32 sequences x 512 pages x 8 KV heads; finding the n-th
// largest bit by bit 4 us of a sequence's 17, the histogram 1.
//
// Bound: HBM for large batches (the bounds are 4 d bytes per page and KV head, read once), latency
// for one sequence.  32 sequences x 512 pages x 8 KV heads take 25.4 us in a graph (67 MB, 10 us at the
// measured copy rate; 24.5 where they are in L2 already): 14 until all is scored, then 6 for the choice; one
// sequence of 2047 pages 12.5.  Bounds through a cp.async ring, always two rounds in flight, scored no faster
// (26 to 30 us).  A cluster of CTAs shares one
// (sequence, KV head): each scores its share of the pages into the first CTA's shared memory, which then
// chooses.
#include <cooperative_groups.h>

#include <utility>

#include "kv.cuh"

namespace starkv {
namespace {

constexpr int kSelThreads = 128;
constexpr int kBins = 1024;
constexpr int kSelWarps = kSelThreads / 32;
// Error of an fp32 score over S = sum |q_c| |b_c|: d / 8 products of 16 terms accumulate, each losing at
// most 17 x 2^-24 of the running magnitude (<= S) where the unit cuts instead of rounding: 16 x 17 x
// 2^-24 < 2^-15.9 at d = 128.
constexpr float kScoreError = 1.f / 32768.f;
// And at the ends of fp32's range: 2 d products and as many sums, each off by at most 2^-126 where they are
// subnormal (2^9 x 2^-126); where a sum could pass 2^127 the error has no bound, and all pages are scored again.
constexpr float kScoreFloor = 0x1p-117f, kScoreMost = 0x1p126f;
constexpr int kRankAll = kSelThreads;  // pages between that are ranked by comparing all pairs

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

// Shared memory of a CTA: exact keys or the histogram, fp32 keys, list of pages.
__host__ __device__ constexpr int exact_bytes(int max_pages) { return max_pages * 8 > kBins * 4 ? max_pages * 8 : kBins * 4; }
constexpr int select_smem(int max_pages) { return exact_bytes(max_pages) + max_pages * (4 + 2); }

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

// Exact bound of one query head over a page, scaled by a power of two, the same for all pages: eight
// lanes, D / 8 channels each (part = lane % 8); the whole warp shuffles.
template <int F, int D>
__device__ __forceinline__ double exact_bound(const uint16_t* q, const uint8_t* bounds, int part) {
  constexpr int W = D / 64;  // 16-byte loads of a lane
  // undoes field_double's factor, up to a power of two that keeps the largest query finite
  const double up = __hiloint2double((1023 + (F == STARKV_KV_F16 ? 1000 : 880)) << 20, 0);
  double a = 0.0, z = 0.0;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const uint4 l4 = reinterpret_cast<const uint4*>(bounds)[8 * j + part];
    const uint4 u4 = reinterpret_cast<const uint4*>(bounds)[8 * j + part + D / 8];
    const uint4 q4 = reinterpret_cast<const uint4*>(q)[8 * j + part];
    const uint32_t l[4] = {l4.x, l4.y, l4.z, l4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w}, w[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = kv_unpack<F>(w[i]);
      a = fma(x.x * up, field_double<F>((x.x < 0.f ? l[i] : u[i]) << 16), a);
      z = fma(x.y * up, field_double<F>((x.y < 0.f ? l[i] : u[i]) & 0xffff0000u), z);
    }
  }
  a += z;
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a;
}

// Flags bad ones of n entries of a sequence's block table from the i0-th (whole CTA): those that no scoring
// looks at.
__device__ __forceinline__ void flag_unscored(const KvPool& P, int b, int i0, int n) {
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    const int pg = P.block_table[(long long)b * P.max_pages + i0 + i];
    if (pg < 0 || pg >= P.num_pages) atomicOr(P.status, STARKV_DEV_BOUNDS);
  }
}

template <int F, int D>
__global__ void __launch_bounds__(kSelThreads, 4) kv_select_kernel(const KvSelectParams p) {
  constexpr int NJ = D / 32;   // 16-byte loads per row and lane
  constexpr int RP = 16;       // pages of a warp's round
  extern __shared__ __align__(16) uint8_t smem[];
  const KvPool& P = p.pool;
  // in the cluster's first CTA: exact keys of the pages between (before them the histogram), fp32 keys
  // of all pages, the pages between
  unsigned long long* keys64 = reinterpret_cast<unsigned long long*>(smem);
  int* s_bins = reinterpret_cast<int*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + exact_bytes(P.max_pages));
  uint16_t* list = reinterpret_cast<uint16_t*>(keys + P.max_pages);
  __shared__ uint32_t s_mag[kSelMaxCluster];  // largest magnitude of a bound, per CTA of the cluster
  __shared__ uint32_t s_cnt[2][kSelWarps];
  __shared__ uint32_t s_ext[2][kSelWarps];
  __shared__ int s_m, s_in, s_bin;
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x % p.cluster, unit = blockIdx.x / p.cluster;
  const int b = unit / P.Hkv, g = unit % P.Hkv, G = P.H / P.Hkv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, row = lane / 4, t = lane % 4;
  auto started = cluster.barrier_arrive();
  pdl_wait();
  pdl_launch_dependents();
  const int raw = p.seq_lens[b];
  const int len = min(max(raw, 0), P.max_pages * kPage);
  const int pages = (len + kPage - 1) / kPage;
  if (threadIdx.x == 0 && rank == 0 && g == 0 && raw != len) atomicOr(P.status, STARKV_DEV_BOUNDS);
  int* sel = p.sel + (long long)unit * p.n_sel;
  if (pages <= p.n_sel) {  // the same for the whole cluster
    if (rank == 0) {
      for (int i = threadIdx.x; i < p.n_sel; i += kSelThreads) sel[i] = i < pages ? i : -1;
      if (g == 0) flag_unscored(P, b, 0, pages);
    }
    return;
  }
  const int c0 = p.keep_first, nc = pages - p.keep_first - p.keep_last;  // candidates [c0, c0 + nc)
  const int want = p.n_sel - p.keep_first - p.keep_last;
  const uint16_t* q = p.q + ((long long)b * P.H + g * G) * D;
  if (want == 0) {
    if (rank == 0) {
      for (int i = threadIdx.x; i < p.n_sel; i += kSelThreads)
        sel[i] = i < p.keep_first ? i : pages - p.n_sel + i;
      if (g == 0) flag_unscored(P, b, 0, pages);
    }
    return;
  }

  // ---- fp32 scores, and the largest sum |q_c| of a head (every warp for itself)
  float q1 = 0.f;
  {
    cluster.barrier_wait(std::move(started));  // the first CTA's shared memory is there once it has started
    uint32_t* first = cluster.map_shared_rank(keys, 0);
    uint32_t mag = 0;
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) s_bins[i] = 0;
    for (int h0 = 0; h0 < G; h0 += 8) {
      // A fragments: row = head (a head beyond the last stands twice), the lane's channels 8 (t + 4 j) + 0..7
      uint32_t qp[NJ][4], qn[NJ][4];
      float head_sum = 0.f;
      const uint16_t* src = q + min(h0 + row, G - 1) * D + 8 * t;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + 32 * j);
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qn[j][i] = negatives(a[i]);
          qp[j][i] = a[i] ^ qn[j][i];
          const float2 x = kv_unpack<F>(a[i]);
          head_sum += fabsf(x.x) + fabsf(x.y);
        }
      }
      head_sum += __shfl_xor_sync(0xffffffffu, head_sum, 1);
      head_sum += __shfl_xor_sync(0xffffffffu, head_sum, 2);
      q1 = fmaxf(q1, head_sum);
      const int step = p.cluster * kSelWarps * RP;
      const int* table = P.block_table + (long long)b * P.max_pages + c0;
      int i0 = (rank * kSelWarps + warp) * RP, pid[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) pid[k] = i0 + 8 * k + row < nc ? table[i0 + 8 * k + row] : 0;
      for (; i0 < nc; i0 += step) {
        uint4 lo[2][NJ], hi[2][NJ];
        bool have[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool in = i0 + 8 * k + row < nc;
          have[k] = in && pid[k] >= 0 && pid[k] < P.num_pages;
          if (in && !have[k] && t == 0) atomicOr(P.status, STARKV_DEV_BOUNDS);
          const uint4* x = reinterpret_cast<const uint4*>(P.cache + pid[k] * P.page_bytes + (long long)g * 4 * D) + t;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            lo[k][j] = have[k] ? x[4 * j] : make_uint4(0, 0, 0, 0);
            hi[k][j] = have[k] ? x[4 * j + D / 8] : make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)  // the next round's pages
          if (i0 + step + 8 * k + row < nc) pid[k] = table[i0 + step + 8 * k + row];
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
  if (g == 0 && rank == p.cluster - 1) {  // the ends, which are always taken
    flag_unscored(P, b, 0, p.keep_first);
    flag_unscored(P, b, pages - p.keep_last, p.keep_last);
  }
  if (rank != 0) return;

  // ---- the bin of the want-th largest key
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) q1 = fmaxf(q1, __shfl_xor_sync(0xffffffffu, q1, o));
  uint32_t mn = 0xffffffffu, mx = 0;
  for (int i = threadIdx.x; i < nc; i += kSelThreads) mn = min(mn, keys[i]), mx = max(mx, keys[i]);
  mn = __reduce_min_sync(0xffffffffu, mn), mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) s_ext[0][warp] = mn, s_ext[1][warp] = mx;
  if (threadIdx.x == 0) s_m = 0, s_in = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) mn = min(mn, s_ext[0][w]), mx = max(mx, s_ext[1][w]);
  // the first shift by which all keys fall into kBins bins
  const int shift = max(0, 32 - __clz(mx - mn) - (31 - __clz(kBins)));
  for (int i = threadIdx.x; i < nc; i += kSelThreads) atomicAdd(&s_bins[(keys[i] - mn) >> shift], 1);
  __syncthreads();
  {
    constexpr int kOf = kBins / kSelThreads;  // bins of a thread, from the highest
    int bins[kOf], sum = 0;
#pragma unroll
    for (int i = 0; i < kOf; ++i) sum += bins[i] = s_bins[kBins - 1 - (kOf * threadIdx.x + i)];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) s_cnt[0][warp] = inc;
    __syncthreads();
    int above = inc - sum;
    for (int w = 0; w < warp; ++w) above += s_cnt[0][w];
    if (above < want && want <= above + sum) {  // one thread
      int i = 0;
      for (; above + bins[i] < want; ++i) above += bins[i];
      s_bin = kBins - 1 - (kOf * threadIdx.x + i);
    }
    __syncthreads();
  }

  // ---- in, out or between
  {
    const uint32_t k0 = mn + (static_cast<uint32_t>(s_bin) << shift), width = (1u << shift) - 1;
    const uint32_t k1 = mx - k0 < width ? mx : k0 + width;  // the bin's keys: [k0, k1]
    uint32_t mag = 0;
    for (int r = 0; r < p.cluster; ++r) mag = max(mag, s_mag[r]);
    const float most = q1 * kv_unpack<F>(mag).x;  // no product or sum of a score is larger
    const float e2 = most < kScoreMost ? 2.f * (kScoreError * most + kScoreFloor) : __int_as_float(0x7f800000);
    const float v0 = key_value(max(k0, 1u)), v1 = key_value(max(k1, 1u));
    int ins = 0;
    constexpr int kAt = 4;  // keys a thread has in hand
    for (int i0 = threadIdx.x; i0 < nc; i0 += kAt * kSelThreads) {
      uint32_t k[kAt];
#pragma unroll
      for (int j = 0; j < kAt; ++j) k[j] = i0 + j * kSelThreads < nc ? keys[i0 + j * kSelThreads] : 0u;
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const int i = i0 + j * kSelThreads;
        if (i >= nc) break;
        const float x = key_value(k[j]);
        // a bad page has key 0, below every score: among themselves they tie, and are between where the
        // bin reaches down to them
        const bool in = k[j] > k1 && x > v1 + e2;
        const bool out = k[j] == 0 ? k0 > 0 : (k[j] < k0 && x < v0 - e2);
        keys[i] = in ? 0xffffffffu : 0u;
        ins += in;
        if (!in && !out) list[atomicAdd(&s_m, 1)] = static_cast<uint16_t>(i);
      }
    }
    ins = __reduce_add_sync(0xffffffffu, ins);
    if (lane == 0 && ins) atomicAdd(&s_in, ins);
  }
  __syncthreads();
  const int m = s_m, need = want - s_in;  // 1 <= need <= m
  for (int e = threadIdx.x; e < m; e += kSelThreads) keys64[e] = 0ull;  // a bad page's stays
  __syncthreads();
  for (int i0 = 4 * warp; i0 < m * G; i0 += 4 * kSelWarps) {  // four (page, head) a round
    const int i = min(i0 + lane / 8, m * G - 1), e = i / G, h = i - e * G;
    const uint8_t* page = kv_page(P, b, c0 + list[e]);
    const uint8_t* bounds = page ? page + (long long)g * 4 * D : P.cache;  // read, but not used
    const double x = exact_bound<F, D>(q + h * D, bounds, lane % 8);
    if (lane % 8 == 0 && page) atomicMax(&keys64[e], order_key(x));
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
    int n, buf = 0;
    auto total = [&](int x) {  // over the CTA, two buffers in turn: one barrier each
      x = __reduce_add_sync(0xffffffffu, x);
      if (lane == 0) s_cnt[buf][warp] = x;
      __syncthreads();
      x = 0;
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) x += s_cnt[buf][w];
      buf ^= 1;
      return x;
    };
    bool exact = false;
    for (int bit = 63; bit >= 0 && !exact; --bit) {
      const unsigned long long cand = thr | 1ull << bit;
      n = 0;
      for (int e = threadIdx.x; e < m; e += kSelThreads) n += keys64[e] >= cand;
      n = total(n);
      if (n >= need) thr = cand;
      exact = n == need;
    }
    n = 0;
    for (int e = threadIdx.x; e < m; e += kSelThreads) n += keys64[e] > thr;
    n = total(n);
    const int at = need - n;  // pages to take at thr
    int bound = 0;                              // those with an index below the largest bound that holds <= at
    for (int bit = 14; bit >= 0; --bit) {
      const int cand = bound | 1 << bit;
      n = 0;
      for (int e = threadIdx.x; e < m; e += kSelThreads) n += keys64[e] == thr && list[e] < cand;
      n = total(n);
      if (n <= at) bound = cand;
    }
    for (int e = threadIdx.x; e < m; e += kSelThreads)
      if (keys64[e] > thr || (keys64[e] == thr && list[e] < bound)) keys[list[e]] = 0xffffffffu;
  }
  __syncthreads();

  // ---- the chosen pages in order: a thread takes a run of candidates
  const int per = (nc + kSelThreads - 1) / kSelThreads | 1;  // odd: a run's stride meets every bank
  const int i0 = min((int)threadIdx.x * per, nc), i1 = min(i0 + per, nc);
  int mine = 0;
  for (int i = i0; i < i1; ++i) mine += keys[i] != 0;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_cnt[0][warp] = inc;
  __syncthreads();
  int at = c0 + inc - mine;
  for (int w = 0; w < warp; ++w) at += s_cnt[0][w];
  for (int i = i0; i < i1; ++i)
    if (keys[i]) sel[at++] = c0 + i;
  for (int i = threadIdx.x; i < p.keep_first; i += kSelThreads) sel[i] = i;
  for (int i = threadIdx.x; i < p.keep_last; i += kSelThreads) sel[p.n_sel - p.keep_last + i] = pages - p.keep_last + i;
}

template <int F, int D>
cudaError_t select_launch(const KvSelectParams& p, cudaStream_t s) {
  auto kern = kv_select_kernel<F, D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       select_smem(STARKV_KV_MAX_SELECT_PAGES));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
