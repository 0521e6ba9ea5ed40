// Choice of pages for sparse attention over the plain key-value cache.
//
// Mathematics: a key inside the bounds lo <= k <= hi of its page has q.k <= sum_c max(q_c lo_c, q_c hi_c),
// attained at a corner of the box; the score of a page is the largest such bound over the query heads of
// its KV head.  The sums run in fp64: 16-bit factors have exact products there and sums of 64 or
// 128 of them are exact or nearly so, hence the order of two pages does not hang on the order of
// the summation, and equal pages score equally.
//
// Bound: HBM for large batches (the bounds are 4 d bytes per page and KV head, read once), latency
// for one sequence.  A cluster of CTAs shares one (sequence, KV head): each scores its share of the
// pages and leaves the keys in the first CTA's shared memory, which then finds the n-th largest.
#include <cooperative_groups.h>

#include "kv.cuh"

namespace starkv {
namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;

// A 16-bit value as a double times 2^-896 (bf16) or 2^-1008 (fp16), by moving its exponent and
// mantissa fields into place: exact, subnormals included.
template <int FMT>
__device__ __forceinline__ double field_double(uint32_t high16) {  // the value in the upper half
  const int w = static_cast<int>(high16);
  return FMT == STARKV_KV_F16 ? __hiloint2double((w >> 6) & 0x81ffffff, 0)
                              : __hiloint2double((w >> 3) & 0x8fffffff, 0);
}

// Order-preserving map of doubles to unsigned integers.
__device__ __forceinline__ unsigned long long order_key(double x) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// GP: query heads of a KV head that are scored together (1, 2, 4 or 8; a head may stand twice).
template <int FMT, int D, int GP>
__global__ void __launch_bounds__(kSelThreads) kv_select_kernel(const KvSelectParams p) {
  extern __shared__ unsigned long long keys[];  // [max_pages] in the cluster's first CTA
  __shared__ int s_cnt[2][kSelWarps];
  __shared__ unsigned long long s_ext[2][kSelWarps];
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  constexpr int F = FMT == STARKV_KV_F16 ? STARKV_KV_F16 : STARKV_KV_BF16;  // type of q and bounds
  constexpr int CL = D / 32;                                                  // channels of a lane
  constexpr int NP = 32 / GP;                                                 // pages of a warp's round
  const KvPool& P = p.pool;
  const int rank = blockIdx.x % p.cluster, unit = blockIdx.x / p.cluster;
  const int b = unit / P.Hkv, g = unit % P.Hkv, G = P.H / P.Hkv;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
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
  unsigned long long* first = cluster.map_shared_rank(keys, 0);

  if (want > 0) {
    for (int h0 = 0; h0 < G; h0 += GP) {
      // queries times a power of two that undoes field_double's
      double q[GP][CL];
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        const uint16_t* src = p.q + ((long long)b * P.H + g * G + min(h0 + h, G - 1)) * D + lane * CL;
#pragma unroll
        for (int i = 0; i < CL / 2; ++i) {
          const float2 x = kv_unpack<F>(reinterpret_cast<const uint32_t*>(src)[i]);
          const double up = __hiloint2double((1023 + (F == STARKV_KV_F16 ? 1000 : 880)) << 20, 0);
          q[h][2 * i] = x.x * up, q[h][2 * i + 1] = x.y * up;
        }
      }
      for (int i0 = (rank * kSelWarps + warp) * NP; i0 < nc; i0 += p.cluster * kSelWarps * NP) {
        double acc[32];  // [page][head]
        const int mine = min(i0 + lane / GP, nc - 1);
        const uint8_t* page = kv_page(P, b, c0 + mine);
        if (!page && i0 + lane / GP < nc) atomicOr(P.status, STARKV_DEV_BOUNDS);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const uint8_t* pk = reinterpret_cast<const uint8_t*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(page), k * GP));
          uint32_t lo[CL / 2], hi[CL / 2];
          const uint32_t* src = reinterpret_cast<const uint32_t*>(pk + (long long)g * 4 * D) + lane * (CL / 2);
#pragma unroll
          for (int i = 0; i < CL / 2; ++i) {
            lo[i] = pk ? src[i] : 0u;
            hi[i] = pk ? src[D / 2 + i] : 0u;
          }
#pragma unroll
          for (int h = 0; h < GP; ++h) {
            double a = 0.0;
#pragma unroll
            for (int i = 0; i < CL; ++i) {
              const uint32_t l = i % 2 ? lo[i / 2] & 0xffff0000u : lo[i / 2] << 16;
              const uint32_t u = i % 2 ? hi[i / 2] & 0xffff0000u : hi[i / 2] << 16;
              a = fma(q[h][i], field_double<F>(__double2hiint(q[h][i]) < 0 ? l : u), a);
            }
            acc[k * GP + h] = a;
          }
        }
        // 32 sums over 32 lanes: lane i ends with sum i
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (i < o) {
              const double keep = up ? acc[i + o] : acc[i], give = up ? acc[i] : acc[i + o];
              acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
          }
        }
        double best = acc[0];
#pragma unroll
        for (int o = 1; o < GP; o <<= 1) best = fmax(best, __shfl_xor_sync(0xffffffffu, best, o));
        const int i = i0 + lane / GP;
        if (lane % GP == 0 && i < nc) {
          unsigned long long key = page ? order_key(best) : 0ull;
          if (h0 > 0) key = max(key, first[i]);  // written by this thread for the heads before
          first[i] = key;
        }
      }
    }
  }
  cluster.sync();
  if (rank != 0) return;

  // The want-th largest key, bit by bit from the first that differs: thr = the largest value that at least
  // `want` keys reach.
  unsigned long long thr = ~0ull;
  int above = 0;  // keys above thr
  auto total = [&](int v, int buf) {
    v = __reduce_add_sync(0xffffffffu, v);
    if (lane == 0) s_cnt[buf][warp] = v;
    __syncthreads();
    int t = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) t += s_cnt[buf][w];
    return t;
  };
  if (want > 0) {
    unsigned long long mn = ~0ull, mx = 0;
    for (int i = threadIdx.x; i < nc; i += kSelThreads) mn = min(mn, keys[i]), mx = max(mx, keys[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mn = min(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if (lane == 0) s_ext[0][warp] = mn, s_ext[1][warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) mn = min(mn, s_ext[0][w]), mx = max(mx, s_ext[1][w]);
    const int high = 63 - __clzll(mn ^ mx);  // -1: all equal
    thr = high < 63 ? mx & ~((2ull << high) - 1) : 0ull;
    if (high < 0) thr = mx;
    int buf = 0;
    bool exact = false;
    for (int bit = high; bit >= 0 && !exact; --bit) {
      const unsigned long long cand = thr | 1ull << bit;
      int n = 0;
      for (int i = threadIdx.x; i < nc; i += kSelThreads) n += keys[i] >= cand;
      n = total(n, buf);
      buf ^= 1;
      if (n >= want) thr = cand;
      exact = n == want;
    }
    int n = 0;
    for (int i = threadIdx.x; i < nc; i += kSelThreads) n += keys[i] > thr;
    __syncthreads();
    above = total(n, 0);
  }
  // pages in order: those above the threshold, and of those at it the lowest
  const int at = want - above;
  int done_gt = 0, done_eq = 0;
  __syncthreads();
  for (int i0 = 0; want > 0 && i0 < nc; i0 += kSelThreads) {
    const int i = i0 + threadIdx.x;
    const bool gt = i < nc && keys[i] > thr, eq = i < nc && keys[i] == thr;
    const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_cnt[0][warp] = __popc(mg), s_cnt[1][warp] = __popc(me);
    __syncthreads();
    int ng = done_gt, ne = done_eq;
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) ng += s_cnt[0][w], ne += s_cnt[1][w];
      done_gt += s_cnt[0][w], done_eq += s_cnt[1][w];
    }
    const unsigned below = (1u << lane) - 1;
    ng += __popc(mg & below), ne += __popc(me & below);
    if (gt || (eq && ne < at)) sel[c0 + ng + min(ne, at)] = c0 + i;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < p.keep_first; i += kSelThreads) sel[i] = i;
  for (int i = threadIdx.x; i < p.keep_last; i += kSelThreads) sel[p.n_sel - p.keep_last + i] = pages - p.keep_last + i;
}

template <int FMT, int D, int GP>
cudaError_t select_launch(const KvSelectParams& p, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(p.pool.max_pages) * 8;
  auto kern = kv_select_kernel<FMT, D, GP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       STARKV_KV_MAX_SELECT_PAGES * 8);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.pool.batch * p.pool.Hkv * p.cluster));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
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

template <int FMT, int D>
cudaError_t by_group(const KvSelectParams& p, cudaStream_t s) {
  const int G = p.pool.H / p.pool.Hkv;
  if (G == 1) return select_launch<FMT, D, 1>(p, s);
  if (G == 2) return select_launch<FMT, D, 2>(p, s);
  if (G <= 4) return select_launch<FMT, D, 4>(p, s);
  return select_launch<FMT, D, 8>(p, s);
}

}  // namespace

cudaError_t launch_kv_select(const KvSelectParams& p, cudaStream_t s) {
  const int d = p.pool.d;
  if (p.pool.fmt == STARKV_KV_F16)
    return d == 64 ? by_group<STARKV_KV_F16, 64>(p, s) : by_group<STARKV_KV_F16, 128>(p, s);
  return d == 64 ? by_group<STARKV_KV_BF16, 64>(p, s) : by_group<STARKV_KV_BF16, 128>(p, s);
}

}  // namespace starkv
