// Append to the plain key-value cache: rotation, storage, page bounds; and the read-back.
//
// Mathematics: for channel j < d/2 the pair (x_j, x_{j+d/2}) turns by the angle pos theta^(-2j/d);
// its cosine and sine come from the fp32 table (a 128-token tile start times an offset inside
// the tile: one complex product, error about 2e-7).  int8: per token and group of 32 channels the
// scale fp16(absmax / 127) and the codes rint(x / scale), from the fp32 values.
#include "kv.cuh"
#include "store_dev.cuh"

namespace starkv {
namespace {

constexpr int kAppendThreads = 256;

// One CTA per token (and slice of its rows).  A row is one head of q, k or v; D/16 threads share
// it, thread j with channels [8j, 8j+8) of each half: both members of a pair, 16-byte accesses,
// and a scale group is four neighbouring threads.
template <int FMT, int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const KvAppendParams p) {
  constexpr int TPR = D / 16, RPP = kAppendThreads / TPR, HALF = D / 2;
  __shared__ float2 cs[HALF];
  const int n = blockIdx.x, tid = threadIdx.x;
  const int j = tid % TPR;
  const KvPool& P = p.pool;
  pdl_wait();
  pdl_launch_dependents();
  const int b = p.tok_seq[n], pos = p.tok_pos[n];
  const bool pos_ok = pos >= 0 && pos < P.max_pages * kPage;
  uint8_t* page = nullptr;
  if (pos_ok && b >= 0 && b < P.batch) page = kv_page(P, b, pos / kPage);
  if (!page && tid == 0 && blockIdx.y == 0) atomicOr(P.status, STARKV_DEV_BOUNDS);
  if (tid < HALF && pos_ok) {
    const float2 f = p.rope[(pos % kTile) * HALF + tid];
    const float2 g = p.rope[(kTile + pos / kTile) * HALF + tid];
    cs[tid] = make_float2(f.x * g.x - f.y * g.y, f.x * g.y + f.y * g.x);
  }
  __syncthreads();
  const int slot = pos_ok ? pos % kPage : 0;
  const int nq = p.q ? P.H : 0, rows = nq + 2 * P.Hkv;
  float2 c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = pos_ok ? cs[8 * j + i] : make_float2(0.f, 0.f);
  // every thread of a warp makes the same number of rounds (the scale groups shuffle)
  for (int r0 = blockIdx.y * RPP; r0 < rows; r0 += gridDim.y * RPP) {
    const int r = r0 + tid / TPR;
    const bool in = r < rows;
    const int kind = r < nq ? 0 : (r < nq + P.Hkv ? 1 : 2);
    const int h = kind == 0 ? r : (kind == 1 ? r - nq : r - nq - P.Hkv);
    uint4 lo4 = make_uint4(0, 0, 0, 0), hi4 = lo4;
    if (in) {
      const uint16_t* src = kind == 0   ? p.q + n * p.q_stride
                            : kind == 1 ? p.k + n * p.k_stride
                                        : p.v + n * p.v_stride;
      src += h * D + 8 * j;
      lo4 = *reinterpret_cast<const uint4*>(src);
      hi4 = *reinterpret_cast<const uint4*>(src + HALF);
    }
    float lo[8], hi[8];
    const uint32_t lw[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, hw[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = kv_unpack<FMT>(lw[i]), z = kv_unpack<FMT>(hw[i]);
      lo[2 * i] = a.x, lo[2 * i + 1] = a.y, hi[2 * i] = z.x, hi[2 * i + 1] = z.y;
    }
    if (kind != 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = lo[i], y = hi[i];
        lo[i] = x * c[i].x - y * c[i].y;
        hi[i] = y * c[i].x + x * c[i].y;
      }
    }
    uint16_t* dst16 = nullptr;
    if (kind == 0)
      dst16 = p.q_out + ((long long)n * P.H + h) * D;
    else if (FMT != STARKV_KV_INT8 && page)
      dst16 = reinterpret_cast<uint16_t*>(page + P.off_heads + (long long)h * P.head_bytes +
                                          (kind == 2 ? P.off_v : 0)) + slot * D;
    if (in && dst16) {
      uint32_t a[4], z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = kv_pack<FMT>(lo[2 * i], lo[2 * i + 1]);
        z[i] = kv_pack<FMT>(hi[2 * i], hi[2 * i + 1]);
      }
      *reinterpret_cast<uint4*>(dst16 + 8 * j) = make_uint4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<uint4*>(dst16 + HALF + 8 * j) = make_uint4(z[0], z[1], z[2], z[3]);
    }
    if (FMT == STARKV_KV_INT8) {
      float ma = 0.f, mz = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ma = fmaxf(ma, fabsf(lo[i])), mz = fmaxf(mz, fabsf(hi[i]));
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
        mz = fmaxf(mz, __shfl_xor_sync(0xffffffffu, mz, o));
      }
      if (in && kind != 0 && page) {
        const __half sa = store_dev::group_scale(ma, 127.f), sz = store_dev::group_scale(mz, 127.f);
        const float fa = __half2float(sa), fz = __half2float(sz);
        uint8_t* tile = page + P.off_heads + (long long)h * P.head_bytes;
        uint8_t* code = tile + (kind == 2 ? P.off_v : 0) + slot * D;
        __half* sc = reinterpret_cast<__half*>(tile + (kind == 2 ? P.off_vs : P.off_ks)) + slot * (D / 32);
        uint32_t ca[2] = {0, 0}, cz[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ca[i / 4] |= (store_dev::quant_code(lo[i], fa, 127) & 255) << (8 * (i % 4));
          cz[i / 4] |= (store_dev::quant_code(hi[i], fz, 127) & 255) << (8 * (i % 4));
        }
        *reinterpret_cast<uint2*>(code + 8 * j) = make_uint2(ca[0], ca[1]);
        *reinterpret_cast<uint2*>(code + HALF + 8 * j) = make_uint2(cz[0], cz[1]);
        if (j % 4 == 0) {
          sc[j / 4] = sa;
          sc[HALF / 32 + j / 4] = sz;
        }
      }
    }
  }
}

// Bounds of the pages that an append completed: per channel the smallest and largest stored key.
// Runs after the append (its 64 keys may come from several CTAs and calls).  A CTA looks at
// `span` tokens for those in slot 63; one warp reads one (page, KV head): 16-byte loads, a lane
// keeps the same channels in every row.
constexpr int kBoundsWarps = 8;
template <int FMT, int D>
__global__ void __launch_bounds__(32 * kBoundsWarps) kv_bounds_kernel(const KvAppendParams p, int span) {
  constexpr int CH = FMT == STARKV_KV_INT8 ? 16 : 8;  // channels of a 16-byte load
  constexpr int CPR = D / CH, RPW = 32 / CPR;         // loads per row, rows per warp and round
  __shared__ int hit[64];
  __shared__ int hits;
  const KvPool& P = p.pool;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) hits = 0;
  __syncthreads();
  if ((int)threadIdx.x < span) {
    const int n = blockIdx.x * span + threadIdx.x;
    if (n < p.n_tok) {
      const int b = p.tok_seq[n], pos = p.tok_pos[n];
      if (b >= 0 && b < P.batch && pos >= 0 && pos < P.max_pages * kPage && pos % kPage == kPage - 1)
        hit[atomicAdd(&hits, 1)] = n;
    }
  }
  __syncthreads();
  const int items = hits * P.Hkv;
  for (int it = blockIdx.y * kBoundsWarps + warp; it < items; it += gridDim.y * kBoundsWarps) {
    const int n = hit[it / P.Hkv], g = it % P.Hkv;
    uint8_t* page = kv_page(P, p.tok_seq[n], p.tok_pos[n] / kPage);
    if (!page) continue;
    const uint8_t* tile = page + P.off_heads + (long long)g * P.head_bytes;
    const int ck = lane % CPR, r0 = lane / CPR;
    float lo[CH], hi[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) lo[i] = __int_as_float(0x7f800000), hi[i] = __int_as_float(0xff800000);
    const uint4* src = reinterpret_cast<const uint4*>(tile);
    const __half* sc = reinterpret_cast<const __half*>(tile + (FMT == STARKV_KV_INT8 ? P.off_ks : 0));
#pragma unroll 8
    for (int r = r0; r < kPage; r += RPW) {
      const uint4 x = src[r * CPR + ck];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      if (FMT == STARKV_KV_INT8) {
        const float s = __half2float(sc[r * (D / 32) + ck / 2]);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const float v = s * static_cast<float>(static_cast<int8_t>(w[i / 4] >> (8 * (i % 4))));
          lo[i] = fminf(lo[i], v), hi[i] = fmaxf(hi[i], v);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = kv_unpack<FMT>(w[i]);
          lo[2 * i] = fminf(lo[2 * i], v.x), hi[2 * i] = fmaxf(hi[2 * i], v.x);
          lo[2 * i + 1] = fminf(lo[2 * i + 1], v.y), hi[2 * i + 1] = fmaxf(hi[2 * i + 1], v.y);
        }
      }
    }
#pragma unroll
    for (int o = CPR; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
        hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
      }
    if (r0 == 0) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(page + (long long)g * 2 * D * 2) + ck * (CH / 2);
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        dst[i] = kv_pack<FMT>(lo[2 * i], lo[2 * i + 1]);
        dst[D / 2 + i] = kv_pack<FMT>(hi[2 * i], hi[2 * i + 1]);
      }
    }
  }
}

// Read-back: one thread per 8 channels of one (token, KV head).
template <int FMT>
__global__ void __launch_bounds__(256) kv_gather_kernel(const KvGatherParams p) {
  const KvPool& P = p.pool;
  pdl_wait();
  pdl_launch_dependents();
  const int per = P.Hkv * P.d / 8;
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int n = static_cast<int>(idx / per), e = static_cast<int>(idx % per);
  if (n >= p.n_tok) return;
  const int g = e / (P.d / 8), ch = e % (P.d / 8) * 8;
  const int b = p.tok_seq[n], pos = p.tok_pos[n];
  const uint8_t* page = nullptr;
  if (b >= 0 && b < P.batch && pos >= 0 && pos < P.max_pages * kPage) page = kv_page(P, b, pos / kPage);
  if (!page && e == 0) atomicOr(P.status, STARKV_DEV_BOUNDS);
  const uint8_t* tile = page ? page + P.off_heads + (long long)g * P.head_bytes : nullptr;
  const int slot = pos % kPage;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    uint4 o = make_uint4(0, 0, 0, 0);
    if (tile) {
      const uint8_t* src = tile + (kind ? P.off_v : 0);
      if (FMT != STARKV_KV_INT8) {
        o = *reinterpret_cast<const uint4*>(src + ((long long)slot * P.d + ch) * 2);
      } else {
        const uint2 c = *reinterpret_cast<const uint2*>(src + (long long)slot * P.d + ch);
        const float s = __half2float(reinterpret_cast<const __half*>(
            tile + (kind ? P.off_vs : P.off_ks))[slot * (P.d / 32) + ch / 32]);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t cw = i < 2 ? c.x : c.y;
          w[i] = kv_pack<FMT>(s * static_cast<float>(static_cast<int8_t>(cw >> (16 * (i % 2)))),
                              s * static_cast<float>(static_cast<int8_t>(cw >> (16 * (i % 2) + 8))));
        }
        o = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    *reinterpret_cast<uint4*>((kind ? p.v_out : p.k_out) + ((long long)n * P.Hkv + g) * P.d + ch) = o;
  }
}

template <int FMT, int D>
cudaError_t append_launch(const KvAppendParams& p, cudaStream_t s) {
  const int rpp = kAppendThreads / (D / 16);
  const int rows = (p.q ? p.pool.H : 0) + 2 * p.pool.Hkv;
  // few tokens: one CTA per slice of the rows; many: a token's rows in one CTA
  const int slices = p.n_tok < 512 ? (rows + rpp - 1) / rpp : 1;
  cudaError_t e = launch_pdl(kv_append_kernel<FMT, D>, dim3(p.n_tok, slices), dim3(kAppendThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  // few tokens: most may sit in slot 63 at once; many: one in 64 of a prompt does
  const int span = p.n_tok <= 1024 ? 8 : 64;
  return launch_pdl(kv_bounds_kernel<FMT, D>, dim3((p.n_tok + span - 1) / span, span == 8 ? p.pool.Hkv : 1),
                    dim3(32 * kBoundsWarps), 0, s, p, span);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t s) {
  const int d = p.pool.d;
  switch (p.pool.fmt) {
    case STARKV_KV_BF16: return d == 64 ? append_launch<STARKV_KV_BF16, 64>(p, s) : append_launch<STARKV_KV_BF16, 128>(p, s);
    case STARKV_KV_F16: return d == 64 ? append_launch<STARKV_KV_F16, 64>(p, s) : append_launch<STARKV_KV_F16, 128>(p, s);
    case STARKV_KV_INT8: return d == 64 ? append_launch<STARKV_KV_INT8, 64>(p, s) : append_launch<STARKV_KV_INT8, 128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_kv_gather(const KvGatherParams& p, cudaStream_t s) {
  const long long threads = (long long)p.n_tok * p.pool.Hkv * p.pool.d / 8;
  const dim3 grid(static_cast<unsigned>((threads + 255) / 256));
  switch (p.pool.fmt) {
    case STARKV_KV_BF16: return launch_pdl(kv_gather_kernel<STARKV_KV_BF16>, grid, dim3(256), 0, s, p);
    case STARKV_KV_F16: return launch_pdl(kv_gather_kernel<STARKV_KV_F16>, grid, dim3(256), 0, s, p);
    case STARKV_KV_INT8: return launch_pdl(kv_gather_kernel<STARKV_KV_INT8>, grid, dim3(256), 0, s, p);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace starkv
