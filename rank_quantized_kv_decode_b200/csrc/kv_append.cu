// Append to the plain key-value cache: rotation, storage, page bounds; and the read-back.
//
// Mathematics: for channel j < d/2 the pair (x_j, x_{j+d/2}) turns by the angle pos theta^(-2j/d);
// its cosine and sine come from the fp32 table (a 128-token tile start times an offset inside
// the tile: one complex product, error about 2e-7).  int8: per token and group of 32 channels the
// scale fp16(absmax / 127) and the codes rint(x / scale), from the fp32 values.
//
// Bound: HBM for prompts (every row read once and written once; 8192 tokens of 32 + 2 x 8 heads of 128 are
// 202 MB, 31 us at the measured copy rate, and take 40.5), latency for a decode step (3.9 us for 32 tokens).
// A warp's loads of eight rounds (32 rows) are in flight together while it looks up the token, its page
// and its angles; four rounds a warp took 44.5 us, six 42.6, ten 44.1, twelve 50.2.  Of int8, whose rounds
// hold their rows' ranges and codes as well, 1005 tokens of 3 x 32 heads took 27 us with their gather at three
// rounds, 29 at two and four, 30 at six; of the 27 the append takes 22.5 (16 bits: 15.0), the gather 5.7 (4.8).
#include <algorithm>

#include "kv.cuh"
#include "store_dev.cuh"

namespace starkv {
namespace {

constexpr int kAppendWarps = 8;
constexpr int kRounds16 = 8, kRoundsInt8 = 3;  // rounds of a task of many tokens
constexpr int kFusedBoundsMax = 32;  // tokens up to which one launch does both (see the launch)

// A row is one head of q, k or v of a token; D/16 lanes share it, lane j with channels [8j, 8j+8) of
// each half: both members of a pair, 16-byte accesses, and a scale group is four neighbouring lanes.
template <int D>
struct RowMap {
  static constexpr int kLanes = D / 16, kRows = 32 / kLanes;
};

struct Raw {
  uint4 lo, hi;
};
template <int D>
__device__ __forceinline__ Raw load_raw(const uint16_t* row, int j) {
  // read once: leaves L2 to what is written
  return {__ldcs(reinterpret_cast<const uint4*>(row + 8 * j)), __ldcs(reinterpret_cast<const uint4*>(row + D / 2 + 8 * j))};
}

// Cosines and sines of a position for the lane's eight pairs.
template <int D>
__device__ __forceinline__ void angles(const float2* rope, int pos, int j, float2 (&c)[8]) {
  const float4* f = reinterpret_cast<const float4*>(rope + (pos % kTile) * (D / 2) + 8 * j);
  const float4* g = reinterpret_cast<const float4*>(rope + (kTile + pos / kTile) * (D / 2) + 8 * j);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 x = f[i], y = g[i];
    c[2 * i] = make_float2(x.x * y.x - x.y * y.y, x.x * y.y + x.y * y.x);
    c[2 * i + 1] = make_float2(x.z * y.z - x.w * y.w, x.z * y.w + x.w * y.z);
  }
}

// Smaller and larger of two pairs of 16-bit values (a NaN gives way).
template <int FMT>
__device__ __forceinline__ uint32_t pair_min(uint32_t a, uint32_t b) {
  uint32_t r;
  if (FMT == STARKV_KV_F16) asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int FMT>
__device__ __forceinline__ uint32_t pair_max(uint32_t a, uint32_t b) {
  uint32_t r;
  if (FMT == STARKV_KV_F16) asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// +inf and -inf twice: what a minimum and a maximum begin with.
template <int FMT>
constexpr uint32_t kPairInf = FMT == STARKV_KV_F16 ? 0x7c007c00u : 0x7f807f80u;

template <int FMT>
struct Row {
  float lo[8], hi[8];
  __device__ __forceinline__ void set(const Raw& r) {
    const uint32_t l[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w}, h[4] = {r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = kv_unpack<FMT>(l[i]), z = kv_unpack<FMT>(h[i]);
      lo[2 * i] = a.x, lo[2 * i + 1] = a.y, hi[2 * i] = z.x, hi[2 * i + 1] = z.y;
    }
  }
  __device__ __forceinline__ void rotate(const float2 (&c)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = lo[i], y = hi[i];
      lo[i] = x * c[i].x - y * c[i].y;
      hi[i] = y * c[i].x + x * c[i].y;
    }
  }
  __device__ __forceinline__ Raw rounded() const {
    uint32_t a[4], z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = kv_pack<FMT>(lo[2 * i], lo[2 * i + 1]), z[i] = kv_pack<FMT>(hi[2 * i], hi[2 * i + 1]);
    return {make_uint4(a[0], a[1], a[2], a[3]), make_uint4(z[0], z[1], z[2], z[3])};
  }
  float ma, mz;  // largest magnitudes of the lane's two groups
  // Scales of those groups (whole warp).
  __device__ __forceinline__ void scales(__half& sa, __half& sz) {
    ma = mz = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ma = fmaxf(ma, fabsf(lo[i])), mz = fmaxf(mz, fabsf(hi[i]));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
      mz = fmaxf(mz, __shfl_xor_sync(0xffffffffu, mz, o));
    }
    sa = store_dev::group_scale(ma, 127.f), sz = store_dev::group_scale(mz, 127.f);
  }
  // Codes under those scales, rint(x / scale): four bytes a word, lower half then upper half.  x / scale is
  // taken as x times the scale's reciprocal, within 127 x 2^-22 of the rounded quotient: the same integer
  // unless it lies that near a half.  Where one of the eight does, or is no number, or passes 127 (a scale
  // at fp16's end), all are divided.  Adding 1.5 x 2^23 rounds to an integer and leaves it in the low byte.
  static __device__ __forceinline__ void codes8(const float (&x)[8], float f, float most, uint32_t (&c)[2]) {
    const float r = f == 0.f ? 0.f : __frcp_rn(f), magic = 12582912.f;  // scale 0: codes 0
    uint32_t far = most * r < 127.49f ? 0u : 0x7fffffffu, b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = x[i] * r, t = q + magic, d = q - (t - magic);
      b[i] = __float_as_uint(t);
      far = max(far, __float_as_uint(d) & 0x7fffffffu);  // NaN's bits are above every number's
    }
    c[0] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    c[1] = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    if (far > __float_as_uint(0.4999f)) {
      c[0] = c[1] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i / 4] |= (store_dev::quant_code(x[i], f, 127) & 255) << (8 * (i % 4));
    }
  }
  __device__ __forceinline__ void codes(float fa, float fz, uint32_t (&ca)[2], uint32_t (&cz)[2]) const {
    codes8(lo, fa, ma, ca);
    codes8(hi, fz, mz, cz);
  }
  __device__ __forceinline__ void from_codes(float fa, float fz, const uint2 a, const uint2 z) {
    const uint32_t ca[2] = {a.x, a.y}, cz[2] = {z.x, z.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = fa * static_cast<float>(static_cast<int8_t>(ca[i / 4] >> (8 * (i % 4))));
      hi[i] = fz * static_cast<float>(static_cast<int8_t>(cz[i / 4] >> (8 * (i % 4))));
    }
  }
};

__device__ __forceinline__ bool in_table(const KvPool& P, int b, int pos) {
  return b >= 0 && b < P.batch && pos >= 0 && pos < P.max_pages * kPage;
}

// Bounds of one (page, KV head) by one warp, inside the append: `map` gives for each of the 64 slots the
// token of this call that fills it (its key is made again from the input: another warp may still be
// storing it) or -1 (the key is read from the page).  Four lanes a row, 32 channels of each half: D = 128
// takes two warps, `side` 0 and 1.
template <int FMT, int D>
__device__ void bounds_in_call(const KvAppendParams& p, uint8_t* page, int g, int side, const short* map, int lane) {
  const int j = 4 * side + lane % 4, r0 = lane / 4;
  const KvPool& P = p.pool;
  const uint8_t* tile = page + P.off_heads + (long long)g * P.head_bytes;
  const __half* sc = reinterpret_cast<const __half*>(tile + (FMT == STARKV_KV_INT8 ? P.off_ks : 0));
  uint32_t mn[8], mx[8];  // pairs of channels: lower half, upper half
#pragma unroll
  for (int i = 0; i < 8; ++i) mn[i] = kPairInf<FMT>, mx[i] = kPairInf<FMT> | 0x80008000u;
#pragma unroll
  for (int r1 = 0; r1 < kPage; r1 += 8) {
    const int r = r0 + r1, m = map[r];
    Raw raw;
    if (FMT != STARKV_KV_INT8) {
      raw = load_raw<D>(m < 0 ? reinterpret_cast<const uint16_t*>(tile) + r * D : p.k + m * p.k_stride + g * D, j);
      if (m >= 0) {
        Row<FMT> x;
        float2 c[8];
        x.set(raw);
        angles<D>(p.rope, p.tok_pos[m], j, c);
        x.rotate(c);
        raw = x.rounded();
      }
    } else {
      Row<FMT> x;
      if (m >= 0) {
        float2 c[8];
        x.set(load_raw<D>(p.k + m * p.k_stride + g * D, j));
        angles<D>(p.rope, p.tok_pos[m], j, c);
        x.rotate(c);
      } else {
        const float fa = __half2float(sc[r * (D / 32) + j / 4]), fz = __half2float(sc[r * (D / 32) + D / 64 + j / 4]);
        x.from_codes(fa, fz, *reinterpret_cast<const uint2*>(tile + r * D + 8 * j),
                     *reinterpret_cast<const uint2*>(tile + r * D + D / 2 + 8 * j));
      }
      if (__any_sync(0xffffffffu, m >= 0)) {
        __half sa, sz;
        x.scales(sa, sz);  // the whole warp shuffles
        if (m >= 0) {
          uint32_t ca[2], cz[2];
          x.codes(__half2float(sa), __half2float(sz), ca, cz);
          x.from_codes(__half2float(sa), __half2float(sz), make_uint2(ca[0], ca[1]), make_uint2(cz[0], cz[1]));
        }
      }
      raw = x.rounded();
    }
    const uint32_t w[8] = {raw.lo.x, raw.lo.y, raw.lo.z, raw.lo.w, raw.hi.x, raw.hi.y, raw.hi.z, raw.hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) mn[i] = pair_min<FMT>(mn[i], w[i]), mx[i] = pair_max<FMT>(mx[i], w[i]);
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mn[i] = pair_min<FMT>(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], o));
      mx[i] = pair_max<FMT>(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
    }
  if (r0 == 0) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(page) + (long long)g * 2 * D + 8 * j;
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // lower bounds of both halves, then upper
      const uint32_t* v = (k < 2 ? mn : mx) + 4 * (k % 2);
      *reinterpret_cast<uint4*>(dst + k * (D / 2)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

// CTAs on an SM, by the registers that the rounds in flight take.
constexpr int append_ctas(bool bounds, int rounds) { return rounds > 4 || bounds ? 2 : rounds > 2 ? 3 : 4; }

// One warp per task of ROUNDS rounds of a token's rows, their loads in flight together (`slices` tasks a
// token), the tasks in turn where there are more than warps (40.6 us for 8192 tokens; a warp per task 45.9); behind
// them, with BOUNDS, D / 64 warps per (token, KV head) that do something where the token completes its page.
template <int FMT, int D, bool BOUNDS, int ROUNDS>
__global__ void __launch_bounds__(32 * kAppendWarps, append_ctas(BOUNDS, ROUNDS))
    kv_append_kernel(const KvAppendParams p, int slices) {
  using R = RowMap<D>;
  constexpr int kTask = R::kRows * ROUNDS;
  __shared__ short s_map[BOUNDS ? kAppendWarps : 1][kPage];
  const KvPool& P = p.pool;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // fewer than 2^31 tasks: checked by the caller
  unsigned task = blockIdx.x * kAppendWarps + warp;
  const unsigned stores = static_cast<unsigned>(p.n_tok) * slices;
  pdl_wait();
  pdl_launch_dependents();
  if (task >= stores) {
    if (!BOUNDS) return;
    task -= stores;
    const int side = task % (D / 64);
    task /= D / 64;
    const int n = task / P.Hkv, g = task - n * P.Hkv;
    if (n >= p.n_tok) return;
    const int b = p.tok_seq[n], pos = p.tok_pos[n];
    if (!in_table(P, b, pos) || pos % kPage != kPage - 1) return;
    uint8_t* page = kv_page(P, b, pos / kPage);
    if (!page) return;
    short* map = s_map[warp];
    map[lane] = map[lane + 32] = -1;
    __syncwarp();
    for (int m = lane; m < p.n_tok; m += 32)
      if (p.tok_seq[m] == b && p.tok_pos[m] >= 0 && p.tok_pos[m] / kPage == pos / kPage)
        map[p.tok_pos[m] % kPage] = static_cast<short>(m);
    __syncwarp();
    bounds_in_call<FMT, D>(p, page, g, side, map, lane);
    return;
  }
  const int j = lane % R::kLanes;
  for (;;) {
    const int n = task / slices, slice = task - n * slices;
    const int nq = p.q ? P.H : 0, rows = nq + 2 * P.Hkv, first = slice * kTask + lane / R::kLanes;
    Raw raw[ROUNDS];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      const int r = first + i * R::kRows;
      raw[i].lo = raw[i].hi = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const uint16_t* src = r < nq             ? p.q + n * p.q_stride + r * D
                              : r < nq + P.Hkv ? p.k + n * p.k_stride + (r - nq) * D
                                               : p.v + n * p.v_stride + (r - nq - P.Hkv) * D;
        raw[i] = load_raw<D>(src, j);
      }
    }
    const int b = p.tok_seq[n], pos = p.tok_pos[n];
    const bool pos_ok = pos >= 0 && pos < P.max_pages * kPage;
    uint8_t* page = in_table(P, b, pos) ? kv_page(P, b, pos / kPage) : nullptr;
    if (!page && lane == 0 && slice == 0) atomicOr(P.status, STARKV_DEV_BOUNDS);
    const int slot = pos_ok ? pos % kPage : 0;
    float2 c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = make_float2(0.f, 0.f);
    if (pos_ok) angles<D>(p.rope, pos, j, c);
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
      const int r = first + i * R::kRows;
      if (slice * kTask + i * R::kRows >= rows) break;  // the same for the whole warp
      const bool in = r < rows;
      const int kind = r < nq ? 0 : (r < nq + P.Hkv ? 1 : 2);
      const int h = kind == 0 ? r : (kind == 1 ? r - nq : r - nq - P.Hkv);
      Row<FMT> x;
      x.set(raw[i]);
      if (kind != 2) x.rotate(c);
      uint8_t* tile = page + P.off_heads + (long long)h * P.head_bytes + (kind == 2 ? P.off_v : 0);
      uint16_t* dst = nullptr;
      if (kind == 0)
        dst = p.q_out + ((long long)n * P.H + h) * D;
      else if (FMT != STARKV_KV_INT8 && page)
        dst = reinterpret_cast<uint16_t*>(tile) + slot * D;
      if (in && dst) {
        Raw o = x.rounded();
        if (!pos_ok) o.lo = o.hi = make_uint4(0, 0, 0, 0);  // a query's row, whatever it holds (0 x inf is no zero)
        *reinterpret_cast<uint4*>(dst + 8 * j) = o.lo;
        *reinterpret_cast<uint4*>(dst + D / 2 + 8 * j) = o.hi;
      }
      if (FMT == STARKV_KV_INT8 && slice * kTask + (i + 1) * R::kRows > nq) {  // not a round of queries alone
        __half sa, sz;
        x.scales(sa, sz);  // the whole warp shuffles
        if (in && kind != 0 && page) {
          uint32_t ca[2], cz[2];
          x.codes(__half2float(sa), __half2float(sz), ca, cz);
          *reinterpret_cast<uint2*>(tile + slot * D + 8 * j) = make_uint2(ca[0], ca[1]);
          *reinterpret_cast<uint2*>(tile + slot * D + D / 2 + 8 * j) = make_uint2(cz[0], cz[1]);
          if (j % 4 == 0) {
            __half* sc = reinterpret_cast<__half*>(page + P.off_heads + (long long)h * P.head_bytes +
                                                   (kind == 2 ? P.off_vs : P.off_ks)) + slot * (D / 32);
            sc[j / 4] = sa;
            sc[D / 64 + j / 4] = sz;
          }
        }
      }
    }
    task += gridDim.x * kAppendWarps;
    if (task >= stores) return;
  }
}

// Bounds of the pages that an append of many tokens completed, after it: all keys are in the pages.  A
// CTA looks at `span` tokens for those in slot 63 and reads one KV head of their pages, eight rows a warp.
// (A warp per token and head read a page alone: 55 us for an 8192-token append where this took 45, its stores then 4 us slower.)
template <int FMT, int D>
__global__ void __launch_bounds__(256) kv_bounds_kernel(const KvAppendParams p, int span) {
  constexpr int CH = FMT == STARKV_KV_INT8 ? 16 : 8;  // channels of a 16-byte load
  constexpr int CPR = D / CH, RPW = 32 / CPR;         // loads per row, rows per warp and load
  __shared__ int hit[kPage];
  __shared__ int hits;
  __shared__ uint4 s_mn[8][D / 8], s_mx[8][D / 8];  // per warp, eight channels an entry
  const KvPool& P = p.pool;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) hits = 0;
  __syncthreads();
  if ((int)threadIdx.x < span) {
    const int n = blockIdx.x * span + threadIdx.x;
    if (n < p.n_tok && in_table(P, p.tok_seq[n], p.tok_pos[n]) && p.tok_pos[n] % kPage == kPage - 1)
      hit[atomicAdd(&hits, 1)] = n;
  }
  __syncthreads();
  for (int it = 0; it < hits; ++it) {
    const int n = hit[it];
    uint8_t* page = kv_page(P, p.tok_seq[n], p.tok_pos[n] / kPage);
    if (!page) continue;  // the same for the whole CTA
    const uint8_t* tile = page + P.off_heads + (long long)g * P.head_bytes;
    const int ck = lane % CPR, r0 = 8 * warp + lane / CPR;
    uint32_t lo[CH / 2], hi[CH / 2];
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) lo[i] = kPairInf<FMT>, hi[i] = kPairInf<FMT> | 0x80008000u;
    const uint4* src = reinterpret_cast<const uint4*>(tile);
    const __half* sc = reinterpret_cast<const __half*>(tile + (FMT == STARKV_KV_INT8 ? P.off_ks : 0));
#pragma unroll
    for (int r = 0; r < 8; r += RPW) {
      const uint4 x = src[(r0 + r) * CPR + ck];
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t v[CH / 2];
      if (FMT == STARKV_KV_INT8) {
        const float s = __half2float(sc[(r0 + r) * (D / 32) + ck / 2]);
#pragma unroll
        for (int i = 0; i < CH / 2; ++i)
          v[i] = kv_pack<FMT>(s * static_cast<float>(static_cast<int8_t>(w[i / 2] >> (16 * (i % 2)))),
                              s * static_cast<float>(static_cast<int8_t>(w[i / 2] >> (16 * (i % 2) + 8))));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = w[i];
      }
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) lo[i] = pair_min<FMT>(lo[i], v[i]), hi[i] = pair_max<FMT>(hi[i], v[i]);
    }
#pragma unroll
    for (int o = CPR; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) {
        lo[i] = pair_min<FMT>(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
        hi[i] = pair_max<FMT>(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
      }
    if (lane < CPR)
#pragma unroll
      for (int i = 0; i < CH / 8; ++i) {
        s_mn[warp][ck * (CH / 8) + i] = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
        s_mx[warp][ck * (CH / 8) + i] = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
      }
    __syncthreads();
    if (threadIdx.x < D) {  // a pair of channels: the lower bounds, then the upper
      const bool up = threadIdx.x >= D / 2;
      const uint32_t* v = reinterpret_cast<const uint32_t*>(up ? s_mx[0] : s_mn[0]) + threadIdx.x % (D / 2);
      uint32_t a = v[0];
#pragma unroll
      for (int w = 1; w < 8; ++w) a = up ? pair_max<FMT>(a, v[w * (D / 2)]) : pair_min<FMT>(a, v[w * (D / 2)]);
      reinterpret_cast<uint32_t*>(page + (long long)g * 4 * D)[threadIdx.x] = a;
    }
    __syncthreads();
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

template <int FMT, int D, bool BOUNDS, int ROUNDS>
cudaError_t append_rounds(const KvAppendParams& p, cudaStream_t s) {
  constexpr int kTask = RowMap<D>::kRows * ROUNDS;
  const int rows = (p.q ? p.pool.H : 0) + 2 * p.pool.Hkv, slices = (rows + kTask - 1) / kTask;
  const long long tasks = (long long)p.n_tok * (slices + (BOUNDS ? p.pool.Hkv * (D / 64) : 0));
  long long ctas = (tasks + kAppendWarps - 1) / kAppendWarps;
  if (!BOUNDS) ctas = std::min<long long>(ctas, static_cast<long long>(p.sms) * append_ctas(BOUNDS, ROUNDS));
  return launch_pdl(kv_append_kernel<FMT, D, BOUNDS, ROUNDS>, dim3(static_cast<unsigned>(ctas)), dim3(32 * kAppendWarps), 0, s,
                    p, slices);
}

template <int FMT, int D>
cudaError_t append_launch(const KvAppendParams& p, cudaStream_t s) {
  // Few tokens: the bounds in the same launch, where a completed page's warps look through the call's
  // tokens.  More: a launch behind it.  One launch and two took 2.8 and 4.7 us for 32 bf16 tokens of one
  // sequence, 4.1 and 6 for 32 sequences that all complete a page, but 7.3 and 5.8 for 64 of one sequence,
  // whose keys each of those warps makes again.  The host sees the number of tokens, not whose they are: steps
  // of more sequences pay for that rule.  Of 64 and 256 sequences with one token each, one launch and two took
  // 3.2 and 5.0, 3.6 and 5.3 where none completes a page, 4.0 and 6.1, 6.1 and 6.3 where one in 64 does, 4.7 and 7.0,
  // 10.5 and 12.1 where all do.
  if (p.n_tok <= kFusedBoundsMax) return append_rounds<FMT, D, true, 2>(p, s);
  const cudaError_t e = append_rounds<FMT, D, false, FMT == STARKV_KV_INT8 ? kRoundsInt8 : kRounds16>(p, s);
  if (e != cudaSuccess) return e;
  // About 64 CTAs a KV head: a CTA takes its completed pages one after another, of a prompt one in 64 tokens,
  // of a batch of sequences all at once.
  const int span = p.n_tok < 128 ? 2 : p.n_tok > 64 * kPage ? kPage : p.n_tok / 64;
  return launch_pdl(kv_bounds_kernel<FMT, D>, dim3((p.n_tok + span - 1) / span, p.pool.Hkv), dim3(256), 0, s, p, span);
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
