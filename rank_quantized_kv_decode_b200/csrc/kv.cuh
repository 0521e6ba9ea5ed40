// The plain key-value cache: parameter blocks and launchers shared by its kernels and entry points.
#pragma once
#include "internal.cuh"

namespace starkv {

constexpr int kKvRows = 8;         // query heads of one KV head that a warp takes together
// CTAs of the split kernel on an SM (by its registers; a third one took a ragged batch with d 64 from 16.5 to
// 14.1 us, and 32 x 32768 tokens with d 128 from 618 to 637), and the most of a launch, on 148 SMs.
constexpr int kv_split_ctas(int d) { return d == 64 ? 3 : 2; }
constexpr int kv_max_ctas(int d) { return 148 * kv_split_ctas(d); }
constexpr int kKvRounds = 8;       // small chunks per warp that a list is cut into, at most
constexpr int kKvWarps = 4;        // warps of a split CTA

// Tokens of a tile, a warp's step (see the split kernel).
constexpr int kv_tile_tokens(int fmt) { return fmt == STARKV_KV_INT8 ? 32 : 16; }

constexpr int kSelMaxCluster = 16;  // CTAs that share the choice for one (sequence, KV head)

// Where a token or page lies (offsets as in starkv_kv_layout).
struct KvPool {
  uint8_t* cache;
  long long num_pages, page_bytes;
  int off_heads, head_bytes, off_v, off_ks, off_vs;
  int H, Hkv, d, fmt;
  const int* block_table;  // [batch][max_pages]
  int max_pages, batch;
  int* status;
};

struct KvAppendParams {
  KvPool pool;
  const uint16_t *q, *k, *v;  // 16-bit elements; q may be null
  long long q_stride, k_stride, v_stride;
  int n_tok;
  const int *tok_seq, *tok_pos;
  const float2* rope;  // fine [128][d/2] then base [tiles][d/2]
  uint16_t* q_out;     // [n_tok][H][d]
  int sms;             // of the device
};

struct KvGatherParams {
  KvPool pool;
  int n_tok;
  const int *tok_seq, *tok_pos;
  uint16_t *k_out, *v_out;  // [n_tok][Hkv][d]
};

struct KvSelectParams {
  KvPool pool;
  const uint16_t* q;  // [batch][H][d]
  const int* seq_lens;
  int n_sel, keep_first, keep_last;
  int* sel;     // [batch][Hkv][n_sel]
  int cluster;  // CTAs that share one (sequence, KV head)
};

struct KvDecodeParams {
  KvPool pool;
  const uint16_t* q;  // [batch][H][d]
  const int* seq_lens;
  const int* sel;  // [batch][Hkv][n_sel] or null
  int n_sel;
  int window;
  float scale2;     // scale * log2(e)
  uint16_t* out;    // [batch][H][d]
  float* lse;       // [batch][H] or null
  unsigned* counter;  // chunks drawn
  float* rec;       // [piece][rec_rows][d] partial sums; piece = chunk + flat (sequence, KV head, group)
  float2* rec_ml;   // [piece][rec_rows] reference (log2 units), sum
  int rec_rows;     // query heads of a KV head, at most kKvRows
  int groups;       // groups of kKvRows query heads of a KV head
  int grid;         // CTAs of the split kernel
};

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t s);
cudaError_t launch_kv_gather(const KvGatherParams& p, cudaStream_t s);
cudaError_t launch_kv_select(const KvSelectParams& p, cudaStream_t s);
cudaError_t launch_kv_decode(const KvDecodeParams& p, cudaStream_t s);

#ifdef __CUDACC__
// ------------------------------------------------------------------ 16-bit types
template <int FMT>
__device__ __forceinline__ float2 kv_unpack(uint32_t w) {
  if (FMT == STARKV_KV_F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <int FMT>
__device__ __forceinline__ uint32_t kv_pack(float a, float b) {
  uint32_t r;
  if (FMT == STARKV_KV_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    r = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    r = *reinterpret_cast<const uint32_t*>(&h);
  }
  return r;
}

// Page of (sequence b, page index i) or null (flagged by the caller).
__device__ __forceinline__ uint8_t* kv_page(const KvPool& p, int b, int i) {
  const int pg = p.block_table[(long long)b * p.max_pages + i];
  return pg >= 0 && pg < p.num_pages ? p.cache + (long long)pg * p.page_bytes : nullptr;
}
#endif

}  // namespace starkv
