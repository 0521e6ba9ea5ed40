// Entry points of the plain key-value cache: argument checks, page layout, launch shapes.
#include <cmath>
#include <cstring>
#include <mutex>
#include <string>

#include "kv.cuh"

using namespace starkv;

namespace {

starkv_status fail(starkv_status s, const std::string& msg) {
  set_error_message(msg);
  return s;
}
starkv_status cuda_fail(cudaError_t e, const char* where) {
  return fail(STARKV_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

// SM count of the current device, which has to be one the library is built for.
starkv_status device_sms(int& sms) {
  static std::mutex mu;
  static int cache[64];  // 0: not asked yet, -1: another architecture
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= 64) return fail(STARKV_ERR_UNSUPPORTED, "device index above 63");
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    int n = 0, major = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    cache[dev] = major == 10 ? n : -1;
  }
  if (cache[dev] < 0) return fail(STARKV_ERR_UNSUPPORTED, "this library is built for sm_100a (B200)");
  sms = cache[dev];
  return STARKV_OK;
}

size_t kv_rope_bytes(const starkv_kv_layout* lay, int max_pages) {
  const int tiles = (max_pages * kPage + kTile - 1) / kTile;
  return static_cast<size_t>(kTile + tiles) * (lay->cfg.head_dim / 2) * sizeof(float2);
}
int kv_groups(const starkv_kv_layout* lay) {
  return (lay->cfg.n_q_heads / lay->cfg.n_kv_heads + kKvRows - 1) / kKvRows;
}
int kv_record_rows(const starkv_kv_layout* lay) {
  const int G = lay->cfg.n_q_heads / lay->cfg.n_kv_heads;
  return G < kKvRows ? G : kKvRows;
}
constexpr size_t kKvCounterBytes = 256;
constexpr int kKvMaxBatch = 65535;                  // sequences of a decode call (the join's grid)
constexpr int64_t kKvMostTiles = int64_t(1) << 30;  // the kernels number tiles in 32 bits

// Tiles that a decode call may visit, and the most pieces it cuts them into (see the split kernel's list).
int64_t kv_tiles(const starkv_kv_layout* lay, int64_t batch, int64_t max_pages) {
  return batch * lay->cfg.n_kv_heads * kv_groups(lay) * max_pages * (kPage / kv_tile_tokens(lay->cfg.fmt));
}
int64_t kv_pieces(const starkv_kv_layout* lay, int64_t batch) {
  return static_cast<int64_t>(kv_max_ctas(lay->cfg.head_dim)) * kKvWarps * (1 + kKvRounds) + batch * lay->cfg.n_kv_heads * kv_groups(lay);
}
// Workspace: the counter, the sums, then (reference, sum) of the records.
size_t kv_record_bytes(const starkv_kv_layout* lay, int64_t batch) {
  return kKvCounterBytes + static_cast<size_t>(kv_pieces(lay, batch)) * kv_record_rows(lay) *
                               (lay->cfg.head_dim * sizeof(float) + sizeof(float2));
}

starkv_status check_kv_layout(const starkv_kv_layout* lay) {
  if (!lay) return fail(STARKV_ERR_INVALID_ARG, "layout is NULL");
  starkv_kv_layout chk;
  const starkv_status st = starkv_kv_layout_init(&lay->cfg, &chk);
  if (st != STARKV_OK) return st;
  if (std::memcmp(&chk, lay, sizeof(chk)) != 0)
    return fail(STARKV_ERR_INVALID_ARG, "layout was not produced by starkv_kv_layout_init for its config");
  return STARKV_OK;
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// The arguments that every call on the pages shares (the layout is checked).
starkv_status fill_pool(const starkv_kv_layout* lay, const void* cache, int64_t num_pages,
                        const int32_t* block_table, int32_t max_pages, int32_t batch,
                        int32_t* dev_status, KvPool& p) {
  if (max_pages < 1 || max_pages > (1 << 24)) return fail(STARKV_ERR_INVALID_ARG, "max_pages outside [1, 2^24]");
  if (num_pages < 1 || num_pages > INT32_MAX) return fail(STARKV_ERR_INVALID_ARG, "num_pages outside [1, 2^31)");
  if (!cache || !block_table || !dev_status) return fail(STARKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (misaligned(cache)) return fail(STARKV_ERR_INVALID_ARG, "cache must be 16-byte aligned");
  p.cache = const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(cache));
  p.num_pages = num_pages;
  p.page_bytes = lay->page_bytes;
  p.off_heads = static_cast<int>(lay->off_heads);
  p.head_bytes = static_cast<int>(lay->head_bytes);
  p.off_v = static_cast<int>(lay->off_v);
  p.off_ks = static_cast<int>(lay->off_ks);
  p.off_vs = static_cast<int>(lay->off_vs);
  p.H = lay->cfg.n_q_heads;
  p.Hkv = lay->cfg.n_kv_heads;
  p.d = lay->cfg.head_dim;
  p.fmt = lay->cfg.fmt;
  p.block_table = block_table;
  p.max_pages = max_pages;
  p.batch = batch;
  p.status = dev_status;
  return STARKV_OK;
}

}  // namespace

extern "C" {

starkv_status starkv_kv_layout_init(const starkv_kv_config* cfg, starkv_kv_layout* out) {
  if (!cfg || !out) return fail(STARKV_ERR_INVALID_ARG, "cfg/out is NULL");
  const starkv_kv_config& c = *cfg;
  if (c.n_kv_heads < 1 || c.n_kv_heads > STARKV_MAX_KV_HEADS)
    return fail(STARKV_ERR_INVALID_ARG, "n_kv_heads must be in [1, 64]");
  if (c.n_q_heads < c.n_kv_heads || c.n_q_heads % c.n_kv_heads != 0)
    return fail(STARKV_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of n_kv_heads");
  if (c.n_q_heads / c.n_kv_heads > 64)
    return fail(STARKV_ERR_UNSUPPORTED, "at most 64 query heads per KV head");
  if (c.head_dim != 64 && c.head_dim != 128) return fail(STARKV_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (c.fmt != STARKV_KV_BF16 && c.fmt != STARKV_KV_F16 && c.fmt != STARKV_KV_INT8)
    return fail(STARKV_ERR_INVALID_ARG, "unknown cache format");
  if (c.page_tokens != kPage) return fail(STARKV_ERR_UNSUPPORTED, "page_tokens must be 64");
  if (c.reserved != 0) return fail(STARKV_ERR_INVALID_ARG, "reserved must be 0");
  if (!(c.rope_theta > 1.0) || !std::isfinite(c.rope_theta))
    return fail(STARKV_ERR_INVALID_ARG, "rope_theta must be finite and > 1");
  const int64_t d = c.head_dim, el = c.fmt == STARKV_KV_INT8 ? 1 : 2;
  const int64_t scales = c.fmt == STARKV_KV_INT8 ? kPage * (d / STARKV_GROUP) * 2 : 0;
  starkv_kv_layout L;
  std::memset(&L, 0, sizeof(L));
  L.cfg.n_q_heads = c.n_q_heads;
  L.cfg.n_kv_heads = c.n_kv_heads;
  L.cfg.head_dim = c.head_dim;
  L.cfg.fmt = c.fmt;
  L.cfg.page_tokens = c.page_tokens;
  L.cfg.rope_theta = c.rope_theta;
  L.off_heads = 2 * d * 2 * c.n_kv_heads;
  L.off_v = kPage * d * el;
  L.off_ks = scales ? 2 * L.off_v : -1;
  L.off_vs = scales ? 2 * L.off_v + scales : -1;
  L.head_bytes = 2 * L.off_v + 2 * scales;
  L.page_bytes = L.off_heads + c.n_kv_heads * L.head_bytes;
  L.token_bytes = c.n_kv_heads * L.head_bytes / kPage;
  *out = L;
  return STARKV_OK;
}

starkv_status starkv_kv_alloc(const starkv_kv_layout* lay, int64_t num_pages, int32_t batch,
                              int32_t max_pages, starkv_kv_sizes* out) {
  const starkv_status st = check_kv_layout(lay);
  if (st != STARKV_OK) return st;
  if (!out) return fail(STARKV_ERR_INVALID_ARG, "out is NULL");
  if (num_pages < 0 || batch < 0 || batch > kKvMaxBatch)
    return fail(STARKV_ERR_INVALID_ARG, "num_pages < 0 or batch outside [0, 65535]");
  if (max_pages < 1 || max_pages > (1 << 24)) return fail(STARKV_ERR_INVALID_ARG, "max_pages outside [1, 2^24]");
  if (static_cast<uint64_t>(num_pages) > SIZE_MAX / static_cast<uint64_t>(lay->page_bytes))
    return fail(STARKV_ERR_INVALID_ARG, "num_pages * page_bytes does not fit in size_t");
  out->cache_bytes = static_cast<size_t>(num_pages) * lay->page_bytes;
  out->rope_table_bytes = kv_rope_bytes(lay, max_pages);
  if (kv_tiles(lay, batch, max_pages) > kKvMostTiles)
    return fail(STARKV_ERR_INVALID_ARG, "batch * n_kv_heads * max_pages too large for one decode call");
  out->decode_workspace_bytes = kv_record_bytes(lay, batch);
  return STARKV_OK;
}

starkv_status starkv_kv_rope_init(const starkv_kv_layout* lay, int32_t max_pages, void* table,
                                  size_t table_bytes, starkv_stream_t stream) {
  starkv_status st = check_kv_layout(lay);
  if (st != STARKV_OK) return st;
  if (!table) return fail(STARKV_ERR_INVALID_ARG, "table is NULL");
  if (misaligned(table)) return fail(STARKV_ERR_INVALID_ARG, "table must be 16-byte aligned");
  if (max_pages < 1 || max_pages > (1 << 24)) return fail(STARKV_ERR_INVALID_ARG, "max_pages outside [1, 2^24]");
  if (table_bytes < kv_rope_bytes(lay, max_pages)) return fail(STARKV_ERR_WORKSPACE, "rope table too small");
  int sms = 0;
  st = device_sms(sms);
  if (st != STARKV_OK) return st;
  const cudaError_t e =
      launch_rope_init(reinterpret_cast<float2*>(table), lay->cfg.head_dim / 2, kTile,
                       (max_pages * kPage + kTile - 1) / kTile, lay->cfg.rope_theta, lay->cfg.head_dim,
                       reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope init launch");
  return STARKV_OK;
}

starkv_status starkv_kv_append(const starkv_kv_layout* lay, const void* q, int64_t q_stride,
                               const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               int32_t n_tok, const int32_t* tok_seq, const int32_t* tok_pos,
                               const int32_t* block_table, int32_t max_pages, int32_t batch,
                               const void* rope_table, size_t rope_table_bytes, void* cache,
                               int64_t num_pages, void* q_out, int32_t* dev_status,
                               starkv_stream_t stream) {
  starkv_status st = check_kv_layout(lay);
  if (st != STARKV_OK) return st;
  if (n_tok < 0 || batch < 1) return fail(STARKV_ERR_INVALID_ARG, "n_tok < 0 or batch < 1");
  if (n_tok == 0) return STARKV_OK;
  // the kernels number their tasks (at most the rows, and two per KV head) in 32 bits
  if (static_cast<int64_t>(n_tok) * (lay->cfg.n_q_heads + 4 * lay->cfg.n_kv_heads) > INT32_MAX)
    return fail(STARKV_ERR_INVALID_ARG, "n_tok too large for one call; split the tokens");
  KvAppendParams p;
  std::memset(&p, 0, sizeof(p));
  st = fill_pool(lay, cache, num_pages, block_table, max_pages, batch, dev_status, p.pool);
  if (st != STARKV_OK) return st;
  if (!k || !v || !tok_seq || !tok_pos || !rope_table) return fail(STARKV_ERR_INVALID_ARG, "NULL pointer argument");
  if ((q == nullptr) != (q_out == nullptr))
    return fail(STARKV_ERR_INVALID_ARG, "q and q_out go together (both NULL: keys and values only)");
  const int64_t d = lay->cfg.head_dim, qw = lay->cfg.n_q_heads * d, kw = lay->cfg.n_kv_heads * d;
  if ((q && (q_stride < qw || q_stride % 8)) || k_stride < kw || k_stride % 8 || v_stride < kw || v_stride % 8)
    return fail(STARKV_ERR_INVALID_ARG, "strides must be multiples of 8 elements and hold a row");
  if (q && q == q_out && q_stride != qw)
    return fail(STARKV_ERR_INVALID_ARG, "q_out may be q only where q's rows are contiguous");
  if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(q_out) || misaligned(rope_table))
    return fail(STARKV_ERR_INVALID_ARG, "q, k, v, q_out and rope_table must be 16-byte aligned");
  if (rope_table_bytes < kv_rope_bytes(lay, max_pages))
    return fail(STARKV_ERR_WORKSPACE, "rope table smaller than needed for max_pages");
  int sms = 0;
  st = device_sms(sms);
  if (st != STARKV_OK) return st;
  p.q = reinterpret_cast<const uint16_t*>(q);
  p.k = reinterpret_cast<const uint16_t*>(k);
  p.v = reinterpret_cast<const uint16_t*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.n_tok = n_tok;
  p.tok_seq = tok_seq;
  p.tok_pos = tok_pos;
  p.rope = reinterpret_cast<const float2*>(rope_table);
  p.q_out = reinterpret_cast<uint16_t*>(q_out);
  p.sms = sms;
  const cudaError_t e = launch_kv_append(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv append launch");
  return STARKV_OK;
}

starkv_status starkv_kv_gather(const starkv_kv_layout* lay, const void* cache, int64_t num_pages,
                               const int32_t* tok_seq, const int32_t* tok_pos, int32_t n_tok,
                               const int32_t* block_table, int32_t max_pages, int32_t batch,
                               void* k_out, void* v_out, int32_t* dev_status, starkv_stream_t stream) {
  starkv_status st = check_kv_layout(lay);
  if (st != STARKV_OK) return st;
  if (n_tok < 0 || batch < 1) return fail(STARKV_ERR_INVALID_ARG, "n_tok < 0 or batch < 1");
  if (n_tok == 0) return STARKV_OK;
  KvGatherParams p;
  std::memset(&p, 0, sizeof(p));
  st = fill_pool(lay, cache, num_pages, block_table, max_pages, batch, dev_status, p.pool);
  if (st != STARKV_OK) return st;
  if (!tok_seq || !tok_pos || !k_out || !v_out) return fail(STARKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (misaligned(k_out) || misaligned(v_out))
    return fail(STARKV_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
  if (static_cast<int64_t>(n_tok) * p.pool.Hkv * p.pool.d / 8 > (int64_t(1) << 38))
    return fail(STARKV_ERR_INVALID_ARG, "n_tok too large for one call; split the tokens");
  int sms = 0;
  st = device_sms(sms);
  if (st != STARKV_OK) return st;
  p.n_tok = n_tok;
  p.tok_seq = tok_seq;
  p.tok_pos = tok_pos;
  p.k_out = reinterpret_cast<uint16_t*>(k_out);
  p.v_out = reinterpret_cast<uint16_t*>(v_out);
  const cudaError_t e = launch_kv_gather(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv gather launch");
  return STARKV_OK;
}

starkv_status starkv_kv_select(const starkv_kv_layout* lay, const void* q, const void* cache,
                               int64_t num_pages, const int32_t* block_table, int32_t max_pages,
                               const int32_t* seq_lens, int32_t batch, int32_t n_sel,
                               int32_t keep_first, int32_t keep_last, int32_t* sel,
                               int32_t* dev_status, starkv_stream_t stream) {
  starkv_status st = check_kv_layout(lay);
  if (st != STARKV_OK) return st;
  if (batch < 0) return fail(STARKV_ERR_INVALID_ARG, "batch < 0");
  if (keep_first < 0 || keep_last < 1 || n_sel < 1 || keep_first > n_sel || keep_last > n_sel - keep_first)
    return fail(STARKV_ERR_INVALID_ARG, "needs keep_first >= 0, keep_last >= 1 and keep_first + keep_last <= n_sel");
  if (max_pages > STARKV_KV_MAX_SELECT_PAGES)
    return fail(STARKV_ERR_UNSUPPORTED, "at most 16384 pages per sequence");
  if (batch == 0) return STARKV_OK;
  KvSelectParams p;
  std::memset(&p, 0, sizeof(p));
  st = fill_pool(lay, cache, num_pages, block_table, max_pages, batch, dev_status, p.pool);
  if (st != STARKV_OK) return st;
  if (!q || !seq_lens || !sel) return fail(STARKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (misaligned(q)) return fail(STARKV_ERR_INVALID_ARG, "q must be 16-byte aligned");
  if (static_cast<int64_t>(batch) * p.pool.Hkv > (int64_t(1) << 27))
    return fail(STARKV_ERR_INVALID_ARG, "batch * n_kv_heads above 2^27");
  int sms = 0;
  st = device_sms(sms);
  if (st != STARKV_OK) return st;
  p.q = reinterpret_cast<const uint16_t*>(q);
  p.seq_lens = seq_lens;
  p.n_sel = n_sel;
  p.keep_first = keep_first;
  p.keep_last = keep_last;
  p.sel = sel;
  // CTAs per (sequence, KV head): four of them fit on an SM; none without a round of pages (64).  One, two
  // and sixteen took 30.7, 26.4 and 38.4 us at 32 x 512 pages and 8 KV heads (256 pairs; two by this rule),
  // one, four and sixteen 45.5, 18.7 and 12.5 at 1 x 2047 (8 pairs; sixteen).
  const int64_t units = static_cast<int64_t>(batch) * p.pool.Hkv;
  p.cluster = 1;
  while (p.cluster < kSelMaxCluster && units * p.cluster * 2 <= 4 * sms && p.cluster * 64 < max_pages) p.cluster *= 2;
  const cudaError_t e = launch_kv_select(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv select launch");
  return STARKV_OK;
}

starkv_status starkv_kv_decode(const starkv_kv_layout* lay, const void* q, const void* cache,
                               int64_t num_pages, const int32_t* block_table, int32_t max_pages,
                               const int32_t* seq_lens, int32_t batch, const int32_t* sel,
                               int32_t n_sel, const starkv_kv_decode_opts* opts, void* out, float* lse,
                               void* workspace, size_t workspace_bytes, int32_t* dev_status,
                               starkv_stream_t stream) {
  starkv_status st = check_kv_layout(lay);
  if (st != STARKV_OK) return st;
  const starkv_kv_decode_opts none = {};
  const starkv_kv_decode_opts& o = opts ? *opts : none;
  if (batch < 0 || batch > kKvMaxBatch) return fail(STARKV_ERR_INVALID_ARG, "batch outside [0, 65535]");
  if (!(o.scale >= 0.f) || o.scale > 1e38f) return fail(STARKV_ERR_INVALID_ARG, "scale must lie in [0, 1e38]");
  if (o.window < 0 || o.max_ctas < 0 || o.reserved != 0)
    return fail(STARKV_ERR_INVALID_ARG, "window or max_ctas < 0, or reserved not 0");
  if (sel && n_sel < 1) return fail(STARKV_ERR_INVALID_ARG, "n_sel < 1");
  if (sel && o.window > 0) return fail(STARKV_ERR_INVALID_ARG, "a selection and a window do not go together");
  if (batch == 0) return STARKV_OK;
  KvDecodeParams p;
  std::memset(&p, 0, sizeof(p));
  st = fill_pool(lay, cache, num_pages, block_table, max_pages, batch, dev_status, p.pool);
  if (st != STARKV_OK) return st;
  if (!q || !seq_lens || !out || !workspace) return fail(STARKV_ERR_INVALID_ARG, "NULL pointer argument");
  if (misaligned(q) || misaligned(out) || misaligned(workspace))
    return fail(STARKV_ERR_INVALID_ARG, "q, out and workspace must be 16-byte aligned");
  if (kv_tiles(lay, batch, max_pages) > kKvMostTiles)
    return fail(STARKV_ERR_INVALID_ARG, "batch * n_kv_heads * max_pages too large for one decode call");
  if (workspace_bytes < kv_record_bytes(lay, batch)) return fail(STARKV_ERR_WORKSPACE, "decode workspace too small");
  int sms = 0;
  st = device_sms(sms);
  if (st != STARKV_OK) return st;
  p.q = reinterpret_cast<const uint16_t*>(q);
  p.seq_lens = seq_lens;
  p.sel = sel;
  p.n_sel = n_sel;
  p.window = o.window;
  const float scale = o.scale > 0.f ? o.scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(p.pool.d)));
  p.scale2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.out = reinterpret_cast<uint16_t*>(out);
  p.lse = lse;
  p.groups = kv_groups(lay);
  // as many CTAs as fit on the device, and no more than there can be pages
  const int64_t most = static_cast<int64_t>(batch) * p.pool.Hkv * p.groups * (sel && n_sel < max_pages ? n_sel : max_pages);
  int64_t grid = static_cast<int64_t>(sms) * kv_split_ctas(p.pool.d);
  if (o.max_ctas > 0 && o.max_ctas < grid) grid = o.max_ctas;
  if (grid > kv_max_ctas(p.pool.d)) grid = kv_max_ctas(p.pool.d);
  if (grid > most) grid = most;
  p.grid = static_cast<int>(grid);
  p.counter = reinterpret_cast<unsigned*>(workspace);
  p.rec = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + kKvCounterBytes);
  p.rec_rows = kv_record_rows(lay);
  p.rec_ml = reinterpret_cast<float2*>(p.rec + static_cast<size_t>(kv_pieces(lay, batch)) * p.rec_rows * p.pool.d);
  const cudaError_t e = launch_kv_decode(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv decode launch");
  return STARKV_OK;
}

}  // extern "C"
