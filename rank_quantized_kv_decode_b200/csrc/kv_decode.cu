// Decode attention over the plain key-value cache: a split kernel and a join.
//
// Mathematics, per query head: s_t = scale q.k_t, o = sum_t e^{s_t} v_t / sum_t e^{s_t}, in one pass
// with a running reference m (log2 units): p_t = 2^{s_t log2e - m}, l = sum p_t, O = sum p_t v_t in
// fp32; raising m multiplies l and O by 2^{m_old - m_new}.  Parts of a sequence join by
// M = max m_i, l = sum l_i 2^{m_i - M}, O likewise.
//
// Bound: HBM.  Every byte of the visited keys and values is read once for each eight query heads of a KV
// head: a ninth makes the list twice as long (8 x 32768 bf16 tokens, d 128: 32 query over 4 KV heads take
// 96 us, 64 over 4 163; 64 over 8 174, 128 over 8 308).  4 FLOP per byte and query head at 16 bits; the
// products run on mma.sync m16n8k16, whose 16 rows hold the query heads in the upper half.  For P.V the
// lower half holds what the weights lost in rounding to 16 bits (p = hi + lo), so that the weights count
// with 16 bits of mantissa (bf16) or 22 (fp16) at no further instruction.  tcgen05 would give the same
// products of 8 rows a 128-row tile.
//
// Split: a warp works alone.  Its unit is a tile of 16 tokens (int8: 32) of one KV head; the tiles of all
// sequences and KV heads form one list, cut into chunks wherever the sequences begin, and a chunk's part
// of one sequence and head is a piece.  Lengths are known on the device only, so every warp derives the
// list from them.  Chunks are the same whoever takes them, so results do not hang on timing; who takes
// them does: warp w starts with the large chunk w and draws small ones from a counter.  (SMs get
// different shares of the memory's rate: with equal static shares of 32 x 32768 tokens they ended
// between 497 and 646 us; drawing the last quarter took the call from 652 to 612.)  A piece that is a
// whole sequence is written out at once, else as a partial record, and the join adds the records of a
// sequence in order.  Each warp has its own ring of tiles in shared memory, filled by cp.async, and no
// barrier with another: four warps that shared a page met once per piece, 1.6 us of a CTA's loads each.
// (TMA copies of the same tiles, issued by one lane: no faster at 32 x 32768 tokens and slower for short
// ones, 22.1 us against 19.4 at a ragged fp16 batch.)
//
// Measured, in a graph: 6.9 TB/s at 32 x 32768 bf16 tokens with 8 KV heads (621 us), 6.2 at 8 x 4096 with
// 32 (87 us: 4.6 us until the first tile and 3 of the join count there), 4.4 at 131072 int8 tokens (64.5 us).
// int8 has no unit near its limit (issue 48 %, DRAM 53 %, tensor pipe 26 %): two warps a scheduler (64 fp32
// sums a lane for d 128) do not cover one another's latencies while they decode codes; twelve warps an SM
// spilled and took 92 us.
#include <algorithm>

#include "kv.cuh"

namespace starkv {
namespace {

constexpr float kLazy = 8.f;  // the reference follows the running maximum when that is 2^8 above it:
                              // weights stay below 2^8, and O is rescaled a few times per sequence
// Tiles a warp above which some are drawn.  Drawing pays where the SMs' shares of the memory's rate differ by
// more than the small chunks cost: 32 x 32768 bf16 tokens (443 tiles a warp) took 612 us with it and 652
// without, 8 x 4096 with 32 KV heads (55) 88.6 and 92.8.  With d 128 and 8 KV heads in 8 sequences, drawing
// and equal shares took, in us: bf16 at 28 tiles 53.3 and 50.9, 44: 77.2 and 74.5, 64: 106 and 105, 96: 151 and
// 151; int8 at 28 70 and 63, 44: 105 and 92, 96: 201 and 184.  One number does not fit them all: 40 lies below the
// border of those lists.
constexpr unsigned kStatic = 40;
constexpr unsigned kDrawnPart = 4;  // one tile in so many is drawn: one in 2, 3, 4 took 634, 626, 621 us at 32 x 32768
constexpr int kSmall = 8;           // tiles of a drawn chunk at least (4: 92.3 us at 8 x 4096, 8: 90.2); at most
                                    // kKvRounds chunks a warp, about
constexpr float kLn2 = 0.69314718055994531f;

// Weights of fp16 products are scaled by 2^7 (the factor is part of the reference): with kLazy they
// stay below 2^15, and fp16's subnormals begin 2^-21 below the maximum instead of 2^-14.
template <int FMT>
constexpr float kShift = FMT == STARKV_KV_BF16 ? 0.f : 7.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// fp16, upper rows only, onto zero.
__device__ __forceinline__ void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, "
      "{%9,%9,%9,%9};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(0u), "r"(a2), "r"(b0), "r"(b1), "f"(0.f));
}

// Loads from shared memory that stay in order with the waits (volatile) but, unlike with a memory clobber, let
// everything else be scheduled around them.
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}

// 16 bytes global -> shared; zeros when not `on` (the address is not read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------ shape of a warp's ring
template <int FMT, int D>
struct Ring {
  static constexpr bool kInt8 = FMT == STARKV_KV_INT8;
  // Tokens of a tile: 16; int8, whose time is instructions, 32, so that the steps of a tile that are
  // not per token count half as much.
  static constexpr int kTok = kv_tile_tokens(FMT);
  static constexpr int kParts = kPage / kTok;  // tiles of a page
  static constexpr int kRow = kInt8 ? D : 2 * D;  // bytes of a token's keys (or values)
  static constexpr int kKeys = kTok * kRow;       // one tile's keys
  static constexpr int kScales = kInt8 ? kTok * (D / 32) * 2 : 0;
  static constexpr int kStage = 2 * kKeys + 2 * kScales;
  static constexpr int kCtas = kv_split_ctas(D);  // per SM
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kBytes = kStage * kStages;
  static constexpr int kSmem = kKvWarps * kBytes;
  // What a chunk's place changes by (exclusive or) from row r, below `rows`, to row r + rows, beside the
  // rows' pitch: chunk_at's permutation.
  static __device__ constexpr uint32_t turn(int rows) {
    return !kInt8 ? (rows & 7) << 4 : D == 128 ? (rows >> 1 & 2) << 5 : 0;
  }
};

// Offset of a 16-byte chunk of a tile's row in shared memory: the chunks are permuted so that the
// fragment loads touch every bank once.
template <bool INT8, int D>
__device__ __forceinline__ int chunk_at(int row, int c) {
  if (!INT8) return row * 2 * D + ((c ^ (row & 7)) << 4);
  if (D == 128) return row * D + (((c >> 1) ^ ((row ^ (row >> 1)) & 3)) << 5) + ((c & 1) << 4);
  return row * D + (((c >> 1) ^ ((row >> 1) & 1)) << 5) + ((c & 1) << 4);
}

// ------------------------------------------------------------------ the list of tiles
// Pages of a sequence that a call visits: [first, first + count) of the sequence, or count places
// of its selection.
struct Span {
  int len, first, count;
};
__device__ __forceinline__ Span span_of(const KvDecodeParams& p, int b) {
  Span s;
  s.len = min(max(p.seq_lens[b], 0), p.pool.max_pages * kPage);
  const int pages = (s.len + kPage - 1) / kPage;
  s.first = p.window > 0 ? max(0, s.len - p.window) / kPage : 0;
  s.count = p.sel ? min(pages, p.n_sel) : pages - s.first;
  return s;
}

// The list of tiles (at most 2^30: checked by the caller) and its chunks, the same in every warp and in
// the join: one large chunk for each warp, then small ones that the warps draw as they get there.
struct Cut {  // chunk i has base + 1 tiles where i < more, else base
  int n, base, more;
  __device__ __forceinline__ Cut() : n(0), base(1), more(0) {}
  __device__ __forceinline__ Cut(unsigned tiles, unsigned chunks)
      : n(chunks), base(tiles / chunks), more(tiles - chunks * (tiles / chunks)) {}
  __device__ __forceinline__ int start(int i) const { return i * base + min(i, more); }
  __device__ __forceinline__ int chunk_of(int u) const {
    const int edge = more * (base + 1);
    return u < edge ? u / (base + 1) : more + (u - edge) / base;
  }
};
struct List {
  int n, edge;  // chunks, tiles of the large ones
  Cut large, small;
  __device__ __forceinline__ int start(int i) const {
    return i < large.n ? large.start(i) : edge + small.start(i - large.n);
  }
  __device__ __forceinline__ int chunk_of(int u) const {
    return u < edge ? large.chunk_of(u) : large.n + small.chunk_of(u - edge);
  }
};
__device__ __forceinline__ List list_of(const KvDecodeParams& p, int lane, int per_page) {
  unsigned all = 0;
  for (int b = lane; b < p.pool.batch; b += 32) all += span_of(p, b).count;
  all = __reduce_add_sync(0xffffffffu, all) * (p.pool.Hkv * p.groups * per_page);
  List l;
  l.n = l.edge = 0;
  if (all == 0) return l;
  const unsigned warps = p.grid * kKvWarps;
  // SMs differ by a quarter in the bytes they get; below kStatic tiles a warp a share is too short to divide
  const unsigned rest = all > warps * kStatic ? all / kDrawnPart : 0;
  l.edge = all - rest;
  l.large = Cut(all - rest, min(all, warps));
  if (rest > 0) {
    const unsigned size = max((rest + warps * kKvRounds - 1) / (warps * kKvRounds), (unsigned)kSmall);
    l.small = Cut(rest, (rest + size - 1) / size);
  }
  l.n = l.large.n + l.small.n;
  return l;
}

// What a warp is loading: tiles of one piece.
struct Piece {
  int b, hv;            // sequence; KV head (and group of its query heads)
  int chunk, chunk_left;  // its chunk, and the tiles left of that
  int tile, left, size;   // next tile of the sequence's, tiles left of the piece, tiles of the sequence
  Span s;
  int page0, page, at;  // first page of the piece; of page `lane` of it: the block table's entry, and the
                        // index in the sequence (-1: none)
};

// Page numbers of the piece, one per lane (whole warp).
__device__ __forceinline__ void load_pages(const KvDecodeParams& p, Piece& c, int lane, int per_page) {
  c.page0 = c.tile / per_page;
  const int i = c.page0 + lane;
  c.page = -1;
  c.at = -1;
  if (i < c.s.count && i * per_page < c.tile + c.left) {
    c.at = c.s.first + i;
    if (p.sel) c.at = p.sel[((long long)c.b * p.pool.Hkv + c.hv / p.groups) * p.n_sel + i];
    if (c.at >= 0 && c.at < (c.s.len + kPage - 1) / kPage) {
      c.page = p.pool.block_table[(long long)c.b * p.pool.max_pages + c.at];  // looked at by page_of
    } else if (c.at != -1) {
      atomicOr(p.pool.status, STARKV_DEV_BOUNDS);
      c.at = -1;
    }
  }
}

// The first piece of a chunk (whole warp).
__device__ __forceinline__ Piece piece_of(const KvDecodeParams& p, const List& list, int lane, int per_page, int chunk) {
  Piece c;
  const int heads = p.pool.Hkv * p.groups;
  const int u = list.start(chunk);
  c.chunk = chunk;
  c.chunk_left = list.start(chunk + 1) - u;
  int before = 0;
  for (int b0 = 0;; b0 += 32) {
    const int b = b0 + lane;
    const int n = b < p.pool.batch ? span_of(p, b).count * heads * per_page : 0;
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const unsigned m = __ballot_sync(0xffffffffu, before + inc > u);
    if (m || b0 + 32 >= p.pool.batch) {  // found: u lies inside the list
      const int l = m ? __ffs(m) - 1 : 0;
      c.b = b0 + l;
      const int in = u - before - __shfl_sync(0xffffffffu, inc - n, l);
      c.s = span_of(p, c.b);
      c.size = c.s.count * per_page;
      c.hv = in / c.size;
      c.tile = in - c.hv * c.size;
      break;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  c.left = min(c.size - c.tile, c.chunk_left);
  load_pages(p, c, lane, per_page);
  return c;
}

// The next piece of the same chunk.
__device__ __forceinline__ void next_piece(const KvDecodeParams& p, Piece& c, int lane, int per_page) {
  c.tile = 0;
  if (++c.hv == p.pool.Hkv * p.groups) {
    c.hv = 0;
    do {
      c.s = span_of(p, ++c.b);
    } while (c.s.count == 0);
    c.size = c.s.count * per_page;
  }
  c.left = min(c.size, c.chunk_left);
  load_pages(p, c, lane, per_page);
}

// ------------------------------------------------------------------ loads
// The page that a warp is in: where the head's tile of it lies (null: none), and what counts of its 64
// rows: [lo, hi).
struct Page {
  const uint8_t* src;
  int lo, hi;
};
// Page i of the piece (whole warp).
__device__ __forceinline__ Page page_of(const KvDecodeParams& p, const Piece& c, int i) {
  Page t{nullptr, 0, 0};
  const int page = __shfl_sync(0xffffffffu, c.page, i - c.page0), at = __shfl_sync(0xffffffffu, c.at, i - c.page0);
  if (at < 0) return t;
  if (page < 0 || page >= p.pool.num_pages) {
    atomicOr(p.pool.status, STARKV_DEV_BOUNDS);
    return t;
  }
  t.src = p.pool.cache + page * p.pool.page_bytes + p.pool.off_heads + (long long)(c.hv / p.groups) * p.pool.head_bytes;
  t.hi = min(max(c.s.len - at * kPage, 0), kPage);
  t.lo = p.window > 0 ? min(max(c.s.len - p.window - at * kPage, 0), kPage) : 0;
  return t;
}

// Where a tile lies, and which of its rows count: [lo, hi).
struct Tile {
  const uint8_t* src;  // the head's tile of the page
  int lo, hi;
};
template <int TOK>
__device__ __forceinline__ Tile tile_of(const Page& g, int part) {
  return {g.src, min(max(g.lo - part * TOK, 0), TOK), min(max(g.hi - part * TOK, 0), TOK)};
}

template <int FMT, int D>
__device__ __forceinline__ void load_tile(const KvDecodeParams& p, const Tile& t, uint32_t stage, int part, int lane) {
  using R = Ring<FMT, D>;
  // round i takes chunk lane + 32 i: the row moves by 32 / CPR, the place in shared memory by 512 bytes and
  // the permutation's change, known here
  constexpr int CPR = R::kRow / 16, N = R::kTok * CPR / 32, step = 32 / CPR;
  const uint8_t* k = t.src + part * R::kKeys + lane * 16;
  const uint8_t* v = k + p.pool.off_v;
  const int row = lane / CPR;
  const uint32_t to = stage + chunk_at<R::kInt8, D>(row, lane % CPR);
  if (t.lo == 0 && t.hi == R::kTok) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t at = (to ^ R::turn(i * step)) + 512 * i;
      cp16(at, k + 512 * i);
      cp16(at + R::kKeys, v + 512 * i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t at = (to ^ R::turn(i * step)) + 512 * i;
      const bool on = row + i * step >= t.lo && row + i * step < t.hi;
      cp16(at, k + 512 * i, on);
      cp16(at + R::kKeys, v + 512 * i, on);
    }
  }
  if constexpr (R::kInt8) {
    constexpr int SC = R::kScales / 16;  // 16-byte chunks of a tile's scales (several tokens each)
    if (lane < 2 * SC) {
      const int which = lane / SC, i = lane % SC;
      cp16(stage + 2 * R::kKeys + lane * 16,
           t.src + (which ? p.pool.off_vs : p.pool.off_ks) + part * R::kScales + i * 16, true);
    }
  }
}

// ------------------------------------------------------------------ one warp's running sums
template <int FMT, int D>
struct Sums {
  static constexpr bool kInt8 = FMT == STARKV_KV_INT8;
  static constexpr bool kBf = FMT == STARKV_KV_BF16;
  static constexpr int kTok = Ring<FMT, D>::kTok, kHalves = kTok / 8;  // 8-token columns of products
  uint32_t q[D / 16][2];  // A fragments of the queries: rows 0..7 (the lower half is zero)
  float qs;               // factor of the dot products: scale log2(e), int8: times the query's power of two
  float o[D / 8][4];      // O: [0,1] of the weights' high part, [2,3] of the low part
  float m, l;             // of row lane / 4; l is this lane's share

  __device__ __forceinline__ void begin(const KvDecodeParams& p, int b, int hv, int lane) {
    const int g = hv / p.groups, G = p.pool.H / p.pool.Hkv;
    const int row = hv % p.groups * kKvRows + lane / 4, t = lane % 4;
    const bool in = row < G;
    const uint16_t* src = p.q + ((long long)b * p.pool.H + g * G + (in ? row : 0)) * D;
    qs = p.scale2;
    if (!kInt8) {
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          q[s][i] = in ? *reinterpret_cast<const uint32_t*>(src + 16 * s + 8 * i + 2 * t) : 0u;
    } else {
      // fp16 queries: scaled by a power of two to a magnitude near 1, so that bf16's eight bits are
      // exact down to 2^-16 of the largest.  Channels 32 j + 8 t + (0..7) of scale group j.
      float x[D / 32][8], mx = 0.f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + 32 * j + 8 * t);
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = kv_unpack<STARKV_KV_BF16>(a[i]);
          x[j][2 * i] = in ? f.x : 0.f, x[j][2 * i + 1] = in ? f.y : 0.f;
          mx = fmaxf(mx, fmaxf(fabsf(x[j][2 * i]), fabsf(x[j][2 * i + 1])));
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = min(max(__float_as_int(mx) >> 23, 1), 253);
      const float down = __int_as_float((254 - e) << 23);
      qs *= __int_as_float(e << 23);
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[2 * j + i / 2][i % 2] = kv_pack<STARKV_KV_F16>(x[j][2 * i] * down, x[j][2 * i + 1] * down);
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m = __int_as_float(0xff800000);
    l = 0.f;
  }

  // Scores (dot products) of the tile's tokens 8 h + 2t, 8 h + 2t + 1 for row lane / 4.
  __device__ __forceinline__ void scores(uint32_t stage, int lane, float (&s)[2 * kHalves]) const {
    using R = Ring<FMT, D>;
    if constexpr (!kInt8) {
      const int mi = lane / 8;
      const uint32_t from = stage + chunk_at<false, D>(lane % 8 + 8 * (mi >> 1), mi & 1);
#pragma unroll
      for (int h = 0; h < kHalves; h += 2) {
        float c[2][4] = {};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t f[4];
          ldsm4(f, (from ^ (k << 5)) + 8 * h * R::kRow);
          mma16816<kBf>(c[0], q[k][0], 0u, q[k][1], 0u, f[0], f[1]);
          mma16816<kBf>(c[1], q[k][0], 0u, q[k][1], 0u, f[2], f[3]);
        }
        s[2 * h] = c[0][0], s[2 * h + 1] = c[0][1], s[2 * h + 2] = c[1][0], s[2 * h + 3] = c[1][1];
      }
    } else {
      const int g = lane / 4, t = lane % 4;
      const uint32_t from = stage + chunk_at<true, D>(g, 0) + 8 * t;
      const uint32_t sc = stage + 2 * R::kKeys + 2 * t * (D / 16);
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        // the fp32 scales of this lane's two result columns
        float f[2][D / 32];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[2];
          if constexpr (D == 128) {
            const uint2 x = lds64(sc + (8 * h + i) * (D / 16));
            w[0] = x.x, w[1] = x.y;
          } else {
            w[0] = lds32(sc + (8 * h + i) * (D / 16));
          }
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            const float2 x = kv_unpack<STARKV_KV_F16>(w[j]);
            f[i][2 * j] = x.x, f[i][2 * j + 1] = x.y;
          }
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint2 w = lds64((from ^ (j << 5)) + 8 * h * R::kRow);
          uint32_t x[4];
          halves(w.x, x[0], x[1]);
          halves(w.y, x[2], x[3]);
          float c[4];
          mma16816_zero(c, q[2 * j][0], q[2 * j][1], x[0], x[1]);
          mma16816<false>(c, q[2 * j + 1][0], 0u, q[2 * j + 1][1], 0u, x[2], x[3]);
          s[2 * h] = j ? fmaf(c[0], f[0][j], s[2 * h]) : c[0] * f[0][j];
          s[2 * h + 1] = j ? fmaf(c[1], f[1][j], s[2 * h + 1]) : c[1] * f[1][j];
        }
      }
    }
  }

  // Four codes as fp16 pairs, exact: code + 128 under the exponent of 1024, minus 1152.
  static __device__ __forceinline__ uint32_t less1152(uint32_t w) {
    const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&w), k);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ void halves(uint32_t codes, uint32_t& a, uint32_t& b) {
    const uint32_t u = codes ^ 0x80808080u;
    a = less1152(__byte_perm(u, 0x64646464u, 0x4140));
    b = less1152(__byte_perm(u, 0x64646464u, 0x4342));
  }

  // Adds the tile's rows [lo, hi) of keys and values at `stage`.
  __device__ __forceinline__ void add(uint32_t stage, int lo, int hi, int lane) {
    using R = Ring<FMT, D>;
    constexpr int N = 2 * kHalves;  // scores of a lane
    const int t = lane % 4;
    float s[N];
    scores(stage, lane, s);
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] *= qs;
    const bool partial = lo > 0 || hi < kTok;
    if (partial) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = 2 * t + (i & 1) + 8 * (i >> 1);
        if (row < lo || row >= hi) s[i] = __int_as_float(0xff800000);
      }
    }
    float mx = fmaxf(s[0], s[1]);
#pragma unroll
    for (int i = 2; i < N; i += 2) mx = fmaxf(mx, fmaxf(s[i], s[i + 1]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    mx -= kShift<FMT>;  // m carries the shift: weights are 2^(s - m)
    const bool up = mx > m + kLazy;
    if (__any_sync(0xffffffffu, up)) {
      const float f = up ? ex2(m - mx) : 1.f;
      if (up) m = mx;
      l *= f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] *= f, o[i][1] *= f, o[i][2] *= f, o[i][3] *= f;
    }
    const float ref = m == __int_as_float(0xff800000) ? 0.f : m;
    // weights as hi + lo in 16 bits: rows 0..7 and 8..15 of the A fragments
    constexpr int PF = kBf ? STARKV_KV_BF16 : STARKV_KV_F16;
    uint32_t ah[kHalves], al[kHalves];
#pragma unroll
    for (int i = 0; i < kHalves; ++i) {
      const float w0 = ex2(s[2 * i] - ref), w1 = ex2(s[2 * i + 1] - ref);
      l += w0 + w1;
      ah[i] = kv_pack<PF>(w0, w1);
      const float2 h = kv_unpack<PF>(ah[i]);
      al[i] = kv_pack<PF>(w0 - h.x, w1 - h.y);
    }
    const uint32_t vs = stage + R::kKeys;
    if constexpr (!kInt8) {
      const int mi = lane / 8;
      const uint32_t from = vs + chunk_at<false, D>(lane % 8 + 8 * (mi & 1), mi >> 1);
#pragma unroll
      for (int h = 0; h < kHalves; h += 2)
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t f[4];
          ldsm4t(f, (from ^ (n << 5)) + 8 * h * R::kRow);
          mma16816<kBf>(o[2 * n], ah[h], al[h], ah[h + 1], al[h + 1], f[0], f[1]);
          mma16816<kBf>(o[2 * n + 1], ah[h], al[h], ah[h + 1], al[h + 1], f[2], f[3]);
        }
    } else {
      // Column n = lane / 4 of product (jj, i) is channel 8 (n + 8 jj) + i: a lane decodes eight
      // neighbouring channels of four tokens, code times scale rounded once to fp16.
      const int g = lane / 4;
      uint32_t sc = stage + 2 * R::kKeys + R::kScales;
      if (partial) {  // whatever the scales of rows that do not count hold
        for (int i = lane; i < R::kScales / 4; i += 32) {
          const int r = i / (D / 64);
          if (r < lo || r >= hi) asm volatile("st.shared.u32 [%0], %1;" ::"r"(sc + 4 * i), "r"(0u) : "memory");
        }
        __syncwarp();
      }
      sc += 2 * t * (D / 16) + 2 * (g >> 2);
      // rows 2t and 2t + 1, unit g of eight channels
      const uint32_t fx = vs + chunk_at<true, D>(2 * t, g >> 1) + 8 * (g & 1);
      const uint32_t fy = vs + chunk_at<true, D>(2 * t + 1, g >> 1) + 8 * (g & 1);
#pragma unroll
      for (int h = 0; h < kHalves; h += 2)
#pragma unroll
        for (int jj = 0; jj < D / 64; ++jj) {
          uint32_t b[2][8];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint2 x = lds64((fx ^ (jj << 6)) + 8 * (h + e) * R::kRow);
            const uint2 y = lds64((fy ^ (jj << 6)) + 8 * (h + e) * R::kRow);
            const uint32_t at = sc + 8 * (h + e) * (D / 16) + 4 * jj;
            const uint32_t f2 = __byte_perm(lds16(at), lds16(at + D / 16), 0x5410);
            const __half2 f = *reinterpret_cast<const __half2*>(&f2);
#pragma unroll
            for (int w2 = 0; w2 < 2; ++w2) {
              const uint32_t xa = (w2 ? x.y : x.x) ^ 0x80808080u, ya = (w2 ? y.y : y.x) ^ 0x80808080u;
              const uint32_t z[2] = {__byte_perm(xa, ya, 0x5140), __byte_perm(xa, ya, 0x7362)};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t c = less1152(__byte_perm(z[i / 2], 0x64646464u, i % 2 ? 0x4342 : 0x4140));
                const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&c), f);
                b[e][4 * w2 + i] = *reinterpret_cast<const uint32_t*>(&r);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            mma16816<false>(o[8 * jj + i], ah[h], al[h], ah[h + 1], al[h + 1], b[0][i], b[1][i]);
        }
    }
  }

  // The sums of the piece of (b, hv): the result where it is the whole sequence, else a record.  They go
  // through the warp's free stage `at`, so that rows leave in whole lines (64 stores of 8 bytes a lane
  // from the fragments took 2.6 us).
  __device__ __forceinline__ void end(const KvDecodeParams& p, int b, int hv, bool whole, int chunk, uint8_t* at, int lane) {
    constexpr int kPitch = D + 8, kLanes = D / 4;  // floats of a row (rows a quarter of the banks apart); lanes of a row
    static_assert(kKvRows * kPitch * 4 <= Ring<FMT, D>::kStage, "a stage takes the sums");
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const int g = lane / 4, t = lane % 4, G = p.pool.H / p.pool.Hkv;
    const int head0 = hv % p.groups * kKvRows, rows = min(G - head0, kKvRows);
    const long long row0 = (long long)b * p.pool.H + hv / p.groups * G + head0;
    const long long rec0 = ((long long)chunk + (long long)b * p.pool.Hkv * p.groups + hv) * p.rec_rows;
    const float inv = m == __int_as_float(0xff800000) ? 0.f : 1.f / l;
    if (t == 0 && g < rows) {
      if (!whole) p.rec_ml[rec0 + g] = make_float2(m, l);
      else if (p.lse) p.lse[row0 + g] = kLn2 * (m + log2f(l));
    }
    float* mine = reinterpret_cast<float*>(at) + g * kPitch;
    if constexpr (!kInt8) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(mine + 8 * n + 2 * t) = make_float2(o[n][0] + o[n][2], o[n][1] + o[n][3]);
    } else {
#pragma unroll
      for (int jj = 0; jj < D / 64; ++jj)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 8; i += 4)
            *reinterpret_cast<float4*>(mine + 8 * (2 * t + e + 8 * jj) + i) =
                make_float4(o[8 * jj + i][e] + o[8 * jj + i][e + 2], o[8 * jj + i + 1][e] + o[8 * jj + i + 1][e + 2],
                            o[8 * jj + i + 2][e] + o[8 * jj + i + 2][e + 2], o[8 * jj + i + 3][e] + o[8 * jj + i + 3][e + 2]);
    }
    __syncwarp();
    for (int r0 = 0; r0 < rows; r0 += 32 / kLanes) {
      const int r = r0 + lane / kLanes, c = lane % kLanes;
      const float f = __shfl_sync(0xffffffffu, inv, 4 * min(r, kKvRows - 1));
      if (r < rows) {
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(at) + r * kPitch + 4 * c);
        if (whole)
          reinterpret_cast<uint2*>(p.out + (row0 + r) * D)[c] = make_uint2(kv_pack<FMT>(v.x * f, v.y * f), kv_pack<FMT>(v.z * f, v.w * f));
        else
          reinterpret_cast<float4*>(p.rec + (rec0 + r) * D)[c] = v;
      }
    }
  }
};

// Weight of a part with reference m under the common reference M (-inf: nothing there).
__device__ __forceinline__ float part_weight(float m, float M) {
  return m == __int_as_float(0xff800000) ? 0.f : ex2(m - M);
}


// Sets the counter of chunks drawn to zero before a split kernel that may draw, whatever the workspace holds.
// In a graph it adds 0.3 us to 8 x 1000 tokens under a block table of 2048 pages (11.6 us), outside 1 us.
__global__ void kv_counter_kernel(unsigned* counter) {
  pdl_launch_dependents();
  pdl_wait();
  *counter = 0;
}

template <int FMT, int D>
__global__ void __launch_bounds__(32 * kKvWarps, Ring<FMT, D>::kCtas) kv_split_kernel(const KvDecodeParams p) {
  using R = Ring<FMT, D>;
  extern __shared__ __align__(1024) uint8_t smem[];  // the fragments' addresses are formed by exclusive or
  // what the tile in a stage of a warp's ring is: sequence, KV head, chunk, and [lo, hi) with flags
  __shared__ int4 s_what[kKvWarps][R::kStages];
  constexpr int kFirst = 1 << 16, kLast = 1 << 17, kWhole = 1 << 18, kThere = 1 << 19;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t ring = smem_u32(smem) + warp * R::kBytes;
  const int worker = blockIdx.x * kKvWarps + warp, workers = gridDim.x * kKvWarps;

  pdl_wait();
  pdl_launch_dependents();
  const List list = list_of(p, lane, R::kParts);
  if (worker >= list.n) return;
  Piece c = piece_of(p, list, lane, R::kParts, worker);
  unsigned drawn = 0;  // lane 0: the draw of the chunk after c's, made when c's begins
  auto draw = [&]() {
    if (lane == 0 && list.n > workers) drawn = atomicAdd(p.counter, 1u);
  };
  draw();
  int wr = 0, rd = 0;
  bool first = true, whole = false;  // the next tile is its piece's first; the piece is a whole sequence
  bool on = true;                    // there are tiles left
  Page page;
  auto issue = [&]() {
    int4 what = make_int4(0, 0, 0, 0);
    if (on) {
      const int part = c.tile % R::kParts;
      if (first || part == 0) page = page_of(p, c, c.tile / R::kParts);
      const Tile t = tile_of<R::kTok>(page, part);
      if (t.lo < t.hi) load_tile<FMT, D>(p, t, ring + wr * R::kStage, part, lane);
      what = make_int4(c.b, c.hv, c.chunk, t.lo | t.hi << 8 | kThere);
      if (first) what.w |= kFirst, whole = c.left == c.size;
      if (whole) what.w |= kWhole;
      first = false;
      ++c.tile, --c.left, --c.chunk_left;
      if (c.left == 0) {
        what.w |= kLast;
        first = true;
        if (c.chunk_left > 0) {
          next_piece(p, c, lane, R::kParts);
        } else {
          int id = list.n;
          // chunks drawn before it: at most one past the end for each warp
          if (list.n > workers) id = workers + static_cast<int>(__shfl_sync(0xffffffffu, drawn, 0));
          on = id < list.n;
          if (on) {
            draw();
            c = piece_of(p, list, lane, R::kParts, id);
          }
        }
      } else if (c.tile == (c.page0 + 32) * R::kParts) {
        load_pages(p, c, lane, R::kParts);
      }
    }
    if (lane == 0) s_what[warp][wr] = what;
    cp_commit();
    wr = wr + 1 == R::kStages ? 0 : wr + 1;
  };
#pragma unroll
  for (int i = 0; i < R::kStages - 1; ++i) issue();

  Sums<FMT, D> sums;
  for (;;) {
    issue();
    cp_wait<R::kStages - 1>();
    __syncwarp();
    const int4 what = s_what[warp][rd];
    if (!(what.w & kThere)) break;
    if (what.w & kFirst) sums.begin(p, what.x, what.y, lane);
    const int lo = what.w & 255, hi = what.w >> 8 & 255;
    if (lo < hi) sums.add(ring + rd * R::kStage, lo, hi, lane);
    if (what.w & kLast)
      sums.end(p, what.x, what.y, what.w & kWhole, what.z, smem + warp * R::kBytes + rd * R::kStage, lane);
    __syncwarp();  // the stage is free for the next issue
    rd = rd + 1 == R::kStages ? 0 : rd + 1;
  }
  cp_wait<0>();
}

// Joins the records of the sequences that several chunks shared; writes zeros for empty ones.  One CTA
// per (sequence, query head); a record is read by eight lanes (D / 8 channels each), so that the eight
// warps read 32 records a round, four rounds in flight.
constexpr int kJoinWarps = 8;
template <int FMT, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_join_kernel(const KvDecodeParams p) {
  constexpr int N4 = D / 32;  // 16-byte loads of a lane's share of a record
  __shared__ float s_l[kJoinWarps], s_acc[kJoinWarps][D];
  const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32, part = lane % 8;
  const int G = p.pool.H / p.pool.Hkv, heads = p.pool.Hkv * p.groups;
  const int g = h / G, hv = g * p.groups + h % G / kKvRows, r = h % G % kKvRows;
  constexpr int per_page = Ring<FMT, D>::kParts;
  // The lengths may be read before the wait: the split kernel, which does not write them, let this one
  // start only after its own wait for all that came before.
  const long long row = (long long)b * p.pool.H + h;
  const int raw = p.seq_lens[b], count = span_of(p, b).count;
  const List list = list_of(p, lane, per_page);
  int before = 0;
  for (int i = lane; i < b; i += 32) before += span_of(p, i).count;
  before = __reduce_add_sync(0xffffffffu, before) * heads * per_page + hv * count * per_page;
  // the chunks of this head's tiles
  const int c0 = count ? list.chunk_of(before) : 0, c1 = count ? list.chunk_of(before + count * per_page - 1) : 0;
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0 && h == 0 && (raw < 0 || raw > p.pool.max_pages * kPage)) atomicOr(p.pool.status, STARKV_DEV_BOUNDS);
  if (count == 0) {
    if (threadIdx.x < D / 2) reinterpret_cast<uint32_t*>(p.out + row * D)[threadIdx.x] = 0;
    if (p.lse && threadIdx.x == 0) p.lse[row] = __int_as_float(0xff800000);
    return;
  }
  if (c0 == c1) return;
  const long long rec0 = (long long)b * heads + hv;
  auto at = [&](int i) { return (rec0 + i) * p.rec_rows + r; };
  float M = __int_as_float(0xff800000);
  for (int i = c0 + lane; i <= c1; i += 32) M = fmaxf(M, p.rec_ml[at(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float l = 0.f, acc[4 * N4] = {};
#pragma unroll 4
  for (int i = c0 + threadIdx.x / 8; i <= c1; i += 4 * kJoinWarps) {
    const float2 x = p.rec_ml[at(i)];
    const float f = part_weight(x.x, M);
    l = fmaf(f, x.y, l);
    const float4* rec = reinterpret_cast<const float4*>(p.rec + at(i) * D) + part;
#pragma unroll
    for (int k = 0; k < N4; ++k) {
      const float4 v = rec[8 * k];
      acc[4 * k] = fmaf(f, v.x, acc[4 * k]), acc[4 * k + 1] = fmaf(f, v.y, acc[4 * k + 1]);
      acc[4 * k + 2] = fmaf(f, v.z, acc[4 * k + 2]), acc[4 * k + 3] = fmaf(f, v.w, acc[4 * k + 3]);
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int k = 0; k < 4 * N4; ++k) acc[k] += __shfl_xor_sync(0xffffffffu, acc[k], o);
  }
  if (lane < 8) {
#pragma unroll
    for (int k = 0; k < N4; ++k)
      *reinterpret_cast<float4*>(&s_acc[warp][32 * k + 4 * part]) =
          make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
  }
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (threadIdx.x < D / 2) {
    float x = 0.f, y = 0.f;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      l += s_l[w];
      x += s_acc[w][2 * threadIdx.x], y += s_acc[w][2 * threadIdx.x + 1];
    }
    const float inv = M == __int_as_float(0xff800000) ? 0.f : 1.f / l;
    reinterpret_cast<uint32_t*>(p.out + row * D)[threadIdx.x] = kv_pack<FMT>(x * inv, y * inv);
    if (p.lse && threadIdx.x == 0) p.lse[row] = kLn2 * (M + log2f(l));
  }
}

// Whether some lengths make a list of this call that is drawn from (see list_of).
bool may_draw(const KvDecodeParams& p, int per_page) {
  long long pages = p.pool.max_pages;
  if (p.sel) pages = std::min<long long>(pages, p.n_sel);
  else if (p.window > 0) pages = std::min(pages, (p.window - 1LL + kPage - 1) / kPage + 1);
  return pages * p.pool.batch * p.pool.Hkv * p.groups * per_page > static_cast<long long>(p.grid) * kKvWarps * kStatic;
}

template <int FMT, int D>
cudaError_t decode_launch(const KvDecodeParams& p, cudaStream_t s) {
  using R = Ring<FMT, D>;
  static_assert(R::kCtas * (R::kSmem + 2048) <= 228 * 1024, "the CTAs of an SM share its memory");
  cudaError_t e = cudaFuncSetAttribute(kv_split_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem);
  if (e == cudaSuccess && may_draw(p, R::kParts)) e = launch_pdl(kv_counter_kernel, dim3(1), dim3(1), 0, s, p.counter);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kv_split_kernel<FMT, D>, dim3(p.grid), dim3(32 * kKvWarps), R::kSmem, s, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv_join_kernel<FMT, D>, dim3(p.pool.H, p.pool.batch), dim3(32 * kJoinWarps), 0, s, p);
}

}  // namespace

cudaError_t launch_kv_decode(const KvDecodeParams& p, cudaStream_t s) {
  const int d = p.pool.d;
  switch (p.pool.fmt) {
    case STARKV_KV_BF16: return d == 64 ? decode_launch<STARKV_KV_BF16, 64>(p, s) : decode_launch<STARKV_KV_BF16, 128>(p, s);
    case STARKV_KV_F16: return d == 64 ? decode_launch<STARKV_KV_F16, 64>(p, s) : decode_launch<STARKV_KV_F16, 128>(p, s);
    case STARKV_KV_INT8: return d == 64 ? decode_launch<STARKV_KV_INT8, 64>(p, s) : decode_launch<STARKV_KV_INT8, 128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace starkv
