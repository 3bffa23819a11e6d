// Decode attention of drafted-token trees over the paged, compressed cache.
//
// For node i of a sequence with L cached tokens, at position pos = L + depth:
//   s_hj = sm_scale q_h . v_j,  p = softmax_j(s),  o_h = sum_j p_hj v_j
// over the entries j < floor(max(0, pos + 1 - W) / r) (or the node's top-k),
// the cached tokens [max(0, pos + 1 - W), L) and the node's ancestors with
// itself; then the inverse RoPE at pos, and bf16.
//
// Work is cut into units of up to 64 rows (a row is one node's head): rows of
// one sequence in order, or of one node where every node reads its own top-k
// or heads is a multiple of 64. Per tile of 128 items a unit computes
//   S^T[128 items x 64 rows] = V . Q^T     and     O^T[512 x 64] += V^T . P^T
// on tcgen05. One entry meets hundreds of rows, so the operator is bound by
// the products, and those by the shared-memory bytes of their operands: an
// MMA of M = 128, N = 64, K = 32 bytes reads 6 KB, 48 cycles, against 32 of
// math. Everything follows from keeping those bytes low:
//   - V stays as its fp8 codes, the K-major A of the first product and the
//     MN-major A of the second from one copy. Nothing is converted, and an
//     item costs 512 bytes, not 1024.
//   - q and P are two e4m3 terms each, hi + lo / 16: four significant bits
//     and four of what is left, 2^-9 of a value (and 2^-11, split2), where bf16
//     keeps 2^-8 and an f16 operand 2^-11; a bf16 q is exact. Two fp8 products
//     cost what one f16 product does, but V need not be converted: a third term, or
//     f16 operands, would cost half of the products again, or V's bytes twice. Against
//     fp64 the outputs are off by 0.0017 to 0.0019 (relative, all of a case), the plain
//     form in fp32 by 0.0017: the bf16 result. q's two terms are one N = 128 operand, so
//     V is read once for both.
//   - A bf16 row (window token, drafted token, bf16 entry) is two images hi and
//     lo of the same kind, scaled by a power of two: two fp8 tiles.
//   - e4m3 spans 2^-9 .. 448. P's terms carry a power-of-two scale for each row
//     and 32 items (the block scale of mxf8f6f4), so a weight keeps its
//     precision next to a dominating one elsewhere. Without it a long tail of
//     small weights would round to zero together.
// The normaliser and the running reference are fp32. With block scales P needs
// no fixed range, so the reference moves only when a score passes it by 2^20.
//
// Warps: 0-15 softmax (a thread has 4 items of the tile and 4 of the rows) and
// the unit's epilogue, 16-19 load tiles, 20 issues the MMAs, 21 and 22 resolve
// the even and odd tiles' row addresses ahead, 23 loads the units' Q. The prep
// kernel has written every Q as the image its products read, and every raw row
// as its two terms, once for all units that use it.
//
// Loads: entries that every node sees come as TMA boxes of 64 rows (fp8 pages of
// ratio 4, or rows that the prep kernel gathered: staged_rows), other rows by
// 16-byte asynchronous copies. A row of 512 bytes a request would suit neither:
// a TMA instruction takes about 50 cycles whatever it brings.
//
// Schedule: the tiles of all units are one list; the prep kernel gives each
// block of the grid (one per SM) an equal share by estimated cost. A block that
// runs all tiles of a unit writes its output, any other leaves a partial result
// (O, m, l) that the merge kernel joins: a long context with few rows is split
// over the whole GPU.
//
// Measured (work is 2 x 2 x 512 flops per node, head and item), in calls in a row: 64
// sequences of 4K to 64K tokens, 8 nodes, 64 heads 870 to 890 us, 670 TFLOP/s, at the power
// limit's clock (730 to 760 us in a short burst of graph replays); one of 131001 tokens
// with 31 nodes 180 us, 740 TFLOP/s (168 to 171 in a burst). A tile takes 4300 cycles:
// 3200 of them are its operands and its own 64 KB at 128 bytes a cycle, the rest is the
// part of the softmax that the next scores do not cover. Small calls take 31 to 33 us, the
// latency of three dependent launches with code that each block runs once; the
// loops are kept short for that, and in steady state too: unrolled ones lost 3 to 8
// percent to instruction fetch.
#include "tc.cuh"
#include "tree.cuh"

namespace v4kv {

namespace {

constexpr int kR = 64;    // rows of a unit
constexpr int kT = 128;   // items of a tile
constexpr int kD = 512;
constexpr int kThreads = 768;
constexpr int kRing = 4;  // tiles whose rows are resolved ahead
constexpr float kNone = -1e30f;  // reference of a row that has seen nothing
constexpr float kRaise = 20.f;   // log2 by which a score may pass its reference
constexpr int kPairs = 256;     // rotated pairs of a row at most
constexpr int kPrepRows = 4;    // rows a warp of the prep kernel splits
constexpr int kStageRows = 8;   // entries it copies

// shared memory (bytes from a 1024-aligned base)
constexpr uint32_t kQOff = 0;                 // 4 x [128 rows (64 hi, 64 lo) x 128 dims]
constexpr uint32_t kVOff = 65536;             // 2 stages of 4 x [128 items x 128 dims]
constexpr uint32_t kStage = 65536;
constexpr uint32_t kChunk = 16384;
constexpr uint32_t kPOff = 196608;            // [128 items x (64 hi, 64 lo)]
constexpr uint32_t kMetaOff = 212992;         // [kRing][128] {scale, log2 |scale|, 1 / |scale|, 0 or -inf}
constexpr uint32_t kPtrOff = kMetaOff + kRing * 2048;  // [kRing][128] row addresses
constexpr uint32_t kRowOff = kPtrOff + kRing * 1024; // [64] the rows' references
constexpr uint32_t kAncOff = kRowOff + 512;   // [64] ancestors of the row's node, 128 bits
constexpr uint32_t kVisOff = kAncOff + 1024;  // [64] {visible entries, first visible token, node}
constexpr uint32_t kRedOff = kVisOff + 1024;  // [2][4][32] reductions over a warp's items
constexpr uint32_t kSfOff = kRedOff + 1024;   // [64] block scales of P, a byte per 32 items
constexpr uint32_t kFacOff = kSfOff + 256;    // [64] per-row factors
constexpr uint32_t kBarOff = kFacOff + 256;
constexpr uint32_t kMiscOff = kBarOff + 320;
constexpr uint32_t kSmemBytes = kMiscOff + 64 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory per block");

// tensor-memory columns
constexpr uint32_t kOCol = 0;      // O^T: 4 x 64
constexpr uint32_t kSCol = 256;    // S^T: 64 of the hi terms, 64 of the lo terms
constexpr uint32_t kOne = 384;     // block scales 1 (four columns each from here on)
constexpr uint32_t kLow = 388;     // block scales 1/16
constexpr uint32_t kSfQ = 392;     // q: 64 rows of 1, 64 of 1/16
constexpr uint32_t kSfHi = 396;    // P
constexpr uint32_t kSfLo = 400;
constexpr uint32_t kCols = 512;

struct Bars {
  uint64_t kv_full[2][4];   // per stage and 128 dims
  uint64_t kv_empty[2][2];  // per stage and 256 dims
  uint64_t addr_full[kRing], addr_free[kRing];
  uint64_t raw_full;        // bf16 entries have landed, to be split
  uint64_t ready, q_full, q_empty, s_full, s_free, p_full, pv_done, drain;
};
static_assert(sizeof(Bars) <= 320, "barrier area");

// What the prep kernel leaves in the workspace.
struct TreeWs {
  uint4* anc;         // [total_nodes] the node and its ancestors, a bit each
  int32_t* depth;     // [total_nodes]
  float2* rope;       // [total_nodes][rope_dim / 2] cos, sin at the node's position
  uint8_t* q;         // the units' Q as shared-memory images, 64 KB each
  float* q_factor;    // their rows' score factors, 64 each
  int4* units;        // [images][4] Unit's fields
  uint8_t* raw;       // rows of the windows and trees as two e4m3 terms, 512 bytes each
  float2* raw_meta;   // their {scale, 0 or -inf: no such row}
  uint8_t* ent;       // gathered entries (staged): 512 bytes each, or two e4m3 terms of a bf16 one
  float2* ent_meta;   // their {scale, 0 or -inf: no such row}
  long long* cost;    // [batch + 1] prefix sums over sequences
  int32_t* tiles;     // [batch + 1]
  int4* rec;          // [grid + 1] a block's first tile: {index, its unit, -, tile in that}
  float* part_o;      // [2 grid][64][512]
  float2* part_ml;    // [2 grid][64]
};

struct Params {
  TreeArgs a;
  TreeWs w;
  int grid;
  int ratio_log, spb_log;  // of main_cache
  int hc;        // units per node (per_node)
  int per_node;  // a unit's rows belong to one node: own top-k, or as 64 heads fill it; then only its ancestors are listed, and nothing is masked
  int rope_blocks; // prep blocks per sequence for its nodes
  int raw_blocks;  // prep blocks per sequence for its raw rows
  int max_units;   // units of a sequence at most
  int boxes;     // tiles of entries that every node sees are loaded by TMA
  int staged;    // entries of a sequence in w.ent, 0: the boxes are pages
  const uint8_t* box_data;  // what they are taken from, and its rows
  int box_rows, box_bytes;
  CUtensorMap map;  // boxes of 64 rows x 128 bytes of box_data
};

__device__ __forceinline__ int seq_len(const TreeArgs& a, int b) {
  return min(max(a.seq_lens[b], 0), a.max_len);
}

// Tile counts and costs of a sequence's units (all of one sequence alike).
struct SeqPlan {
  TreeSeq s;
  int L, units, te, tr;
};

// The raw rows of a sequence in the workspace, consecutive: the cached tokens
// that any node sees, then the nodes.
__device__ __forceinline__ size_t raw_row0(const TreeArgs& a, const SeqPlan& q, int b) {
  return (size_t)b * min(a.window_len - 1, a.max_len) + q.s.first;
}
__device__ __forceinline__ int raw_w0(const TreeArgs& a, const SeqPlan& q) {
  return min(q.L, max(0, q.L + 1 - a.window_len));
}

// A unit's index, of its Q image and its fields: consecutive within a sequence
// and distinct, as a sequence's units are at most one more than its rows fill.
__device__ __forceinline__ int unit_index(const Params& p, const SeqPlan& q, int b, int u) {
  return p.per_node ? q.s.first * p.hc + u : b + (int)((long long)q.s.first * p.a.heads / kR) + u;
}

// Costs of a tile of fp8 entries, of a tile of two images and of a unit, in about
// 540 cycles. They balance the blocks, and were fitted: against 8, 16 and 8
// (the images' bytes) 64 sequences of 4K to 64K tokens take 727 us, not 752, and 32
// of 128K to 1M tokens at ratio 128 take 370, not 385; small calls are as before.
constexpr int kCostFp8 = 8, kCostTwo = 22, kCostSeg = 16;

__device__ __forceinline__ SeqPlan plan_of(const Params& p, int b, int32_t* st) {
  const TreeArgs& a = p.a;
  SeqPlan q;
  q.s = tree_seq(a.cu_nodes, b, a.total_nodes, a.max_nodes, st);
  q.L = seq_len(a, b);
  const int n = q.s.n;
  q.units = p.per_node ? n * p.hc : (n * a.heads + kR - 1) / kR;
  const int seen = max(0, q.L + n - a.window_len) >> p.ratio_log;  // by the deepest node there can be
  q.te = ((a.topk ? a.k : seen) + kT - 1) / kT;
  const int raw = p.per_node ? min(q.L + n, a.window_len) : min(q.L, a.window_len - 1) + n;
  q.tr = (raw + kT - 1) / kT;
  return q;
}

__device__ __forceinline__ int unit_cost(const Params& p, const SeqPlan& q) {
  return kCostSeg + q.te * (p.a.main.dtype == V4KV_FP8_E4M3 ? kCostFp8 : kCostTwo) + q.tr * kCostTwo;
}

__device__ __forceinline__ int tile_at_cost(const Params& p, const SeqPlan& q, int off) {
  const int cm = p.a.main.dtype == V4KV_FP8_E4M3 ? kCostFp8 : kCostTwo;
  off -= kCostSeg;
  if (off <= 0) return 0;
  if (off < q.te * cm) return off / cm;
  return min(q.te + (off - q.te * cm) / kCostTwo, q.te + q.tr - 1);
}

// A unit: its rows, and the items its tiles hold.
struct Unit {
  int g, tile;         // index, the walk's position in it
  int row0, nrows;     // rows of q and out
  int te, tr;          // tiles of entries, of raw rows
  int n_ent, n_all;    // entries in the list (top-k slots, or those that the deepest row sees); seen by every row
  int w0, n_win;       // first cached token in the list, and how many
  int n_tree;          // nodes in the list
  int node0, first;    // its first node, and the sequence's
  int L, b;
  int raw, raw_tree;   // the raw rows of the list's first token and of the sequence's first node
  int next;            // next unit's index, -1 behind the last
};

__device__ __forceinline__ void unit_load(const Params& p, Unit& x, int g) {
  const int4* r = p.w.units + (size_t)g * 4;
  const int4 a = r[0], b = r[1], c = r[2], d = r[3];
  x.g = g;
  x.tile = 0;
  x.row0 = a.x; x.nrows = a.y; x.te = a.z; x.tr = a.w;
  x.n_ent = b.x; x.n_all = b.y; x.w0 = b.z; x.n_win = b.w;
  x.n_tree = c.x; x.node0 = c.y; x.first = c.z; x.L = c.w;
  x.b = d.x; x.raw = d.y; x.raw_tree = d.z; x.next = d.w;
}

// to the next tile, of the next unit after a unit's last
__device__ __forceinline__ void tile_next(const Params& p, Unit& x) {
  if (++x.tile == x.te + x.tr && x.next >= 0) unit_load(p, x, x.next);
}

// prep: unit u of sequence b, from the depths of the sequence's nodes
__device__ __forceinline__ void unit_store(const Params& p, const SeqPlan& q, int b, int u, const int* depth, int next) {
  const TreeArgs& a = p.a;
  const int L = q.L, W = a.window_len;
  int node0, nrows, row0, lo, hi, n_tree;
  if (p.per_node) {
    node0 = u / p.hc;
    const int h0 = (u - node0 * p.hc) * kR;
    nrows = min(kR, a.heads - h0);
    row0 = (q.s.first + node0) * a.heads + h0;
    lo = hi = depth[node0];
    n_tree = lo + 1;
  } else {
    const int r0 = u * kR;
    nrows = min(kR, q.s.n * a.heads - r0);
    row0 = q.s.first * a.heads + r0;
    node0 = r0 / a.heads;
    const int last = (r0 + nrows - 1) / a.heads;
    lo = V4KV_MAX_TREE_NODES;
    hi = 0;
    for (int i = node0; i <= last; ++i) {
      lo = min(lo, depth[i]);
      hi = max(hi, depth[i]);
    }
    n_tree = last + 1;
  }
  const int w0 = min(L, max(0, L + lo + 1 - W)), base = (int)raw_row0(a, q, b) - raw_w0(a, q);
  int4* r = p.w.units + (size_t)unit_index(p, q, b, u) * 4;
  r[0] = make_int4(row0, nrows, q.te, q.tr);
  r[1] = a.topk ? make_int4(a.k, a.k, w0, L - w0)
                : make_int4(max(0, L + hi + 1 - W) >> p.ratio_log, max(0, L + lo + 1 - W) >> p.ratio_log, w0, L - w0);
  r[2] = make_int4(n_tree, q.s.first + node0, q.s.first, L);
  r[3] = make_int4(b, base + w0, base + L, next);
}

// A tile: whether its items are entries, the first one's index in its list,
// how many there are, and how many images its rows have.
struct Tile {
  bool entries;
  int first, count, images;
};

__device__ __forceinline__ Tile tile_of(const Params& p, const Unit& x) {
  Tile t;
  t.entries = x.tile < x.te;
  t.first = (t.entries ? x.tile : x.tile - x.te) * kT;
  t.count = min(kT, (t.entries ? x.n_ent : x.n_win + x.n_tree) - t.first);
  t.images = t.entries && p.a.main.dtype == V4KV_FP8_E4M3 ? 1 : 2;
  return t;
}

// entries that every node of a sequence sees
__device__ __forceinline__ int seen_by_all(const Params& p, int L) {
  return max(0, L + 1 - p.a.window_len) >> p.ratio_log;
}
__device__ __forceinline__ bool box_tile(const Params& p, const Unit& x, const Tile& t) {
  return p.boxes && t.entries && t.first + kT <= seen_by_all(p, x.L);
}

__device__ __forceinline__ void named_sync(int id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool named_or(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "bar.red.or.pred b, %2, 256, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}

using f2 = unsigned long long;  // two fp32 values
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Two e4m3 terms of a pair: x = hi + lo / 16. What is left of x is formed in half
// precision, which rounds x by 2^-11 beside lo's 2^-9 (a bf16 value and the difference
// are exact): fp32 takes twice the instructions, in the loop that bounds the sweep.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const uint16_t h = float2_to_e4m3x2(x, y);
  const __half2 r = __hmul2(__hsub2(__floats2half2_rn(x, y), e4m3x2_to_half2(h)), __float2half2_rn(16.f));
  hi = h;
  __half2_raw rr = *reinterpret_cast<const __half2_raw*>(&r);
  lo = __nv_cvt_halfraw2_to_fp8x2(rr, __NV_SATFINITE, __NV_E4M3);
}

// the terms of 16 consecutive values times m
__device__ __forceinline__ void split16(const float* v, float m, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h0, h1, l0, l1;
    split2(v[4 * i] * m, v[4 * i + 1] * m, h0, l0);
    split2(v[4 * i + 2] * m, v[4 * i + 3] * m, h1, l1);
    h[i] = h0 | (h1 << 16);
    l[i] = l0 | (l1 << 16);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

__device__ __forceinline__ void bf16x16(const uint4* p, float* v) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4 r = p[k];
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[8 * k + 2 * i] = __uint_as_float(w[i] << 16);
      v[8 * k + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// The power of two that takes a row's largest magnitude (its fp32 bits) into
// [2^7, 2^8), and its inverse. Rows below 2^-118 keep 2^-126 as their unit.
__device__ __forceinline__ float scale_up(uint32_t amax) {
  return __uint_as_float((261u - max(amax >> 23, 8u)) << 23);
}
__device__ __forceinline__ float scale_down(uint32_t amax) {
  return __uint_as_float((max(amax >> 23, 8u) - 7u) << 23);
}

// block scaled fp8 MMA: D (+)= (A sfa) (B sfb), scales per row and 32 elements of K
constexpr uint32_t idesc_mx(int N, int mn, int sfb_byte) {
  return ((uint32_t)sfb_byte << 4) | ((uint32_t)mn << 15) | ((uint32_t)mn << 16) |
         ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27);
}
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(x), "r"(y),
               "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(x) : "memory");
}

// 16 lanes x 16 columns: thread t gets, for k = 0, 1, r[4k + 0/1] = (lane t/4,
// columns 8k + 2(t%4) + 0/1) and r[4k + 2/3] = (lane t/4 + 8, the same columns)
__device__ __forceinline__ void tmem_ld16x256_x2(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}

// ------------------------------------------------------------------ loading

// what the softmax needs of an item: its scale, and for the weight of its raw
// codes log2 |scale| and 1 / |scale|. A scale that is not finite stands for NaN, a zero
// scale for zero codes: the item has no value but counts in the normaliser, which is
// summed as 2^(score + log2 |scale|) / |scale|. So is one taken whose scale is below
// 2^kLowest, or 2^-kApart of the largest in its block of 32 items. Otherwise that sum could
// leave fp32: a weight may reach 2^(kRaise + 8 - log2 |scale|) of the reference, and a sum may
// hold 2^21 of them; and a weight of 2^-45 of the block's largest or more would lose its
// power beside a scale that is larger still. P carries 2^-21 of a block's largest weight
// times scale, so that such a value is far below its bits.
// Any log2 does for an item without a value, and it gets one below those of its block
// (`top` is the largest of them, kNoTop if there is none): near them, so that neither
// drives the other's power out of fp32, and 40 lower, so that they keep their bits in P
// beside a row of zeros of up to 2^50 times their weight, but not below kLowest.
constexpr float kNoTop = 0.f, kBelow = 40.f, kLowest = -76.f, kApart = 60.f;
__device__ __forceinline__ float4 item_meta(float scale, bool there, float top) {
  if (!there) return make_float4(0.f, 0.f, 0.f, -INFINITY);
  if (!isfinite(scale)) return make_float4(__int_as_float(0x7fffffff), 0.f, 1.f, 0.f);
  const float m = fabsf(scale), l2 = log2f(m);
  if (l2 >= fmaxf(top - kApart, kLowest)) return make_float4(scale, l2, 1.f / m, 0.f);
  const float lg = fmaxf(top - kBelow, kLowest);
  return make_float4(0.f, lg, exp2f(-lg), 0.f);
}

// floor(log2 |scale|) of an item with a value
__device__ __forceinline__ int scale_exponent(float scale, bool there) {
  const int e = (int)(__float_as_uint(scale) >> 23 & 0xff);  // 0: zero or subnormal, 255: not finite
  return there && e >= 127 + (int)kLowest && e < 255 ? e - 127 : -128;
}
__device__ __forceinline__ float block_top(int e) { return e > -128 ? (float)e : kNoTop; }

// An fp8 row of zeros has codes 0 and, as the compressor writes it, the scale 1: beside rows
// of ordinary scales (2^-9) its weight would take their bits in P. So of a row whose
// scale is 2^kWide or more above its block's smallest (`low`) the codes are looked at: a
// row of zeros gets the scale 0. Nearly always 16 bytes settle it.
constexpr int kWide = 4;
__device__ __forceinline__ float scale_of_codes(float scale, unsigned long long row, int low) {
  if (scale_exponent(scale, row != 0) < low + kWide) return scale;
  const uint4* c = reinterpret_cast<const uint4*>(row);
#pragma unroll 1
  for (int k = 0; k < kD / 16; ++k) {
    const uint4 v = c[k];
    if ((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) return scale;
  }
  return 0.f;
}
// (127: no item has a value)
__device__ __forceinline__ int low_exponent(int e) { return e > -128 ? e : 127; }

// Whether all of a tile's items have values, with scales within 2^kWide: then no item
// stands out, and no block's largest is asked for (kAnyTop does). A lane gives four.
constexpr float kAnyTop = -128.f;
__device__ __forceinline__ bool alike(const float* s, bool a, bool b, bool c, bool d) {
  const bool there[4] = {a, b, c, d};
  int low = 127, high = -128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = scale_exponent(s[i], true);
    if (there[i]) {
      low = min(low, e);
      high = max(high, e);
    }
  }
  low = __reduce_min_sync(0xffffffffu, low);
  return low > -128 && __reduce_max_sync(0xffffffffu, high) < low + kWide;
}

// Lane l resolves items l, l + 32, l + 64, l + 96 of a tile: their rows'
// addresses (0: no such item) and scales. The loads go in phases (top-k entry,
// block table, scale), the four of a phase independent of one another.
__device__ __forceinline__ void resolve_tile(const Params& p, const Unit& x, const Tile& t, int lane,
                                             unsigned long long* rows, float4* meta) {
  const TreeArgs& a = p.a;
  if (!t.entries) {
    const uint4 m4 = p.w.anc[x.node0];
#pragma unroll 1
    for (int r = 0; r < 4; ++r) {
      const int k = lane + 32 * r;
      int n = t.first + k;
      unsigned long long at = 0;
      float2 mt = make_float2(0.f, -INFINITY);
      if (k < t.count) {
        if (n < x.n_win) {
          n += x.raw;
        } else {
          n -= x.n_win;
          if (p.per_node) {  // the n-th of the node's ancestors
            uint32_t m = m4.x;
            int up = 0;
            if (n >= __popc(m)) { n -= __popc(m); m = m4.y; up = 32; }
            if (up == 32 && n >= __popc(m)) { n -= __popc(m); m = m4.z; up = 64; }
            if (up == 64 && n >= __popc(m)) { n -= __popc(m); m = m4.w; up = 96; }
            for (; n > 0; --n) m &= m - 1;
            n = up + __ffs(m) - 1;
          }
          n += x.raw_tree;
        }
        mt = p.w.raw_meta[n];
        // a row whose page is missing has not been written: zeros are taken for it
        if (mt.y == 0.f) at = reinterpret_cast<unsigned long long>(p.w.raw) + (size_t)n * (2 * kD);
      }
      rows[k] = at;
      const bool there = mt.y == 0.f;
      meta[k] = item_meta(mt.x, there, block_top(__reduce_max_sync(0xffffffffu, scale_exponent(mt.x, there))));
    }
    return;
  }
  const PoolArgs& pool = a.main;
  const int32_t* bt = pool.block_table + (size_t)x.b * pool.max_blocks;
  if (box_tile(p, x, t)) {
    if (p.staged) {
      const size_t row = (size_t)x.b * p.staged + t.first;
      if (lane < 2) rows[64 * lane] = reinterpret_cast<unsigned long long>(p.w.ent) + (row + 64 * lane) * p.box_bytes;
      float scale[4], top[4] = {kAnyTop, kAnyTop, kAnyTop, kAnyTop};
      bool there[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float2 mt = p.w.ent_meta[row + lane + 32 * r];
        scale[r] = mt.x;
        there[r] = mt.y == 0.f;
      }
      if (!alike(scale, there[0], there[1], there[2], there[3])) {
#pragma unroll
        for (int r = 0; r < 4; ++r) top[r] = block_top(__reduce_max_sync(0xffffffffu, scale_exponent(scale[r], there[r])));
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) meta[lane + 32 * r] = item_meta(scale[r], there[r], top[r]);
      return;
    }
    // two whole pages: only their first rows' addresses are asked for
    const int j = t.first + 64 * (lane >> 4);  // lanes 0 .. 15: the first page's items, 4 each
    const int blk = j >> 6, pg = blk < pool.max_blocks ? bt[blk] : -1;
    const bool there = pg >= 0 && pg < pool.num_pages;
    if (!there && (lane & 15) == 0)
      flag(a.dev_status, blk < pool.max_blocks ? V4KV_DEV_BAD_PAGE : V4KV_DEV_BAD_SLOT);
    const size_t slot = (size_t)(there ? pg : 0) * 64;
    if ((lane & 15) == 0)
      rows[64 * (lane >> 4)] = there ? reinterpret_cast<unsigned long long>(pool.data) + slot * kD : 0;
    const float4 s4 = *reinterpret_cast<const float4*>(pool.scales + slot + 4 * (lane & 15));
    float scale[4] = {s4.x, s4.y, s4.z, s4.w}, top = kAnyTop;
    if (!alike(scale, there, there, there, there)) {
      int low = 127, e = -128;
#pragma unroll
      for (int i = 0; i < 4; ++i) low = min(low, low_exponent(scale_exponent(scale[i], there)));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (there) scale[i] = scale_of_codes(scale[i], reinterpret_cast<unsigned long long>(pool.data) + (slot + 4 * (lane & 15) + i) * kD, low);
        e = max(e, scale_exponent(scale[i], there));
      }
      __syncwarp();
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) e = max(e, __shfl_xor_sync(0xffffffffu, e, o));
      top = block_top(e);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) meta[4 * lane + i] = item_meta(scale[i], there, top);
    return;
  }
  int j[4], pg[4], err = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int k = lane + 32 * r;
    j[r] = k < t.count ? t.first + k : -1;
    if (a.topk && j[r] >= 0) j[r] = a.topk[(size_t)x.node0 * a.k + j[r]];
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    pg[r] = -1;
    if (j[r] < 0) continue;
    if (a.topk && j[r] >= (x.L + a.ratio - 1) >> p.ratio_log) {
      err |= V4KV_DEV_BAD_INDEX;
      j[r] = -1;
    } else if (j[r] >> p.spb_log >= pool.max_blocks) {
      err |= V4KV_DEV_BAD_SLOT;
      j[r] = -1;
    } else {
      pg[r] = bt[j[r] >> p.spb_log];
    }
  }
  const bool fp8 = pool.dtype == V4KV_FP8_E4M3;
  float scale[4];
  unsigned long long at[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    scale[r] = 1.f;
    at[r] = 0;
    if (j[r] < 0) continue;
    if (pg[r] < 0 || pg[r] >= pool.num_pages) {
      err |= V4KV_DEV_BAD_PAGE;
    } else {
      const size_t slot = ((size_t)pg[r] << p.spb_log) + (j[r] & (pool.spb - 1));
      if (fp8) scale[r] = pool.scales[slot];
      at[r] = reinterpret_cast<unsigned long long>(pool.data) + slot * (fp8 ? kD : 2 * kD);
    }
  }
  float top[4] = {kAnyTop, kAnyTop, kAnyTop, kAnyTop};
  if (!alike(scale, at[0] != 0, at[1] != 0, at[2] != 0, at[3] != 0)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool there = at[r] != 0;
      if (fp8) {
        scale[r] = scale_of_codes(scale[r], at[r], __reduce_min_sync(0xffffffffu, low_exponent(scale_exponent(scale[r], there))));
        __syncwarp();
      }
      top[r] = block_top(__reduce_max_sync(0xffffffffu, scale_exponent(scale[r], there)));
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    rows[lane + 32 * r] = at[r];
    meta[lane + 32 * r] = item_meta(scale[r], at[r] != 0, top[r]);
  }
  if (err) flag(a.dev_status, err);
}

// Codes that some rows of the unit must not see may not be NaN (0 * NaN): such
// a row is taken as zeros with a NaN scale, which reaches the rows that see it.
__device__ __forceinline__ bool has_nan_code(uint4 c) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
  return bad;
}

// largest magnitude of 16 bf16 values per lane over a warp, as fp32 bits
__device__ __forceinline__ uint32_t amax_bf16(const uint4* r) {
  const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
  return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16)) << 16;
}

// a lane's 16 dims of a bf16 row as two terms; the row's scale (0 for a row of
// zeros; NaN, and zero terms, for a row that is not finite)
__device__ __forceinline__ float split_row(const uint4* raw, uint4& hi, uint4& lo) {
  const uint32_t m = amax_bf16(raw);
  if (m >= 0x7f800000u) {
    hi = lo = make_uint4(0, 0, 0, 0);
    return __int_as_float(0x7fffffff);
  }
  float v[16];
  bf16x16(raw, v);
  split16(v, scale_up(m), hi, lo);
  return m == 0 ? 0.f : scale_down(m);
}

// Eight rows from r0 on whose 32 bytes of bf16 a lane were copied to where the
// lane's two terms go: split in place, and their scales put down.
__device__ __noinline__ void split_rows(const unsigned long long* rows, int r0, int lane, uint8_t* hi_dst,
                                        uint8_t* lo_dst, float4* meta) {
#pragma unroll 2
  for (int r = r0; r < r0 + 8; ++r) {
    const uint32_t off = (lane >> 3) * kChunk + tc::sw128_off(r, lane & 7);
    uint4 raw[2], hi, lo;
    raw[0] = *reinterpret_cast<uint4*>(hi_dst + off);
    raw[1] = *reinterpret_cast<uint4*>(lo_dst + off);
    const float scale = split_row(raw, hi, lo);
    if (rows[r] && lane == 0) meta[r].x = scale;
    *reinterpret_cast<uint4*>(hi_dst + off) = hi;
    *reinterpret_cast<uint4*>(lo_dst + off) = lo;
  }
}

// ------------------------------------------------------------------ the sweep

// O^T's columns of a warp's 16 rows times the rows' factors
__device__ __noinline__ void scale_rows(uint32_t o, const float* fac) {
#pragma unroll 1
  for (int g = 0; g < 8; ++g) {
    const uint32_t at = o + kR * (g >> 1) + 8 * (g & 1);
    uint32_t r8[8];
    tmem_ld8(at, r8);
    tc::tmem_wait_ld();
#pragma unroll
    for (int n = 0; n < 8; ++n) r8[n] = __float_as_uint(__uint_as_float(r8[n]) * fac[8 * (g & 1) + n]);
    tmem_st8(at, r8);
  }
}

__device__ __noinline__ uint32_t rows_seeing(uint32_t seen, const Unit& x, bool entries, int r0, int row,
                                             const int4* vis, const uint4* anc) {
#pragma unroll 1
  for (int j = 0; j < 4; ++j) {
    const int r = r0 + 8 * j;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      bool v;
      if (entries) {
        v = r < vis[row + m].x;
      } else if (r < x.n_win) {
        v = x.w0 + r >= vis[row + m].y;
      } else {
        const int k = min(r - x.n_win, V4KV_MAX_TREE_NODES - 1);
        v = (reinterpret_cast<const uint32_t*>(anc + m)[k >> 5] >> (k & 31)) & 1;
      }
      if (!v) seen &= ~(1u << (4 * j + m));
    }
  }
  return seen;
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1) tree_attend_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = tc::smem_u32(smem_raw);
  const uint32_t pad = ((raw_addr + 1023u) & ~1023u) - raw_addr;
  uint8_t* sm = smem_raw + pad;
  const uint32_t sbase = raw_addr + pad;
  Bars* bars = reinterpret_cast<Bars*>(sm + kBarOff);
  float4* meta = reinterpret_cast<float4*>(sm + kMetaOff);
  float* row_ref = reinterpret_cast<float*>(sm + kRowOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kMiscOff + 4);
  const TreeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < 8; ++s) tc::mbar_init(&bars->kv_full[s >> 2][s & 3], 4);
    for (int s = 0; s < 4; ++s) tc::mbar_init(&bars->kv_empty[s >> 1][s & 1], 1);
    for (int s = 0; s < kRing; ++s) {
      tc::mbar_init(&bars->addr_full[s], 32);
      tc::mbar_init(&bars->addr_free[s], 1);
    }
    tc::mbar_init(&bars->raw_full, 4);
    tc::mbar_init(&bars->ready, 4);
    tc::mbar_init(&bars->q_full, 1);
    tc::mbar_init(&bars->q_empty, 1);
    tc::mbar_init(&bars->s_full, 1);
    tc::mbar_init(&bars->s_free, 16);
    tc::mbar_init(&bars->p_full, 16);
    tc::mbar_init(&bars->pv_done, 1);
    tc::mbar_init(&bars->drain, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 20) tc::tmem_alloc(tmem_slot, kCols);
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  // what the prep kernel stored is read by bulk copies
  asm volatile("fence.proxy.async.global;" ::: "memory");
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int4 rec = p.w.rec[blockIdx.x];
  const int n_tiles = p.w.rec[blockIdx.x + 1].x - rec.x;
  if (n_tiles <= 0) {
    if (warp == 20) tc::tmem_free(tmem, kCols);
    return;
  }
  Unit x;
  unit_load(p, x, rec.y);
  x.tile = rec.w;

  if (warp == 23) {
    // ======================= the units' Q, as their last one's products are done
    bool ok = true;
    uint32_t seg = 0;
    for (int i = 0; i < n_tiles && ok; ++seg) {
      if (seg > 0) ok = tc::mbar_wait(&bars->q_empty, (seg - 1) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(&bars->q_full, 65536);
        const uint8_t* src = p.w.q + (size_t)x.g * 65536;
        for (int k = 0; k < 4; ++k)
          tc::bulk_load(sbase + kQOff + k * 16384, src + k * 16384, 16384, &bars->q_full);
      }
      i += x.te + x.tr - x.tile;
      if (i < n_tiles) unit_load(p, x, x.next);
    }
    if (!ok) {
      *abort_flag = 1;
      flag(a.dev_status, V4KV_DEV_TIMEOUT);
    }
    // the last copy has landed before the block's shared memory is released
    volatile int never = 0;
    if (seg > 0 && !tc::mbar_wait(&bars->q_full, (seg - 1) & 1, &never)) flag(a.dev_status, V4KV_DEV_TIMEOUT);
  } else if (warp >= 21) {
    // ======================= row addresses and scales, up to kRing tiles ahead.
    // Tile number `done` of the block (tiles without items do not count) is in
    // slot done % kRing.
    uint32_t done = 0;
    bool ok = true;
    for (int i = 0; i < n_tiles && ok; ++i) {
      const Tile t = tile_of(p, x);
      if (t.count > 0) {
        if ((done & 1) == (uint32_t)(warp - 21)) {
          const uint32_t s = done % kRing;
          if (done >= kRing) ok = tc::mbar_wait(&bars->addr_free[s], ((done - kRing) / kRing) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          resolve_tile(p, x, t, lane, reinterpret_cast<unsigned long long*>(sm + kPtrOff) + s * kT, meta + s * kT);
          tc::mbar_arrive(&bars->addr_full[s]);
        }
        ++done;
      }
      tile_next(p, x);
    }
    if (!ok) {
      *abort_flag = 1;
      flag(a.dev_status, V4KV_DEV_TIMEOUT);
    }
  } else if (warp >= 16 && warp < 20) {
    // ======================= tiles into the stages. `im` counts images: image
    // im lives in stage im % 2.
    const int w = warp - 16;
    bool ok = true;
    uint32_t im = 0, done = 0;
    // image m's place is free (the first 256 dims of it, then the others)
    auto wait_empty = [&](uint32_t m, int c) {
      return m < 2 || tc::mbar_wait(&bars->kv_empty[m & 1][c], ((m - 2) >> 1) & 1, abort_flag);
    };
    for (int i = 0; i < n_tiles && ok; ++i) {
      const Tile t = tile_of(p, x);
      if (t.count > 0) {
        const uint32_t s = im & 1, slot = done % kRing;
        const unsigned long long* rows = reinterpret_cast<const unsigned long long*>(sm + kPtrOff) + slot * kT;
        ok = tc::mbar_wait(&bars->addr_full[slot], (done / kRing) & 1, abort_flag);
        if (box_tile(p, x, t)) {
          // 2 x 64 rows in order, every one visible: two boxes per 128 dims,
          // as the last tile's product leaves them. All four warps wait and
          // arrive, so that none falls a phase behind.
          int y[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            // a page that is missing is read behind the pool's end: zeros
            y[k] = rows[64 * k] ? (int)((rows[64 * k] - reinterpret_cast<unsigned long long>(p.box_data)) / p.box_bytes)
                                : p.box_rows;
#pragma unroll 1
          for (int n = 0; n < 4 * t.images; ++n) {  // 128 bytes of the rows
            const int c = n & 3;
            const uint32_t m = im + (n >> 2), at = m & 1;
            if ((c & 1) == 0) ok = __all_sync(0xffffffffu, ok && wait_empty(m, c >> 1));
            if (!ok) break;
            if (lane == 0) {
              if (w > 0) {
                tc::mbar_arrive(&bars->kv_full[at][c]);
              } else {
                tc::mbar_arrive_expect_tx(&bars->kv_full[at][c], kChunk);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  tc::tma_load_2d(sbase + kVOff + at * kStage + c * kChunk + k * (kChunk / 2), &p.map, 128 * n, y[k],
                                  &bars->kv_full[at][c]);
              }
            }
          }
          if (!ok) break;
        } else {
          for (int k = 0; k < t.images; ++k)
            for (int c = 0; c < 2; ++c) ok = ok && wait_empty(im + k, c);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          float4* mt = meta + slot * kT;
          uint8_t* dst = sm + kVOff + s * kStage;
          const uint32_t d0 = sbase + kVOff + s * kStage, d1 = sbase + kVOff + (s ^ 1) * kStage;
          if (t.images == 1) {
            // rows from `safe` on are hidden from some of the unit's rows
            const int safe = max(0, min(32, x.n_all - t.first - 32 * w));
            if (safe == 32) {  // no branch per row: 71 -> 67 us with 512 chosen entries a node
              const unsigned long long mine = rows[32 * w + lane], none = reinterpret_cast<unsigned long long>(a.main.data);
              const uint32_t d2 = d0 + (lane >> 3) * kChunk + 4096 * w;
#pragma unroll 8
              for (int r = 0; r < 32; ++r) {
                const unsigned long long src = __shfl_sync(0xffffffffu, mine, r);
                cp_async16(d2 + tc::sw128_off(r, lane & 7), reinterpret_cast<const uint8_t*>(src ? src : none) + 16 * lane,
                           src != 0);
              }
            } else {
#pragma unroll 4
              for (int r = 0; r < 32; ++r) {
                const uint8_t* src = reinterpret_cast<const uint8_t*>(rows[32 * w + r]);
                if (r < safe || !src)
                  cp_async16(d0 + (lane >> 3) * kChunk + tc::sw128_off(32 * w + r, lane & 7),
                             src ? src + 16 * lane : static_cast<const uint8_t*>(a.main.data), src != nullptr);
              }
            }
            for (int r = safe; r < 32; ++r) {
              const uint4* src = reinterpret_cast<const uint4*>(rows[32 * w + r]);
              if (!src) continue;
              uint4 v = src[lane];
              if (__any_sync(0xffffffffu, has_nan_code(v))) {
                v = make_uint4(0, 0, 0, 0);
                if (lane == 0) mt[32 * w + r] = item_meta(__int_as_float(0x7fffffff), true, kNoTop);
              }
              *reinterpret_cast<uint4*>(dst + (lane >> 3) * kChunk + tc::sw128_off(32 * w + r, lane & 7)) = v;
            }
          } else {
            // raw rows: their two terms. bf16 entries: the lane's 32 bytes.
            const uint32_t step = t.entries ? 32 : 16, second = t.entries ? 16 : kD;
#pragma unroll 8
            for (int r = 0; r < 32; ++r) {
              const uint8_t* src = reinterpret_cast<const uint8_t*>(rows[32 * w + r]);
              const uint32_t off = (lane >> 3) * kChunk + tc::sw128_off(32 * w + r, lane & 7);
              const uint8_t* from = src ? src + step * lane : p.w.raw;
              cp_async16(d0 + off, from, src != nullptr);
              cp_async16(d1 + off, src ? from + second : from, src != nullptr);
            }
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (t.images == 2 && t.entries) {  // the softmax warps, idle now, split them
            if (lane == 0) tc::mbar_arrive(&bars->raw_full);
          } else if (lane < 4) {
            for (int k = 0; k < t.images; ++k) tc::mbar_arrive(&bars->kv_full[(im + k) & 1][lane]);
          }
        }
        im += t.images;
        ++done;
      }
      tile_next(p, x);
    }
    if (!ok) {
      *abort_flag = 1;
      flag(a.dev_status, V4KV_DEV_TIMEOUT);
    }
  } else if (warp == 20) {
    // ======================= MMA issue: the whole warp runs the loop, one lane
    // elected once issues
    const bool leader = tc::elect_one();
    const uint64_t v_k = tc::sw128_desc(sbase + kVOff, 16, 1024), v_m = tc::sw128_desc(sbase + kVOff, 1024, 1024);
    const uint64_t q_k = tc::sw128_desc(sbase + kQOff, 16, 1024);
    const uint64_t p_h = tc::sw128_desc(sbase + kPOff, 1024, 1024), p_l = tc::sw128_desc(sbase + kPOff + 64, 1024, 1024);
    bool ok = true;
    uint32_t im = 0;  // images before the current tile
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(bar, parity, abort_flag));
    };
    auto poll = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, tc::mbar_poll(bar, parity)); };
    auto poll_kv = [&](uint32_t m) {
      bool all = true;
#pragma unroll
      for (int c = 0; c < 4; ++c) all = all && tc::mbar_poll(&bars->kv_full[m & 1][c], (m >> 1) & 1);
      return __all_sync(0xffffffffu, all);
    };
    // S^T of a tile whose images begin at `m`, 128 dims at a time as they land
    auto issue_s = [&](uint32_t m, int images) {
      for (int k = 0; k < images && ok; ++k) {
        const uint32_t s = (m + k) & 1;
        const uint64_t vk = v_k + (uint64_t)(s * (kStage >> 4));
        const uint32_t sfa = tmem + (k ? kLow : kOne);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          wait_all(&bars->kv_full[s][c], ((m + k) >> 1) & 1);
          if (!ok) break;
          tc::tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_mx(tmem + kSCol, vk + (uint64_t)((c * kChunk + kk * 32) >> 4),
                     q_k + (uint64_t)((c * kChunk + kk * 32) >> 4), idesc_mx(128, 0, 0), sfa, tmem + kSfQ,
                     (k | c | kk) ? 1u : 0u);
          }
          __syncwarp();
        }
      }
      if (ok && leader) tc::mma_commit(&bars->s_full);
      __syncwarp();
    };
    // the first tile with items from the walk's position on; `i` its index
    // among the block's tiles, segments that end without one get their commit
    int i = 0;
    uint32_t done = 0, seg = 0;
    bool opened = false;      // the segment's Q has been waited for
    bool s_issued = false;    // the current tile's S has been issued
    uint32_t filled = 0;      // O^T holds something of this segment
    Tile t = tile_of(p, x);
    wait_all(&bars->ready, 0);  // the constant block scales are in tensor memory
    tc::tc_fence_after();
    while (i < n_tiles && ok) {
      const bool seg_last = x.tile + 1 == x.te + x.tr || i + 1 == n_tiles;
      if (!opened) {
        wait_all(&bars->q_full, seg & 1);
        if (!ok) break;
        opened = true;
        filled = 0;
      }
      if (t.count > 0 && !s_issued) issue_s(im, t.images);
      if (seg_last && leader) tc::mma_commit(&bars->q_empty);
      __syncwarp();
      // the next tile, while the softmax works on this one
      tile_next(p, x);
      const Tile nt = i + 1 < n_tiles ? tile_of(p, x) : Tile{false, 0, 0, 0};
      s_issued = false;
      if (t.count > 0 && ok) {
        // Whichever is ready first: this tile's P, or the next tile with S free
        // in tensor memory (the softmax has read this one's).
        bool ahead = !seg_last && nt.count > 0 && t.images == 1 && nt.images == 1;
        const long long t0 = clock64();
        while (true) {
          if (ahead && poll(&bars->s_free, done & 1) && poll_kv(im + 1)) {
            tc::tc_fence_after();
            issue_s(im + 1, 1);
            s_issued = true;
            ahead = false;
            if (!ok) break;
          }
          if (ahead ? poll(&bars->p_full, done & 1)
                    : __all_sync(0xffffffffu, tc::mbar_wait(&bars->p_full, done & 1, abort_flag)))
            break;
          if (!ahead || *abort_flag || clock64() - t0 > tc::kWaitCycles) ok = false;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        if (!ok) break;
        tc::tc_fence_after();
        if (leader) {
          const int nk = (t.count + 31) >> 5;
          for (int k = 0; k < t.images; ++k) {
            const uint32_t s = (im + k) & 1;
            const uint64_t vm = v_m + (uint64_t)(s * (kStage >> 4));
            const uint32_t sfa = tmem + (k ? kLow : kOne);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (kk < nk) {
                  mma_mx(tmem + kOCol + kR * c, vm + (uint64_t)((c * kChunk + kk * 4096) >> 4),
                         p_h + (uint64_t)((kk * 4096) >> 4), idesc_mx(64, 1, kk), sfa, tmem + kSfHi,
                         (filled | k | kk) ? 1u : 0u);
                  mma_mx(tmem + kOCol + kR * c, vm + (uint64_t)((c * kChunk + kk * 4096) >> 4),
                         p_l + (uint64_t)((kk * 4096) >> 4), idesc_mx(64, 1, kk), sfa, tmem + kSfLo, 1u);
                }
              if (c & 1) tc::mma_commit(&bars->kv_empty[s][c >> 1]);
            }
          }
          tc::mma_commit(&bars->addr_free[done % kRing]);
        }
        __syncwarp();
        filled = 1;
        im += t.images;
        ++done;
      }
      if (seg_last) {
        if (leader) tc::mma_commit(&bars->pv_done);
        __syncwarp();
        ++seg;
        opened = false;
      }
      t = nt;
      ++i;
    }
    if (!ok && leader) {
      *abort_flag = 1;
      flag(a.dev_status, V4KV_DEV_TIMEOUT);
    }
    // every MMA has completed before tensor memory is freed
    if (leader) tc::mma_commit(&bars->drain);
    __syncwarp();
    volatile int never = 0;
    if (!tc::mbar_wait(&bars->drain, 0, &never) && leader) flag(a.dev_status, V4KV_DEV_TIMEOUT);
    __syncwarp();
  } else {
    // ======================= softmax: warp w of quarter qd has items 32 w .. 32 w
    // + 31 and rows 16 qd .. 16 qd + 15; a thread items 32 w + lane / 4 + 8 j
    // (j < 4) and rows 16 qd + 4 c + m (c = lane % 4, m < 4). That is how the
    // 16x256b tensor-memory load deals out S when row 4 c + 2 k + e of a quarter
    // sits in Q's row 8 k + 2 c + e: a row's maximum over the items takes three
    // shuffles and the thread's part of P is four consecutive bytes of a row.
    // The two quarters of a half meet at a barrier per tile.
    const int qd = warp >> 2, w = warp & 3, c4 = lane & 3, hh = qd >> 1;
    const int bar = 1 + hh;
    const int row_t = 16 * qd + 4 * c4;        // the thread's first row
    const int row_h = row_t & 31;              // in its half
    const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
    float* red = reinterpret_cast<float*>(sm + kRedOff) + 128 * hh;       // [4][32]
    float* fac = reinterpret_cast<float*>(sm + kFacOff);                  // [64]
    uint8_t* sf = sm + kSfOff + 128 * hh;                                  // [32][4]
    volatile int* raise = reinterpret_cast<volatile int*>(sm + kMiscOff + 16) + 2 * hh;
    const uint4* anc = reinterpret_cast<const uint4*>(sm + kAncOff) + row_t;
    const int4* vis = reinterpret_cast<const int4*>(sm + kVisOff);
    if (qd == 0) {
      const uint32_t one = 0x7f7f7f7fu, low = 0x7b7b7b7bu;
      tmem_st4(lanes + kOne, one, one, one, one);
      tmem_st4(lanes + kLow, low, low, low, low);
      tmem_st4(lanes + kSfQ, one, one, low, low);
      tmem_st4(lanes + kSfHi, one, one, one, one);
      tmem_st4(lanes + kSfLo, one, one, one, one);
      tc::tmem_wait_st();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->ready);
    }
    if (w == 0 && lane < 2 && !(qd & 1)) raise[lane] = 0;
    bool ok = true, seg_open = true, any = false;
    int seg_tile0 = 0;
    uint32_t im = 0, done = 0, seg = 0, split = 0;
    float l[4], fa[4], ref[4];
    for (int i = 0; i < n_tiles; ++i) {
      if (seg_open) {
        // the rows' factors, references and masks
        seg_open = false;
        any = false;
        seg_tile0 = x.tile;
        const float4 f = *reinterpret_cast<const float4*>(p.w.q_factor + (size_t)x.g * kR + row_t);
        fa[0] = f.x; fa[1] = f.y; fa[2] = f.z; fa[3] = f.w;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          l[m] = 0.f;
          ref[m] = kNone;
        }
        if (w == 0 && lane < 16) {
          const int n = 16 * qd + lane;
          int node = x.node0;  // per_node: the only one
          if (!p.per_node && n < x.nrows) node = (x.row0 + n) / a.heads;
          const int w0 = max(0, x.L + p.w.depth[node] + 1 - a.window_len);
          reinterpret_cast<uint4*>(sm + kAncOff)[n] = p.w.anc[node];
          reinterpret_cast<int4*>(sm + kVisOff)[n] = make_int4(w0 >> p.ratio_log, w0, node, 0);
          row_ref[n] = kNone;
        }
        named_sync(bar);
      }
      const Tile t = tile_of(p, x);
      const bool seg_last = x.tile + 1 == x.te + x.tr || i + 1 == n_tiles;
      if (t.count > 0) {
        if (t.images == 2 && t.entries && !box_tile(p, x, t)) {
          // bf16 entries: eight rows a warp
          ok = tc::mbar_wait(&bars->raw_full, split & 1, abort_flag);
          if (named_or(bar, !ok)) {
            ok = false;
            break;
          }
          ++split;
          const uint32_t slot = done % kRing, s = im & 1;
          split_rows(reinterpret_cast<const unsigned long long*>(sm + kPtrOff) + slot * kT, 8 * warp, lane,
                     sm + kVOff + s * kStage, sm + kVOff + (s ^ 1) * kStage, meta + slot * kT);
          tc::fence_proxy_async_smem();
          named_sync(bar);
          if (w == 0) {  // the block's 32 rows have been split
            float4* mt = meta + slot * kT + 32 * qd + lane;
            const float scale = mt->x;
            const bool there = mt->w == 0.f;
            *mt = item_meta(scale, there, block_top(__reduce_max_sync(0xffffffffu, scale_exponent(scale, there))));
            __syncwarp();
            if (lane < 8) tc::mbar_arrive(&bars->kv_full[lane >> 2][lane & 3]);
          }
        }
        ok = tc::mbar_wait(&bars->s_full, done & 1, abort_flag);
        tc::tc_fence_after();
        // the items' {scale, log2 |scale|, 1 / |scale|} and the scores u[j][m],
        // log2 of a weight of the item's codes
        float u[4][4], inv[4];
        uint32_t seen = 0;  // bit 4 j + m: row m sees item j
        bool plain = true;  // all scales positive
        const float4* mts = meta + (done % kRing) * kT + 32 * w + (lane >> 2);
        {
          uint32_t h[2][8], q[2][8];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            tmem_ld16x256_x2(lanes + ((uint32_t)(16 * k) << 16) + kSCol + 16 * qd, h[k]);
            tmem_ld16x256_x2(lanes + ((uint32_t)(16 * k) << 16) + kSCol + kR + 16 * qd, q[k]);
          }
          float ks[4], lg[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 mt = mts[8 * j];
            ks[j] = mt.x;
            lg[j] = mt.y;
            inv[j] = mt.z;
            seen |= (mt.w == 0.f ? 0xfu : 0u) << (4 * j);
            plain &= mt.x > 0.f;
          }
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int m = 0; m < 4; m += 2) {
              const int r = 4 * (m >> 1) + 2 * (j & 1);
              const f2 sum = add2(pack2(__uint_as_float(h[j >> 1][r]), __uint_as_float(h[j >> 1][r + 1])),
                                  pack2(__uint_as_float(q[j >> 1][r]), __uint_as_float(q[j >> 1][r + 1])));
              unpack2(fma2(mul2(sum, pack2(ks[j], ks[j])), pack2(fa[m], fa[m + 1]), pack2(lg[j], lg[j])), u[j][m],
                      u[j][m + 1]);
            }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->s_free);
        if (!p.per_node && (!t.entries || t.first + kT > x.n_all)) {
          const Unit y = x;
          seen = rows_seeing(seen, y, t.entries, t.first + 32 * w + (lane >> 2), row_t, vis, anc);
        }
        if (seen != 0xffffu) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int m = 0; m < 4; ++m)
              if (!(seen >> (4 * j + m) & 1)) u[j][m] = -INFINITY;
        }
        // Per row, the exponent ex that puts the warp's 32 weights below 2^8,
        // the largest in [2^7, 2^8): a weight is 2^ex times what is stored.
        float ex[4], lt[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) ex[m] = fmaxf(fmaxf(u[0][m], u[1][m]), fmaxf(u[2][m], u[3][m]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
#pragma unroll
          for (int m = 0; m < 4; ++m) ex[m] = fmaxf(ex[m], __shfl_xor_sync(0xffffffffu, ex[m], o));
        bool high = false;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          ex[m] = floorf(ex[m]) - 7.f;
          high |= ex[m] > ref[m] + kRaise;
        }
#pragma unroll
        for (int m = 0; m < 4; m += 2) {
          const f2 c = pack2(ex[m] == -INFINITY ? 0.f : -ex[m], ex[m + 1] == -INFINITY ? 0.f : -ex[m + 1]);
          f2 sum = pack2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            unpack2(add2(pack2(u[j][m], u[j][m + 1]), c), u[j][m], u[j][m + 1]);
            u[j][m] = fast_exp2(u[j][m]);
            u[j][m + 1] = fast_exp2(u[j][m + 1]);
            sum = fma2(pack2(u[j][m], u[j][m + 1]), pack2(inv[j], inv[j]), sum);
          }
          unpack2(sum, lt[m], lt[m + 1]);
        }
        if (__any_sync(0xffffffffu, !plain)) {
          // signs, and items of no value
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float ks = mts[8 * j].x;
#pragma unroll
            for (int m = 0; m < 4; ++m) u[j][m] = ks == 0.f ? 0.f : ks < 0.f ? -u[j][m] : u[j][m];
          }
        }
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t h0, h1, l0, l1;
          split2(u[j][0], u[j][1], h0, l0);
          split2(u[j][2], u[j][3], h1, l1);
          hw[j] = h0 | (h1 << 16);
          lw[j] = l0 | (l1 << 16);
        }
        if (__any_sync(0xffffffffu, high) && lane == 0) raise[done & 1] = 1;
        // the last tile's product has read P and its scales
        if (im > 0) ok = ok && tc::mbar_wait(&bars->kv_empty[(im - 1) & 1][1], ((im - 1) >> 1) & 1, abort_flag);
        tc::tc_fence_after();  // O and P's scales are read and written below
        if (!__all_sync(0xffffffffu, ok) && lane == 0) {
          *abort_flag = 1;
          raise[done & 1] = 2;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int item = 32 * w + (lane >> 2) + 8 * j;
          *reinterpret_cast<uint32_t*>(sm + kPOff + tc::sw128_off(item, qd) + 4 * c4) = hw[j];
          *reinterpret_cast<uint32_t*>(sm + kPOff + tc::sw128_off(item, 4 + qd) + 4 * c4) = lw[j];
        }
        // The block scales 2^(ex - ref), a byte per row and warp: lane
        // 4 m + c writes row 4 c + m of the quarter.
        auto put_scales = [&]() {
          float e = ex[0], r = ref[0];
#pragma unroll
          for (int m = 1; m < 4; ++m)
            if (lane >> 2 == m) {
              e = ex[m];
              r = ref[m];
            }
          const float d = e == -INFINITY ? -122.f : fminf(fmaxf(e - r, -122.f), 120.f);
          if (lane < 16) sf[4 * (row_h + (lane >> 2)) + w] = (uint8_t)((int)d + 127);
        };
        put_scales();
        named_sync(bar);
        tc::fence_proxy_async_smem();
        const int up = raise[done & 1];
        if (up) {
          if (up == 2) {  // a wait gave up: the half's warps leave together
            ok = false;
            break;
          }
          // a row's weights passed its reference by 2^kRaise: raise it, and
          // O^T (the product before this tile is done), sums and scales with it
#pragma unroll
          for (int m = 0; m < 4; ++m)
            if (lane < 4) red[32 * w + row_h + m] = ex[m];
          named_sync(bar);
          if (w == 0 && lane == 0 && !(qd & 1)) raise[done & 1] = 0;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int n = row_h + m;
            const float nm = fmaxf(fmaxf(fmaxf(red[n], red[32 + n]), fmaxf(red[64 + n], red[96 + n])), ref[m]);
            const float f = exp2f(ref[m] - nm);
            ref[m] = nm;
            l[m] *= f;
            if (w == 0 && lane < 4) {
              fac[row_t + m] = f;
              row_ref[row_t + m] = nm;
            }
          }
          put_scales();
          named_sync(bar);
          if (any) scale_rows(lanes + kOCol + 16 * qd, fac + 16 * qd);
        }
        any = true;
        // the two quarters write the hi and the lo terms' scales of the half
        const uint32_t word = reinterpret_cast<const uint32_t*>(sf)[lane];
        tmem_st1(lanes + (qd & 1 ? kSfLo : kSfHi) + hh, qd & 1 ? word - 0x04040404u : word);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->p_full);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          // 2^(ex - ref), an integer power below 2^21
          const float d = fmaxf(ex[m] - ref[m], -127.f);
          l[m] = fmaf(lt[m], __int_as_float(((int)d + 127) << 23), l[m]);
        }
        im += t.images;
        ++done;
      }
      if (seg_last) {
        ok = tc::mbar_wait(&bars->pv_done, seg & 1, abort_flag);
        if (named_or(bar, !ok)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        ++seg;
        // the rows' sums over all items
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          float sum = l[m];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (lane < 4) red[32 * w + row_h + m] = sum;
        }
        named_sync(bar);
        const bool whole = seg_tile0 == 0 && x.tile + 1 == x.te + x.tr;
        // a block's first segment's partial result is its slot 0, its last one's slot 1
        const size_t slot = 2 * (size_t)blockIdx.x + (i + 1 - (x.tile + 1 - seg_tile0) > 0 ? 1 : 0);
        if (w == 0 && lane < 16) {
          const int n = (16 * qd & 31) + lane;
          const float sum = (red[n] + red[32 + n]) + (red[64 + n] + red[96 + n]);
          fac[16 * qd + lane] = whole ? (sum != 0.f ? 1.f / sum : 0.f) : 1.f;  // a NaN stays one
          if (!whole) p.w.part_ml[slot * kR + 16 * qd + lane] = make_float2(row_ref[16 * qd + lane], sum);
        }
        named_sync(bar);
        // O^T: lane = dim, column = row
        const int pairs = a.rope.rope_dim >> 1;
#pragma unroll 1
        for (int g = 0; g < 8; ++g) {
          const int d = 128 * (g >> 1) + 32 * w + lane, r0 = 16 * qd + 8 * (g & 1);
          const int pair = (d - a.rope.rope_offset) >> 1;
          const bool rot = whole && d >= a.rope.rope_offset && pair < pairs;
          uint32_t r8[8];
          float v[8];
          tmem_ld8(lanes + kOCol + kR * (g >> 1) + r0, r8);
          tc::tmem_wait_ld();
#pragma unroll
          for (int n = 0; n < 8; ++n) v[n] = any ? __uint_as_float(r8[n]) * fac[r0 + n] : 0.f;
          if (__any_sync(0xffffffffu, rot)) {
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const float other = __shfl_xor_sync(0xffffffffu, v[n], 1);
              if (rot) {
                const float2 f = p.w.rope[(size_t)vis[r0 + n].z * pairs + pair];
                v[n] = (d & 1) ? __fadd_rn(__fmul_rn(other, -f.y), __fmul_rn(v[n], f.x))
                               : __fsub_rn(__fmul_rn(v[n], f.x), __fmul_rn(other, -f.y));
              }
            }
          }
          if (!whole) {
            float* o = p.w.part_o + (slot * kR + r0) * kD + d;
#pragma unroll
            for (int n = 0; n < 8; ++n)
              if (r0 + n < x.nrows) o[n * kD] = v[n];
          } else {
            // even lanes store a pair of dims of rows r0 + 2 k, odd lanes of the row after
            uint32_t* o = reinterpret_cast<uint32_t*>(a.out + (size_t)(x.row0 + r0 + (lane & 1)) * kD + (d & ~1));
#pragma unroll
            for (int n = 0; n < 8; n += 2) {
              const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? v[n] : v[n + 1], 1);
              const float lo = lane & 1 ? got : v[n], hi = lane & 1 ? v[n + 1] : got;
              if (r0 + n + (lane & 1) < x.nrows)
                o[n * (kD / 2)] = float_to_bf16_bits(lo) | ((uint32_t)float_to_bf16_bits(hi) << 16);
            }
          }
        }
        named_sync(bar);  // fac and the references are free
        seg_open = true;
      }
      tile_next(p, x);
    }
    if (!ok) {
      *abort_flag = 1;
      flag(a.dev_status, V4KV_DEV_TIMEOUT);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 20) {
    tc::tc_fence_after();
    tc::tmem_free(tmem, kCols);
  }
}

// Units whose tiles more than one block ran. grid (blocks, 8), a warp per row:
// block c joins the unit that its range begins inside, if it is the first to
// begin there.
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ Params p) {
  // What the prep kernel wrote is read before the wait: the sweep launched this
  // grid after its own wait for that kernel.
  tc::pdl_launch_dependents();
  const int c = blockIdx.x;
  const int4 rec = p.w.rec[c];
  const int begin = rec.x - rec.w;  // the unit's first tile
  if (c == 0 || rec.w == 0 || p.w.rec[max(c - 1, 0)].x > begin) {
    tc::pdl_wait();
    return;
  }
  const TreeArgs& a = p.a;
  Unit x;
  unit_load(p, x, rec.y);
  const int end = begin + x.te + x.tr;
  const int row = 8 * blockIdx.y + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  tc::pdl_wait();
  if (row >= x.nrows) return;
  float acc[16], m = kNone, l = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int k = c - 1; k < p.grid && p.w.rec[k].x < end; ++k) {
    if (p.w.rec[k].x == p.w.rec[k + 1].x) continue;
    const size_t slot = 2 * (size_t)k + (p.w.rec[k].x < begin ? 1 : 0);
    const float2 ml = p.w.part_ml[slot * kR + row];
    const float4* o = reinterpret_cast<const float4*>(p.w.part_o + (slot * kR + row) * kD);
    float4 vv[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) vv[q] = o[32 * q + lane];
    const float nm = fmaxf(m, ml.x), f0 = exp2f(m - nm), f1 = exp2f(ml.x - nm);
    m = nm;
    l = l * f0 + ml.y * f1;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 v = vv[q];
      acc[4 * q] = acc[4 * q] * f0 + v.x * f1;
      acc[4 * q + 1] = acc[4 * q + 1] * f0 + v.y * f1;
      acc[4 * q + 2] = acc[4 * q + 2] * f0 + v.z * f1;
      acc[4 * q + 3] = acc[4 * q + 3] * f0 + v.w * f1;
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const int node = (int)((x.row0 + row) / a.heads);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = acc[4 * q + e] * inv;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const int d = 128 * q + 4 * lane + e - a.rope.rope_offset;
      if (d >= 0 && d < a.rope.rope_dim) {
        const float2 f = p.w.rope[(size_t)node * (a.rope.rope_dim >> 1) + (d >> 1)];
        rope_apply(v[e], v[e + 1], f.x, -f.y);
      }
    }
    const uint32_t lo = float_to_bf16_bits(v[0]) | ((uint32_t)float_to_bf16_bits(v[1]) << 16);
    const uint32_t hi = float_to_bf16_bits(v[2]) | ((uint32_t)float_to_bf16_bits(v[3]) << 16);
    reinterpret_cast<uint2*>(a.out + (size_t)(x.row0 + row) * kD)[32 * q + lane] = make_uint2(lo, hi);
  }
}

// In order: blocks for the sequences' nodes (depths, ancestors, units, and 256 of
// the rotations each: a tree of 128 nodes has 16 of them, 37 -> 32 us in all),
// one for the sequences' costs and the grid's ranges, then those for raw rows (a
// warp takes kPrepRows of a sequence) and for Q as two e4m3 terms, once for all
// units, and for entries to be gathered.
__global__ void __launch_bounds__(256) tree_prep_kernel(const __grid_constant__ Params p) {
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  const TreeArgs& a = p.a;
  const int b = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int trees = a.batch * p.rope_blocks;
  if (b < trees) {
    // block `part` of a sequence: 256 of the nodes' rotations, and part 0 the rest
    const int part = blockIdx.x / a.batch, b = blockIdx.x - part * a.batch;
    int32_t* st = part == 0 ? a.dev_status : nullptr;
    __shared__ int parent[V4KV_MAX_TREE_NODES];
    __shared__ int depth[V4KV_MAX_TREE_NODES];
    const TreeSeq s = tree_seq(a.cu_nodes, b, a.total_nodes, a.max_nodes, t == 0 ? st : nullptr);
    if (t == 0 && a.seq_lens[b] > a.max_len) flag(st, V4KV_DEV_OVERFLOW);
    if (t < s.n) parent[t] = tree_parent(a.parents, s.first, t, st);
    __syncthreads();
    if (t < s.n) {
      uint32_t m[4] = {0, 0, 0, 0};
      int d = -1;
      for (int i = t; i >= 0; i = parent[i]) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i >> 5 == k) m[k] |= 1u << (i & 31);
        ++d;
      }
      if (part == 0) {
        p.w.anc[s.first + t] = make_uint4(m[0], m[1], m[2], m[3]);
        p.w.depth[s.first + t] = d;
      }
      depth[t] = d;
    }
    __syncthreads();
    // the units, and behind the last one the next sequence's first
    const SeqPlan plan = plan_of(p, b, nullptr);
    for (int u = t; u < plan.units && part == 0; u += 256) {
      int next = unit_index(p, plan, b, u + 1);
      if (u + 1 == plan.units) {
        next = -1;
        for (int bb = b + 1; bb < a.batch && next < 0; ++bb) {
          const SeqPlan q = plan_of(p, bb, nullptr);
          if (q.units > 0) next = unit_index(p, q, bb, 0);
        }
      }
      unit_store(p, plan, b, u, depth, next);
    }
    const int L = seq_len(a, b), pairs = a.rope.rope_dim >> 1;
    const int k = 256 * part + t;
    if (k < s.n * pairs) {
      const int i = k / pairs;
      float c, sn;
      rope_cs(a.rope, k - i * pairs, (long long)L + depth[i], &c, &sn);
      p.w.rope[(size_t)s.first * pairs + k] = make_float2(c, sn);
    }
    return;
  }
  const int raw_end = trees + 1 + a.batch * p.raw_blocks, q_end = raw_end + 2 * a.batch * p.max_units;
  if (b >= q_end) {
    // kStageRows entries a warp, of the whole tiles that every node sees
    const int per = p.staged / (8 * kStageRows), bb = (b - q_end) / per;
    const int j0 = ((b - q_end) % per * 8 + warp) * kStageRows;
    const int L = seq_len(a, bb);
    if (j0 >= seen_by_all(p, L) / kT * kT) return;
    const TreeSeq s = tree_seq(a.cu_nodes, bb, a.total_nodes, a.max_nodes, nullptr);
    if (s.n == 0) return;
    const size_t row = (size_t)bb * p.staged + j0;
    const PoolArgs& pool = a.main;
    int slot = -1;
    float kept = 0.f;
    if (lane < kStageRows) {
      const int pg = page_of(pool.block_table + (size_t)bb * pool.max_blocks, pool.max_blocks, j0 + lane, pool.spb,
                             pool.num_pages, a.dev_status);
      if (pg >= 0) slot = pg * pool.spb + (j0 + lane) % pool.spb;
      if (pool.dtype == V4KV_FP8_E4M3 && slot >= 0) kept = pool.scales[slot];
    }
    if (pool.dtype == V4KV_BF16) {
      uint4 v[kStageRows][2];
#pragma unroll
      for (int k = 0; k < kStageRows; ++k) {
        const int at = __shfl_sync(0xffffffffu, slot, k);
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pool.data) + (size_t)max(at, 0) * (2 * kD));
#pragma unroll
        for (int e = 0; e < 2; ++e) v[k][e] = at >= 0 ? src[2 * lane + e] : make_uint4(0, 0, 0, 0);
      }
      uint4* dst = reinterpret_cast<uint4*>(p.w.ent + row * (2 * kD)) + lane;
#pragma unroll
      for (int k = 0; k < kStageRows; ++k) {
        uint4 hi, lo;
        const float scale = split_row(v[k], hi, lo);
        dst[k * (2 * kD / 16)] = hi;
        dst[k * (2 * kD / 16) + kD / 16] = lo;
        if (lane == k) p.w.ent_meta[row + k] = make_float2(scale, slot >= 0 ? 0.f : -INFINITY);
      }
      return;
    }
    uint4 v[kStageRows];
#pragma unroll
    for (int k = 0; k < kStageRows; ++k) {
      const int at = __shfl_sync(0xffffffffu, slot, k);
      v[k] = make_uint4(0, 0, 0, 0);
      if (at >= 0) v[k] = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pool.data) + (size_t)at * kD)[lane];
    }
    uint4* dst = reinterpret_cast<uint4*>(p.w.ent + row * kD) + lane;
    unsigned zeros = 0;
#pragma unroll
    for (int k = 0; k < kStageRows; ++k) {
      dst[k * (kD / 16)] = v[k];
      if (!__any_sync(0xffffffffu, (v[k].x | v[k].y | v[k].z | v[k].w) & 0x7f7f7f7fu)) zeros |= 1u << k;
    }
    if (lane < kStageRows)
      p.w.ent_meta[row + lane] = slot < 0 ? make_float2(0.f, -INFINITY)
                                          : make_float2(zeros >> lane & 1 ? 0.f : kept, 0.f);
    return;
  }
  if (b >= raw_end) {
    // half a unit's Q: row 4 c + 2 k + e of a quarter at row 8 k + 2 c + e of it
    // (hi terms) and 64 rows on (lo terms)
    const int g = (b - raw_end) >> 1, hh = (b - raw_end) & 1;
    const int bb = g / p.max_units, uu = g - bb * p.max_units;
    const SeqPlan q = plan_of(p, bb, nullptr);
    if (uu >= q.units) return;
    int nrows;
    size_t row0;
    if (p.per_node) {
      const int i = uu / p.hc, h0 = (uu - i * p.hc) * kR;
      nrows = min(kR, a.heads - h0);
      row0 = (size_t)(q.s.first + i) * a.heads + h0;
    } else {
      nrows = min(kR, q.s.n * a.heads - uu * kR);
      row0 = (size_t)q.s.first * a.heads + uu * kR;
    }
    const int img = unit_index(p, q, bb, uu);
    uint4 raw[kPrepRows][4];
#pragma unroll
    for (int k = 0; k < kPrepRows; ++k) {
      const int n = 32 * hh + kPrepRows * warp + k;
      const size_t at = (row0 + n) * kD + 16 * lane;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        raw[k][e] = make_uint4(0, 0, 0, 0);
        if (n >= nrows) continue;
        if (a.q_dtype == V4KV_FP32) raw[k][e] = reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + at)[e];
        else if (e < 2) raw[k][e] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at)[e];
      }
    }
#pragma unroll
    for (int k = 0; k < kPrepRows; ++k) {
      float v[16];
      if (a.q_dtype == V4KV_FP32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[4 * e] = __uint_as_float(raw[k][e].x);
          v[4 * e + 1] = __uint_as_float(raw[k][e].y);
          v[4 * e + 2] = __uint_as_float(raw[k][e].z);
          v[4 * e + 3] = __uint_as_float(raw[k][e].w);
        }
      } else {
        bf16x16(raw[k], v);
      }
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
      m = __reduce_max_sync(0xffffffffu, m);
      uint4 hi, lo;
      split16(v, scale_up(m), hi, lo);
      const int n = kPrepRows * warp + k;  // row of the half
      const int at = 32 * hh + (n & 16) + 8 * ((n >> 1) & 1) + 2 * ((n >> 2) & 3) + (n & 1);
      uint8_t* dst = p.w.q + (size_t)img * 65536 + (lane >> 3) * kChunk;
      *reinterpret_cast<uint4*>(dst + tc::sw128_off(at, lane & 7)) = hi;
      *reinterpret_cast<uint4*>(dst + tc::sw128_off(kR + at, lane & 7)) = lo;
      if (lane == 0)
        p.w.q_factor[(size_t)img * kR + 32 * hh + n] =
            m >= 0x7f800000u ? __int_as_float(0x7fffffff) : scale_down(m) * (a.sm_scale * 1.4426950408889634f);
    }
    return;
  }
  if (b > trees) {
    const int per = p.raw_blocks, bb = (b - trees - 1) / per;
    const SeqPlan q = plan_of(p, bb, nullptr);
    const int w0 = raw_w0(a, q), n_win = q.L - w0, n = q.s.n > 0 ? n_win + q.s.n : 0;
    const int r0 = ((b - trees - 1) % per * 8 + warp) * kPrepRows;
    const bool fp8 = a.window.dtype == V4KV_FP8_E4M3;
    const size_t base = raw_row0(a, q, bb);
    uint4 raw[kPrepRows][2];
    float scale[kPrepRows];
    int kind[kPrepRows];  // 0: no such row, 1: bf16, 2: fp8
#pragma unroll
    for (int k = 0; k < kPrepRows; ++k) {
      raw[k][0] = raw[k][1] = make_uint4(0, 0, 0, 0);
      scale[k] = 0.f;
      kind[k] = 0;
      const int r = r0 + k;
      if (r >= n) continue;
      const uint4* src = nullptr;
      if (r >= n_win) {
        src = reinterpret_cast<const uint4*>(a.k_tree + (size_t)(q.s.first + r - n_win) * kD);
        kind[k] = 1;
      } else {
        const int tok = w0 + r;
        const int pg = page_of(a.window.block_table + (size_t)bb * a.window.max_blocks, a.window.max_blocks, tok,
                               a.window.spb, a.window.num_pages, a.dev_status);
        if (pg < 0) continue;
        const size_t slot = (size_t)pg * a.window.spb + tok % a.window.spb;
        kind[k] = fp8 ? 2 : 1;
        src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.window.data) + slot * (fp8 ? kD : 2 * kD));
        if (fp8) scale[k] = a.window.scales[slot];
      }
      raw[k][0] = src[kind[k] == 2 ? lane : 2 * lane];
      if (kind[k] == 1) raw[k][1] = src[2 * lane + 1];
    }
#pragma unroll
    for (int k = 0; k < kPrepRows; ++k) {
      if (kind[k] == 0) {
        if (r0 + k < n && lane == 0) p.w.raw_meta[base + r0 + k] = make_float2(0.f, -INFINITY);
        continue;
      }
      uint4 hi = raw[k][0], lo = make_uint4(0, 0, 0, 0);
      if (kind[k] == 1) {
        scale[k] = split_row(raw[k], hi, lo);
      } else if (__any_sync(0xffffffffu, has_nan_code(hi))) {
        hi = lo;
        scale[k] = __int_as_float(0x7fffffff);
      } else if (!__any_sync(0xffffffffu, (hi.x | hi.y | hi.z | hi.w) & 0x7f7f7f7fu)) {
        scale[k] = 0.f;  // a row of zeros
      }
      uint4* dst = reinterpret_cast<uint4*>(p.w.raw + (base + r0 + k) * (2 * kD));
      dst[lane] = hi;
      dst[32 + lane] = lo;
      if (lane == 0) p.w.raw_meta[base + r0 + k] = make_float2(scale[k], 0.f);
    }
    return;
  }
  __shared__ long long csum[8];
  __shared__ int tsum[8];
  long long ccarry = 0;
  int tcarry = 0;
  bool falls = false;
  for (int base = 0; base < a.batch; base += 256) {
    const int bb = base + t;
    long long cost = 0;
    int tiles = 0;
    if (bb < a.batch) {
      const SeqPlan q = plan_of(p, bb, nullptr);
      falls |= a.cu_nodes[bb] > a.cu_nodes[bb + 1];
      cost = (long long)q.units * unit_cost(p, q);
      tiles = q.units * (q.te + q.tr);
    }
    long long ci = cost;
    int ti = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long cy = __shfl_up_sync(0xffffffffu, ci, o);
      const int ty = __shfl_up_sync(0xffffffffu, ti, o);
      if (lane >= o) {
        ci += cy;
        ti += ty;
      }
    }
    if (lane == 31) {
      csum[warp] = ci;
      tsum[warp] = ti;
    }
    __syncthreads();
    for (int k = 0; k < warp; ++k) {
      ci += csum[k];
      ti += tsum[k];
    }
    if (bb < a.batch) {
      p.w.cost[bb] = ccarry + ci - cost;
      p.w.tiles[bb] = tcarry + ti - tiles;
    }
    for (int k = 0; k < 8; ++k) {
      ccarry += csum[k];
      tcarry += tsum[k];
    }
    __syncthreads();
  }
  // Sequences that share rows share the workspace's records of them: nothing runs
  // (the sequences with a negative count have been flagged).
  if (__syncthreads_or(falls)) tcarry = 0;
  const int blocks = min(p.grid, tcarry);
  for (int c = t; c <= p.grid; c += 256) {
    int4 rec = make_int4(tcarry, 0, 0, 0);
    if (c < blocks) {
      const long long target = (long long)c * ccarry / blocks;
      int lo = 0, hi = a.batch - 1;  // the last sequence that begins at or before the target
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (p.w.cost[m] <= target) lo = m; else hi = m - 1;
      }
      const SeqPlan q = plan_of(p, lo, nullptr);
      const int uc = unit_cost(p, q), n = q.te + q.tr;
      const long long off = target - p.w.cost[lo];
      const int u = (int)(off / uc), k = tile_at_cost(p, q, (int)(off % uc));
      rec = make_int4(p.w.tiles[lo] + u * n + k, unit_index(p, q, lo, u), 0, k);
    }
    p.w.rec[c] = rec;
  }
}

namespace {

int units_per_seq(int heads, int max_nodes, int k) {
  return heads % kR == 0 || k > 0 ? max_nodes * ((heads + kR - 1) / kR) : (max_nodes * heads + kR - 1) / kR;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Entries per sequence that the prep kernel copies to consecutive rows, in whole
// tiles, or 0. What is copied comes by TMA boxes of 64 rows, as pages of 64 do;
// every unit of a sequence reads it, so the copy has to be shared.
// fp8 at ratio 128: a page has two entries, and a tile's 128 rows come by 16-byte
// asynchronous copies, 6100 cycles against 3200 of products. With 32 sequences of
// 128K to 1M tokens 382 us against 428 for 16 units each, but 132 against 129 for
// four and 74 against 57 for one.
// bf16: the copy is split into its two terms, which the sweep does again for
// every unit (11000 cycles a tile). 42 sequences of 65K to 844K tokens at ratio 128:
// 425 us against 777 for six units each, 205 against 281 for two. Where each
// block has a tile or less it only adds a step: one sequence of 2000 tokens and
// four units 37 against 35 us, of 9000 47 against 46, of 20000 66 against 73.
int staged_rows(int batch, int heads, int max_nodes, int k, int window_len, int max_len, int ratio, int main_dtype) {
  const bool two = main_dtype != V4KV_FP8_E4M3;
  if ((ratio != 128 && !two) || k > 0) return 0;
  const int units = units_per_seq(heads, max_nodes, k);
  if (units < (two ? 2 : 6)) return 0;
  const long long n = max(0LL, max_len + 1LL - window_len) / ratio / kT * kT;
  if (two && (long long)batch * units < 16 && n < 4096) return 0;
  return batch * n <= (two ? 1LL << 20 : 1LL << 21) ? (int)n : 0;  // at most 1.1 GB
}

size_t layout(TreeWs* w, uint8_t* base, int batch, int heads, int total_nodes, int k, int window_len,
              int max_len, int grid, int staged, int main_dtype) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = base ? base + at : nullptr;
    at += up(bytes);
    return r;
  };
  TreeWs x{};
  x.anc = reinterpret_cast<uint4*>(take((size_t)total_nodes * sizeof(uint4)));
  x.depth = reinterpret_cast<int32_t*>(take((size_t)total_nodes * 4));
  x.rope = reinterpret_cast<float2*>(take((size_t)total_nodes * kPairs * sizeof(float2)));
  // unit_index() at most: whole units per node, or rows in units and one per sequence
  const size_t images = heads % kR == 0 || k > 0 ? (size_t)total_nodes * ((heads + kR - 1) / kR)
                                                 : (size_t)total_nodes * heads / kR + batch + 1;
  x.q = take(images * 65536);
  x.q_factor = reinterpret_cast<float*>(take(images * kR * sizeof(float)));
  x.units = reinterpret_cast<int4*>(take(images * 4 * sizeof(int4)));
  const size_t raws = (size_t)batch * (window_len - 1 < max_len ? window_len - 1 : max_len) + total_nodes;
  x.raw = take(raws * 2 * kD);
  x.raw_meta = reinterpret_cast<float2*>(take(raws * sizeof(float2)));
  x.ent = take((size_t)batch * staged * (main_dtype == V4KV_FP8_E4M3 ? kD : 2 * kD));
  x.ent_meta = reinterpret_cast<float2*>(take((size_t)batch * staged * sizeof(float2)));
  x.cost = reinterpret_cast<long long*>(take(((size_t)batch + 1) * 8));
  x.tiles = reinterpret_cast<int32_t*>(take(((size_t)batch + 1) * 4));
  x.rec = reinterpret_cast<int4*>(take(((size_t)grid + 1) * sizeof(int4)));
  x.part_o = reinterpret_cast<float*>(take((size_t)grid * 2 * kR * kD * 4));
  x.part_ml = reinterpret_cast<float2*>(take((size_t)grid * 2 * kR * sizeof(float2)));
  if (w) *w = x;
  return at;
}

}  // namespace

bool tree_sizes_ok(int batch, int heads, int total_nodes, int max_nodes, int k, int window_len, int max_len, int ratio) {
  const long long most = 0x7fffffffLL, per = (heads + kR - 1) / kR;
  if ((long long)total_nodes * heads > most) return false;
  if ((long long)batch * (window_len - 1 < max_len ? window_len - 1 : max_len) + total_nodes > most) return false;
  // tiles of all units, and blocks of the prep kernel
  const long long units = heads % kR == 0 || k > 0 ? total_nodes * per : (long long)total_nodes * heads / kR + batch + 1;
  const long long te = ((k > 0 ? k : max(0LL, (long long)max_len + max_nodes - window_len) / ratio) + kT - 1) / kT;
  const long long raw = min((long long)max_len, window_len - 1LL) + max_nodes;
  if (units * (te + (raw + kT - 1) / kT) > most) return false;
  return batch * (2 + max_nodes + raw / (8 * kPrepRows) + 2LL * units_per_seq(heads, max_nodes, k)) +
             (1LL << 21) / (8 * kStageRows) < most;
}

size_t tree_workspace_bytes(int batch, int heads, int total_nodes, int max_nodes, int k, int window_len, int max_len,
                            int ratio, int main_dtype, int num_sms) {
  return layout(nullptr, nullptr, batch, heads, total_nodes, k, window_len, max_len, num_sms,
                staged_rows(batch, heads, max_nodes, k, window_len, max_len, ratio, main_dtype), main_dtype);
}

cudaError_t launch_tree_attention(const TreeArgs& a, void* workspace, int num_sms, cudaStream_t stream) {
  Params p{};
  p.a = a;
  p.grid = num_sms;
  p.per_node = a.topk != nullptr || a.heads % kR == 0;
  p.hc = (a.heads + kR - 1) / kR;
  p.max_units = units_per_seq(a.heads, a.max_nodes, a.topk ? a.k : 0);
  p.ratio_log = a.ratio == 4 ? 2 : 7;
  p.spb_log = 8 - p.ratio_log;
  p.rope_blocks = max(1, (a.max_nodes * (a.rope.rope_dim >> 1) + 255) / 256);
  p.raw_blocks = (min(a.window_len - 1, a.max_len) + a.max_nodes + 8 * kPrepRows - 1) / (8 * kPrepRows);
  p.staged = staged_rows(a.batch, a.heads, a.max_nodes, a.topk ? a.k : 0, a.window_len, a.max_len, a.ratio, a.main.dtype);
  layout(&p.w, static_cast<uint8_t*>(workspace), a.batch, a.heads, a.total_nodes, a.topk ? a.k : 0, a.window_len,
         a.max_len, p.grid, p.staged, a.main.dtype);
  cudaError_t e = cudaSuccess;
  const bool pages = a.topk == nullptr && a.main.dtype == V4KV_FP8_E4M3 && a.main.spb == 64 &&
                     (long long)a.main.num_pages * 64 < (1LL << 30) &&
                     (reinterpret_cast<uintptr_t>(a.main.scales) & 15) == 0;  // (their scales are read by fours)
  p.boxes = pages || p.staged > 0;
  if (p.boxes) {
    p.box_data = p.staged ? p.w.ent : static_cast<const uint8_t*>(a.main.data);
    p.box_rows = p.staged ? a.batch * p.staged : a.main.num_pages * 64;
    p.box_bytes = a.main.dtype == V4KV_FP8_E4M3 ? kD : 2 * kD;
    e = encode_cols_u8(&p.map, p.box_data, (uint64_t)p.box_rows, p.box_bytes, 128, 64);
    if (e != cudaSuccess) return e;
  }
  e = cudaFuncSetAttribute(tree_attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_prep_kernel, dim3(1 + a.batch * (p.rope_blocks + p.raw_blocks + 2 * p.max_units + p.staged / (8 * kStageRows))), dim3(256), 0, stream, p);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_attend_kernel, dim3(p.grid), dim3(kThreads), kSmemBytes, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_merge_kernel, dim3(p.grid, kR / 8), dim3(256), 0, stream, p);
}

}  // namespace v4kv
