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
//     and four of what is left, 2^-9 of a value in all, half of bf16's
//     rounding; a bf16 q is exact. Two fp8 products cost what one f16 product
//     does. q's two terms are one N = 128 operand, so V is read once for both.
//   - A bf16 row (window token, drafted token, bf16 entry) is two images hi and
//     lo of the same kind, scaled by a power of two: two fp8 tiles.
//   - e4m3 spans 2^-9 .. 448. P's terms carry a power-of-two scale for each row
//     and 32 items (the block scale of mxf8f6f4), so a weight keeps its
//     precision next to a dominating one elsewhere. Without it a long tail of
//     small weights would round to zero together.
// The normaliser and the running reference are fp32. With block scales P needs
// no fixed range, so the reference moves only when a score passes it by 2^40.
//
// Warps: 0-7 softmax (thread = item of the tile and 32 of the rows; also the
// unit's Q and its epilogue), 8-11 load tiles, 12 issues the MMAs.
//
// Schedule: the tiles of all units are one list; the prep kernel gives each
// block of the grid (one per SM) an equal share by estimated cost. A block that
// runs all tiles of a unit writes its output, any other leaves a partial result
// (O, m, l) that the merge kernel joins: a long context with few rows is split
// over the whole GPU.
#include "tc.cuh"
#include "tree.cuh"

namespace v4kv {

namespace {

constexpr int kR = 64;    // rows of a unit
constexpr int kT = 128;   // items of a tile
constexpr int kD = 512;
constexpr int kThreads = 416;
constexpr float kNone = -1e30f;  // reference of a row that has seen nothing
constexpr float kRaise = 40.f;   // log2 by which a score may pass its reference
constexpr int kPairs = kRopeTable;

// shared memory (bytes from a 1024-aligned base)
constexpr uint32_t kQOff = 0;                 // 4 x [128 rows (64 hi, 64 lo) x 128 dims]
constexpr uint32_t kVOff = 65536;             // 2 stages of 4 x [128 items x 128 dims]
constexpr uint32_t kStage = 65536;
constexpr uint32_t kChunk = 16384;
constexpr uint32_t kPOff = 196608;            // [128 items x (64 hi, 64 lo)]
constexpr uint32_t kMetaOff = 212992;         // [2][128] {scale, 0 or -inf}
constexpr uint32_t kRowOff = kMetaOff + 2048; // [64] {score factor, reference}
constexpr uint32_t kAncOff = kRowOff + 512;   // [64] ancestors of the row's node, 128 bits
constexpr uint32_t kVisOff = kAncOff + 1024;  // [64] {visible entries, first visible token}
constexpr uint32_t kRedOff = kVisOff + 512;   // [8][32] reductions over a warp's items
constexpr uint32_t kSfOff = kRedOff + 1024;   // [64] block scales of P, a byte per 32 items
constexpr uint32_t kFacOff = kSfOff + 256;    // [64] per-row factors
constexpr uint32_t kBarOff = kFacOff + 256;
constexpr uint32_t kMiscOff = kBarOff + 128;
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
  uint64_t kv_full[2], kv_empty[2];
  uint64_t q_full, s_full, p_full, pv_done, drain;
};

// What the prep kernel leaves in the workspace.
struct TreeWs {
  uint4* anc;         // [total_nodes] the node and its ancestors, a bit each
  int32_t* depth;     // [total_nodes]
  float2* rope;       // [total_nodes][kPairs] cos, sin at the node's position
  long long* cost;    // [batch + 1] prefix sums over sequences
  int32_t* tiles;     // [batch + 1]
  int4* rec;          // [grid + 1] a block's first tile: {index, sequence, unit in it, tile in that}
  float* part_o;      // [2 grid][64][512]
  float2* part_ml;    // [2 grid][64]
};

struct Params {
  TreeArgs a;
  TreeWs w;
  int grid;
  int hc;        // units per node (per_node)
  int per_node;  // a unit's rows belong to one node
};

__device__ __forceinline__ int seq_len(const TreeArgs& a, int b) {
  return min(max(a.seq_lens[b], 0), a.max_len);
}

// Tile counts and costs of a sequence's units (all of one sequence alike).
struct SeqPlan {
  TreeSeq s;
  int L, units, te, tr;
};

constexpr int kCostFp8 = 4, kCostTwo = 8, kCostSeg = 4;

__device__ __forceinline__ SeqPlan plan_of(const Params& p, int b, int32_t* st) {
  const TreeArgs& a = p.a;
  SeqPlan q;
  q.s = tree_seq(a.cu_nodes, b, a.total_nodes, a.max_nodes, st);
  q.L = seq_len(a, b);
  const int n = q.s.n;
  q.units = p.per_node ? n * p.hc : (n * a.heads + kR - 1) / kR;
  const int seen = max(0, q.L + n - a.window_len) / a.ratio;  // by the deepest node there can be
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
  int b, u, tile;      // the walk's position
  SeqPlan q;
  int node0;           // first node
  int nrows;
  long long row0;      // first row of out and q
  int n_ent;           // entries in the list (top-k slots, or visible to the deepest row)
  int n_all;           // entries that every row sees
  int w0, n_win;       // first cached token in the list, and how many
  int n_tree;          // nodes in the list
};

__device__ __forceinline__ void unit_set(const Params& p, Unit& x) {
  const TreeArgs& a = p.a;
  const int L = x.q.L, W = a.window_len;
  if (p.per_node) {
    const int i = x.u / p.hc, h0 = (x.u % p.hc) * kR;
    x.node0 = i;
    x.nrows = min(kR, a.heads - h0);
    x.row0 = (long long)(x.q.s.first + i) * a.heads + h0;
    const int d = p.w.depth[x.q.s.first + i];
    x.n_ent = a.topk ? a.k : max(0, L + d + 1 - W) / a.ratio;
    x.n_all = x.n_ent;
    x.w0 = min(L, max(0, L + d + 1 - W));
    x.n_win = L - x.w0;
    x.n_tree = d + 1;
  } else {
    const int r0 = x.u * kR, rows = x.q.s.n * a.heads;
    x.nrows = min(kR, rows - r0);
    x.node0 = r0 / a.heads;
    const int last = (r0 + x.nrows - 1) / a.heads;
    x.row0 = (long long)x.q.s.first * a.heads + r0;
    int lo = V4KV_MAX_TREE_NODES, hi = 0;
    for (int i = x.node0; i <= last; ++i) {
      const int d = p.w.depth[x.q.s.first + i];
      lo = min(lo, d);
      hi = max(hi, d);
    }
    x.n_ent = max(0, L + hi + 1 - W) / a.ratio;
    x.n_all = max(0, L + lo + 1 - W) / a.ratio;
    x.w0 = min(L, max(0, L + lo + 1 - W));
    x.n_win = L - x.w0;
    x.n_tree = last + 1;
  }
}

// next unit (after the last: b == batch)
__device__ __forceinline__ void unit_next(const Params& p, Unit& x) {
  ++x.u;
  x.tile = 0;
  while (x.u >= x.q.units) {
    x.u = 0;
    if (++x.b >= p.a.batch) return;
    x.q = plan_of(p, x.b, nullptr);
  }
  unit_set(p, x);
}

// A tile: whether its items are entries, the first one's index in its list,
// how many there are, and how many images its rows have.
struct Tile {
  bool entries;
  int first, count, images;
};

__device__ __forceinline__ Tile tile_of(const Params& p, const Unit& x) {
  Tile t;
  t.entries = x.tile < x.q.te;
  t.first = (t.entries ? x.tile : x.tile - x.q.te) * kT;
  t.count = min(kT, (t.entries ? x.n_ent : x.n_win + x.n_tree) - t.first);
  t.images = t.entries && p.a.main.dtype == V4KV_FP8_E4M3 ? 1 : 2;
  return t;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void named_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool named_or(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "bar.red.or.pred b, %2, 128, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}

// two e4m3 terms of a pair: x = hi + lo / 16
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const uint16_t h = float2_to_e4m3x2(x, y);
  const float2 f = __half22float2(e4m3x2_to_half2(h));
  hi = h;
  lo = float2_to_e4m3x2((x - f.x) * 16.f, (y - f.y) * 16.f);
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}

// maximum or sum of 32 per-lane values over a warp's lanes: lane l ends with
// the result of value l (31 shuffles)
template <bool kMax>
__device__ __forceinline__ float reduce_scatter32(float* v, int lane) {
#pragma unroll
  for (int n = 16; n > 0; n >>= 1) {
    const bool upper = (lane & n) != 0;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float mine = upper ? v[n + k] : v[k], other = upper ? v[k] : v[n + k];
      const float x = __shfl_xor_sync(0xffffffffu, other, n);
      v[k] = kMax ? fmaxf(mine, x) : mine + x;
    }
  }
  return v[0];
}

// ------------------------------------------------------------------ loading (warps 8-11)

// where an item's row is: null for an item that has none
struct Item {
  const uint8_t* p;
  float scale;
  bool fp8;
};

__device__ __forceinline__ Item item_of(const Params& p, const Unit& x, const Tile& t, int r, int32_t* st) {
  const TreeArgs& a = p.a;
  Item it{nullptr, 0.f, false};
  if (r >= t.count) return it;
  int j = t.first + r;
  const PoolArgs* pool;
  if (t.entries) {
    pool = &a.main;
    if (a.topk) {
      j = a.topk[(size_t)(x.q.s.first + x.node0) * a.k + j];
      if (j < 0) return it;
      if (j >= (x.q.L + a.ratio - 1) / a.ratio) {
        flag(st, V4KV_DEV_BAD_INDEX);
        return it;
      }
    }
  } else if (j < x.n_win) {
    pool = &a.window;
    j += x.w0;
  } else {
    j -= x.n_win;
    if (p.per_node) {  // the j-th of the node's ancestors
      const uint4 m4 = p.w.anc[x.q.s.first + x.node0];
      const uint32_t m[4] = {m4.x, m4.y, m4.z, m4.w};
      int k = 0;
      while (k < 3 && j >= __popc(m[k])) j -= __popc(m[k++]);
      j = 32 * k + (int)__fns(m[k], 0, j + 1);
    }
    it.p = reinterpret_cast<const uint8_t*>(a.k_tree + (size_t)(x.q.s.first + j) * kD);
    it.scale = 1.f;
    return it;
  }
  const int pg = page_of(pool->block_table + (size_t)x.b * pool->max_blocks, pool->max_blocks, j, pool->spb,
                         pool->num_pages, st);
  if (pg < 0) return it;
  const size_t slot = (size_t)pg * pool->spb + j % pool->spb;
  it.fp8 = pool->dtype == V4KV_FP8_E4M3;
  it.scale = it.fp8 ? pool->scales[slot] : 1.f;
  if (!isfinite(it.scale)) it.scale = __int_as_float(0x7fffffff);
  it.p = static_cast<const uint8_t*>(pool->data) + slot * (it.fp8 ? kD : 2 * kD);
  return it;
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

// one row, the whole warp: lane takes dims 16 lane .. 16 lane + 15
__device__ __forceinline__ void load_row(const Item& it, int r, int lane, uint8_t* hi_dst, uint8_t* lo_dst,
                                         float2* meta) {
  const uint32_t off = (lane >> 3) * kChunk + tc::sw128_off(r, lane & 7);
  uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
  float scale = it.scale;
  if (it.p) {
    bool bad;
    if (it.fp8) {
      hi = reinterpret_cast<const uint4*>(it.p)[lane];
      bad = __any_sync(0xffffffffu, has_nan_code(hi));
    } else {
      float v[16];
      bf16x16(reinterpret_cast<const uint4*>(it.p) + 2 * lane, v);
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
      m = __reduce_max_sync(0xffffffffu, m);
      bad = m >= 0x7f800000u;
      split16(v, scale_up(m), hi, lo);
      scale = scale_down(m);
    }
    if (bad) {
      hi = lo = make_uint4(0, 0, 0, 0);
      scale = __int_as_float(0x7fffffff);
    }
  }
  *reinterpret_cast<uint4*>(hi_dst + off) = hi;
  if (lo_dst) *reinterpret_cast<uint4*>(lo_dst + off) = lo;
  if (lane == 0) meta[r] = make_float2(scale, it.p ? 0.f : -INFINITY);
}

// ------------------------------------------------------------------ the sweep

}  // namespace

__global__ void __launch_bounds__(kThreads, 1) tree_attend_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = tc::smem_u32(smem_raw);
  const uint32_t pad = ((raw_addr + 1023u) & ~1023u) - raw_addr;
  uint8_t* sm = smem_raw + pad;
  const uint32_t sbase = raw_addr + pad;
  Bars* bars = reinterpret_cast<Bars*>(sm + kBarOff);
  float2* meta = reinterpret_cast<float2*>(sm + kMetaOff);
  float2* row_ar = reinterpret_cast<float2*>(sm + kRowOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kMiscOff + 4);
  const TreeArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&bars->kv_full[s], 128);
      tc::mbar_init(&bars->kv_empty[s], 1);
    }
    tc::mbar_init(&bars->q_full, 256);
    tc::mbar_init(&bars->s_full, 1);
    tc::mbar_init(&bars->p_full, 256);
    tc::mbar_init(&bars->pv_done, 1);
    tc::mbar_init(&bars->drain, 1);
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  if (warp == 12) tc::tmem_alloc(tmem_slot, kCols);
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int4 rec = p.w.rec[blockIdx.x];
  const int n_tiles = p.w.rec[blockIdx.x + 1].x - rec.x;
  if (n_tiles <= 0) {
    if (warp == 12) tc::tmem_free(tmem, kCols);
    return;
  }
  Unit x;
  x.b = rec.y;
  x.u = rec.z;
  x.tile = rec.w;
  x.q = plan_of(p, x.b, nullptr);
  unit_set(p, x);

  if (warp >= 8 && warp < 12) {
    // ======================= tiles into the stages. `im` counts images: image
    // im lives in stage im % 2.
    const int w = warp - 8;
    int32_t* st = a.dev_status;
    bool ok = true;
    uint32_t im = 0;
    for (int i = 0; i < n_tiles && ok; ++i) {
      const Tile t = tile_of(p, x);
      if (t.count > 0) {
        const uint32_t s = im & 1;
        for (int k = 0; k < t.images; ++k)
          if (im + k >= 2) ok = ok && tc::mbar_wait(&bars->kv_empty[(im + k) & 1], ((im + k - 2) >> 1) & 1, abort_flag);
        if (!ok) break;
        const Item mine = item_of(p, x, t, 32 * w + lane, st);
        float2* mt = meta + s * kT;
        uint8_t* dst = sm + kVOff + s * kStage;
        if (t.images == 1) {
          // rows from `safe` on are hidden from some of the unit's rows
          const int safe = max(0, min(32, x.n_all - t.first - 32 * w));
          mt[32 * w + lane] = make_float2(mine.scale, mine.p ? 0.f : -INFINITY);
          const uint8_t* any = static_cast<const uint8_t*>(a.main.data);
#pragma unroll 8
          for (int r = 0; r < 32; ++r) {
            const uint8_t* src = reinterpret_cast<const uint8_t*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.p), r));
            if (r < safe || !src)
              cp_async16(sbase + kVOff + s * kStage + (lane >> 3) * kChunk + tc::sw128_off(32 * w + r, lane & 7),
                         src ? src + 16 * lane : any, src != nullptr);
          }
          __syncwarp();
          for (int r = safe; r < 32; ++r) {
            Item it;
            it.p = reinterpret_cast<const uint8_t*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.p), r));
            it.scale = __shfl_sync(0xffffffffu, mine.scale, r);
            it.fp8 = true;
            if (it.p) load_row(it, 32 * w + r, lane, dst, nullptr, mt);
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
          uint8_t* lo = sm + kVOff + (s ^ 1) * kStage;
#pragma unroll 4
          for (int r = 0; r < 32; ++r) {
            Item it;
            it.p = reinterpret_cast<const uint8_t*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.p), r));
            it.scale = __shfl_sync(0xffffffffu, mine.scale, r);
            it.fp8 = __shfl_sync(0xffffffffu, (int)mine.fp8, r) != 0;
            load_row(it, 32 * w + r, lane, dst, lo, mt);
          }
        }
        tc::fence_proxy_async_smem();
        for (int k = 0; k < t.images; ++k) tc::mbar_arrive(&bars->kv_full[(im + k) & 1]);
        im += t.images;
      }
      if (++x.tile == x.q.te + x.q.tr && i + 1 < n_tiles) unit_next(p, x);
    }
    if (!ok) {
      *abort_flag = 1;
      flag(a.dev_status, V4KV_DEV_TIMEOUT);
    }
  } else if (warp == 12) {
    // ======================= MMA issue: the whole warp runs the loop, one lane
    // elected once issues
    const bool leader = tc::elect_one();
    const uint64_t v_k = tc::sw128_desc(sbase + kVOff, 16, 1024), v_m = tc::sw128_desc(sbase + kVOff, 1024, 1024);
    const uint64_t q_k = tc::sw128_desc(sbase + kQOff, 16, 1024);
    const uint64_t p_h = tc::sw128_desc(sbase + kPOff, 1024, 1024), p_l = tc::sw128_desc(sbase + kPOff + 64, 1024, 1024);
    bool ok = true, seg_open = true;
    uint32_t im = 0, done = 0, seg = 0;
    uint32_t filled = 0;  // O^T holds something of this segment
    for (int i = 0; i < n_tiles && ok; ++i) {
      const Tile t = tile_of(p, x);
      const bool seg_last = x.tile + 1 == x.q.te + x.q.tr || i + 1 == n_tiles;
      if (seg_open) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait_spin(&bars->q_full, seg & 1, abort_flag));
        if (!ok) break;
        seg_open = false;
        filled = 0;
      }
      if (t.count > 0) {
        for (int k = 0; k < t.images && ok; ++k) {
          const uint32_t s = (im + k) & 1;
          ok = __all_sync(0xffffffffu, tc::mbar_wait_spin(&bars->kv_full[s], ((im + k) >> 1) & 1, abort_flag));
          if (!ok) break;
          tc::tc_fence_after();
          if (leader) {
            const uint64_t vk = v_k + (uint64_t)(s * (kStage >> 4));
            const uint32_t sfa = tmem + (k ? kLow : kOne);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_mx(tmem + kSCol, vk + (uint64_t)((c * kChunk + kk * 32) >> 4),
                       q_k + (uint64_t)((c * kChunk + kk * 32) >> 4), idesc_mx(128, 0, 0), sfa, tmem + kSfQ,
                       (k | c | kk) ? 1u : 0u);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (leader) tc::mma_commit(&bars->s_full);
        __syncwarp();
        ok = __all_sync(0xffffffffu, tc::mbar_wait_spin(&bars->p_full, done & 1, abort_flag));
        if (!ok) break;
        tc::tc_fence_after();
        if (leader) {
          const int nk = (t.count + 31) >> 5;
          for (int k = 0; k < t.images; ++k) {
            const uint32_t s = (im + k) & 1;
            const uint64_t vm = v_m + (uint64_t)(s * (kStage >> 4));
            const uint32_t sfa = tmem + (k ? kLow : kOne);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (kk < nk) {
                  mma_mx(tmem + kOCol + kR * c, vm + (uint64_t)((c * kChunk + kk * 4096) >> 4),
                         p_h + (uint64_t)((kk * 4096) >> 4), idesc_mx(64, 1, kk), sfa, tmem + kSfHi,
                         (filled | k | kk) ? 1u : 0u);
                  mma_mx(tmem + kOCol + kR * c, vm + (uint64_t)((c * kChunk + kk * 4096) >> 4),
                         p_l + (uint64_t)((kk * 4096) >> 4), idesc_mx(64, 1, kk), sfa, tmem + kSfLo, 1u);
                }
            tc::mma_commit(&bars->kv_empty[s]);
          }
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
        seg_open = true;
      }
      if (++x.tile == x.q.te + x.q.tr && i + 1 < n_tiles) unit_next(p, x);
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
    // ======================= softmax: thread = item 32 (warp % 4) + lane of the
    // tile and rows 32 hh .. 32 hh + 31. The two halves never wait for each other.
    const int hh = warp >> 2, w = warp & 3, item = 32 * w + lane;
    const int bar = 1 + hh;
    const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
    float* red = reinterpret_cast<float*>(sm + kRedOff) + 128 * hh;       // [4][32]
    float* fac = reinterpret_cast<float*>(sm + kFacOff) + 32 * hh;        // [32]
    uint8_t* sf = sm + kSfOff + 128 * hh;                                  // [32][4]
    const uint4* anc = reinterpret_cast<const uint4*>(sm + kAncOff);
    const int2* vis = reinterpret_cast<const int2*>(sm + kVisOff);
    if (hh == 0) {
      const uint32_t one = 0x7f7f7f7fu, low = 0x7b7b7b7bu;
      tmem_st4(lanes + kOne, one, one, one, one);
      tmem_st4(lanes + kLow, low, low, low, low);
      tmem_st4(lanes + kSfQ, one, one, low, low);
      tmem_st4(lanes + kSfHi, one, one, one, one);
      tmem_st4(lanes + kSfLo, one, one, one, one);
      tc::tmem_wait_st();
    }
    bool ok = true, seg_open = true, any = false;
    int seg_tile0 = 0;
    uint32_t im = 0, done = 0, seg = 0;
    float l[32];
    for (int i = 0; i < n_tiles; ++i) {
      if (seg_open) {
        // the unit's Q (every product that reads the last one's has completed:
        // its S was read), the rows' factors, references and masks
        seg_open = false;
        any = false;
        seg_tile0 = x.tile;
#pragma unroll
        for (int n = 0; n < 32; ++n) l[n] = 0.f;
        for (int k = 0; k < 8; ++k) {
          const int n = 32 * hh + 8 * w + k;
          uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
          uint32_t m = 0;
          if (n < x.nrows) {
            float v[16];
            const size_t at = (size_t)(x.row0 + n) * kD + 16 * lane;
            if (a.q_dtype == V4KV_FP32) {
              const float4* q4 = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 f = q4[e];
                v[4 * e] = f.x; v[4 * e + 1] = f.y; v[4 * e + 2] = f.z; v[4 * e + 3] = f.w;
              }
            } else {
              bf16x16(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at), v);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
            m = __reduce_max_sync(0xffffffffu, m);
            split16(v, scale_up(m), hi, lo);
          }
          uint8_t* dst = sm + kQOff + (lane >> 3) * kChunk;
          *reinterpret_cast<uint4*>(dst + tc::sw128_off(n, lane & 7)) = hi;
          *reinterpret_cast<uint4*>(dst + tc::sw128_off(kR + n, lane & 7)) = lo;
          if (lane == 0)
            row_ar[n] = make_float2(m >= 0x7f800000u ? __int_as_float(0x7fffffff)
                                                     : scale_down(m) * (a.sm_scale * 1.4426950408889634f),
                                    kNone);
        }
        if (!p.per_node && w == 0) {
          const int n = 32 * hh + lane;
          const int node = n < x.nrows ? (int)((x.row0 - (long long)x.q.s.first * a.heads + n) / a.heads) : x.node0;
          const int d = p.w.depth[x.q.s.first + node];
          reinterpret_cast<uint4*>(sm + kAncOff)[n] = p.w.anc[x.q.s.first + node];
          const int w0 = max(0, x.q.L + d + 1 - a.window_len);
          reinterpret_cast<int2*>(sm + kVisOff)[n] = make_int2(w0 / a.ratio, w0);
        }
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        tc::mbar_arrive(&bars->q_full);
        named_sync(bar);
      }
      const Tile t = tile_of(p, x);
      const bool seg_last = x.tile + 1 == x.q.te + x.q.tr || i + 1 == n_tiles;
      if (t.count > 0) {
        ok = tc::mbar_wait_spin(&bars->s_full, done & 1, abort_flag, 32);
        tc::tc_fence_after();
        const float2 mt = meta[(im & 1) * kT + item];
        float s[32];
        {
          uint32_t r32[32];
          tc::tmem_ld32(lanes + kSCol + 32 * hh, r32);
          tc::tmem_wait_ld();
#pragma unroll
          for (int n = 0; n < 32; ++n) s[n] = __uint_as_float(r32[n]);
          tc::tmem_ld32(lanes + kSCol + kR + 32 * hh, r32);
          tc::tmem_wait_ld();
#pragma unroll
          for (int n = 0; n < 32; ++n) s[n] = (s[n] + __uint_as_float(r32[n])) * mt.x;
        }
        // rows that see this item
        uint32_t seen = mt.y == 0.f ? 0xffffffffu : 0u;
        if (!p.per_node && seen && (!t.entries || t.first + kT > x.n_all)) {
          const int r = t.first + item;
          uint32_t bits = 0;
#pragma unroll 4
          for (int n = 0; n < 32; ++n) {
            bool v;
            if (t.entries) {
              v = r < vis[32 * hh + n].x;
            } else if (r < x.n_win) {
              v = x.w0 + r >= vis[32 * hh + n].y;
            } else {
              const int k = r - x.n_win;
              v = (reinterpret_cast<const uint32_t*>(anc + 32 * hh + n)[k >> 5] >> (k & 31)) & 1;
            }
            bits |= (uint32_t)v << n;
          }
          seen = bits;
        }
        // exponents relative to the rows' references (a weight is 2^s[n])
        const float4* ar4 = reinterpret_cast<const float4*>(row_ar + 32 * hh);
        const float extra = fmaxf(0.f, __log2f(fabsf(mt.x)));  // a large scale counts in a weight's size
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < 32; n += 2) {
          const float4 f = ar4[n >> 1];
          float e0 = fmaf(s[n], f.x, -f.y), e1 = fmaf(s[n + 1], f.z, -f.w);
          if (!(seen >> n & 1)) e0 = -INFINITY;
          if (!(seen >> (n + 1) & 1)) e1 = -INFINITY;
          s[n] = e0;
          s[n + 1] = e1;
          top = fmaxf(top, fmaxf(e0, e1));
        }
        if (named_or(bar, top + extra > kRaise || !ok)) {
          if (named_or(bar, !ok)) {
            ok = false;
            break;
          }
          // raise the references to the rows' maxima so far, O^T and the sums with them
          // (the scores are taken from S again: a reference of kNone has swallowed them)
          float u[32];
          {
            uint32_t r32[32], q32[32];
            tc::tmem_ld32(lanes + kSCol + 32 * hh, r32);
            tc::tmem_ld32(lanes + kSCol + kR + 32 * hh, q32);
            tc::tmem_wait_ld();
#pragma unroll
            for (int n = 0; n < 32; n += 2) {
              const float4 f = ar4[n >> 1];
              const float y0 = (__uint_as_float(r32[n]) + __uint_as_float(q32[n])) * mt.x;
              const float y1 = (__uint_as_float(r32[n + 1]) + __uint_as_float(q32[n + 1])) * mt.x;
              s[n] = (seen >> n & 1) ? y0 * f.x : -INFINITY;
              s[n + 1] = (seen >> (n + 1) & 1) ? y1 * f.z : -INFINITY;
              u[n] = s[n] + extra;
              u[n + 1] = s[n + 1] + extra;
            }
          }
          const float mx = reduce_scatter32<true>(u, lane);
          red[32 * w + lane] = mx;
          named_sync(bar);
          if (w == 0) {
            float nm = fmaxf(fmaxf(red[lane], red[32 + lane]), fmaxf(red[64 + lane], red[96 + lane]));
            const float old = row_ar[32 * hh + lane].y;
            nm = fmaxf(nm, old);
            row_ar[32 * hh + lane].y = nm;
            fac[lane] = exp2f(old - nm);
          }
          named_sync(bar);
#pragma unroll
          for (int n = 0; n < 32; ++n) {
            l[n] *= fac[n];
            s[n] -= row_ar[32 * hh + n].y;
          }
          if (any) {
            // S is complete, so the last tile's product into O^T is
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t r32[32];
              tc::tmem_ld32(lanes + kOCol + kR * c + 32 * hh, r32);
              tc::tmem_wait_ld();
#pragma unroll
              for (int n = 0; n < 32; ++n) r32[n] = __float_as_uint(__uint_as_float(r32[n]) * fac[n]);
              tc::tmem_st32(lanes + kOCol + kR * c + 32 * hh, r32);
            }
            tc::tmem_wait_st();
          }
        }
        any = true;
        // weights of the items' codes, their block exponents, and the two terms
        uint32_t mine = 0;
        uint8_t* prow = sm + kPOff;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t hw[4], lw[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int n = 16 * g + 4 * q + e;
              const float pr = fast_exp2(s[n]);
              l[n] += pr;
              const float pw = (seen >> n & 1) ? pr * mt.x : 0.f;
              // largest exponent of the 32 items, as the block scale's byte for [2^7, 2^8)
              const uint32_t b = max(__reduce_max_sync(0xffffffffu, __float_as_uint(pw) & 0x7fffffffu) >> 23, 16u);
              if (lane == n) mine = b - 7u;
              v[e] = pw * __uint_as_float((261u - b) << 23);
            }
            uint32_t h0, h1, l0, l1;
            split2(v[0], v[1], h0, l0);
            split2(v[2], v[3], h1, l1);
            hw[q] = h0 | (h1 << 16);
            lw[q] = l0 | (l1 << 16);
          }
          *reinterpret_cast<uint4*>(prow + tc::sw128_off(item, 2 * hh + g)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
          *reinterpret_cast<uint4*>(prow + tc::sw128_off(item, 4 + 2 * hh + g)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        }
        sf[4 * lane + w] = (uint8_t)mine;
        named_sync(bar);
        const uint32_t word = reinterpret_cast<const uint32_t*>(sf)[lane];
        tmem_st1(lanes + kSfHi + hh, word);
        tmem_st1(lanes + kSfLo + hh, word - 0x04040404u);
        tc::tmem_wait_st();
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        tc::mbar_arrive(&bars->p_full);
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
        {
          float t32[32];
#pragma unroll
          for (int n = 0; n < 32; ++n) t32[n] = l[n];
          red[32 * w + lane] = reduce_scatter32<false>(t32, lane);
        }
        named_sync(bar);
        const bool whole = seg_tile0 == 0 && x.tile + 1 == x.q.te + x.q.tr;
        // a block's first segment's partial result is its slot 0, its last one's slot 1
        const size_t slot = 2 * (size_t)blockIdx.x + (i + 1 - (x.tile + 1 - seg_tile0) > 0 ? 1 : 0);
        if (w == 0) {
          const float sum = (red[lane] + red[32 + lane]) + (red[64 + lane] + red[96 + lane]);
          fac[lane] = whole ? (sum != 0.f ? 1.f / sum : 0.f) : 1.f;  // a NaN stays one
          if (!whole) p.w.part_ml[slot * kR + 32 * hh + lane] = make_float2(row_ar[32 * hh + lane].y, sum);
        }
        named_sync(bar);
        const float2* rope = p.w.rope;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r32[32];
          tc::tmem_ld32(lanes + kOCol + kR * c + 32 * hh, r32);
          tc::tmem_wait_ld();
          const int d = 128 * c + item, pair = ((d & ~1) - a.rope.rope_offset) >> 1;
          const bool rot = whole && d >= a.rope.rope_offset && d < a.rope.rope_offset + a.rope.rope_dim;
#pragma unroll
          for (int n = 0; n < 32; ++n) {
            float v = any ? __uint_as_float(r32[n]) * fac[n] : 0.f;
            const float other = __shfl_xor_sync(0xffffffffu, v, 1);
            const int row = 32 * hh + n;
            if (row >= x.nrows) continue;
            if (!whole) {
              p.w.part_o[(slot * kR + row) * kD + d] = v;
              continue;
            }
            if (rot) {
              const int node = (int)((x.row0 + row) / a.heads);
              float cs, sn;
              if (pair < kPairs) {
                const float2 f = rope[(size_t)node * kPairs + pair];
                cs = f.x;
                sn = f.y;
              } else {
                rope_cs(a.rope, pair, (long long)x.q.L + p.w.depth[node], &cs, &sn);
              }
              v = (d & 1) ? __fadd_rn(__fmul_rn(other, -sn), __fmul_rn(v, cs))
                          : __fsub_rn(__fmul_rn(v, cs), __fmul_rn(other, -sn));
            }
            a.out[(size_t)(x.row0 + row) * kD + d] = float_to_bf16_bits(v);
          }
        }
        named_sync(bar);  // fac and the references are free
        seg_open = true;
      }
      if (++x.tile == x.q.te + x.q.tr && i + 1 < n_tiles) unit_next(p, x);
    }
    if (!ok) {
      *abort_flag = 1;
      flag(a.dev_status, V4KV_DEV_TIMEOUT);
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc::tc_fence_after();
    tc::tmem_free(tmem, kCols);
  }
}

// Units whose tiles more than one block ran. grid (blocks, 8), a warp per row:
// block c joins the unit that its range begins inside, if it is the first to
// begin there.
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ Params p) {
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  const int c = blockIdx.x;
  const int4 rec = p.w.rec[c];
  const int begin = rec.x - rec.w;  // the unit's first tile
  if (c == 0 || rec.w == 0 || rec.y >= p.a.batch || p.w.rec[c - 1].x > begin) return;
  const TreeArgs& a = p.a;
  Unit x;
  x.b = rec.y;
  x.u = rec.z;
  x.tile = 0;
  x.q = plan_of(p, x.b, nullptr);
  unit_set(p, x);
  const int end = begin + x.q.te + x.q.tr;
  const int row = 8 * blockIdx.y + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= x.nrows) return;
  float acc[16], m = kNone, l = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int k = c - 1; k < p.grid && p.w.rec[k].x < end; ++k) {
    if (p.w.rec[k].x == p.w.rec[k + 1].x) continue;
    const size_t slot = 2 * (size_t)k + (p.w.rec[k].x < begin ? 1 : 0);
    const float2 ml = p.w.part_ml[slot * kR + row];
    const float nm = fmaxf(m, ml.x), f0 = exp2f(m - nm), f1 = exp2f(ml.x - nm);
    m = nm;
    l = l * f0 + ml.y * f1;
    const float4* o = reinterpret_cast<const float4*>(p.w.part_o + (slot * kR + row) * kD);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 v = o[32 * q + lane];
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
        float cs, sn;
        if ((d >> 1) < kPairs) {
          const float2 f = p.w.rope[(size_t)node * kPairs + (d >> 1)];
          cs = f.x;
          sn = f.y;
        } else {
          rope_cs(a.rope, d >> 1, (long long)x.q.L + p.w.depth[node], &cs, &sn);
        }
        rope_apply(v[e], v[e + 1], cs, -sn);
      }
    }
    const uint32_t lo = float_to_bf16_bits(v[0]) | ((uint32_t)float_to_bf16_bits(v[1]) << 16);
    const uint32_t hi = float_to_bf16_bits(v[2]) | ((uint32_t)float_to_bf16_bits(v[3]) << 16);
    reinterpret_cast<uint2*>(a.out + (size_t)(x.row0 + row) * kD)[32 * q + lane] = make_uint2(lo, hi);
  }
}

// grid (batch + 1). Block b < batch: depths, ancestors and rotations of its
// sequence's nodes. Block `batch`: the sequences' costs and the blocks' ranges.
__global__ void __launch_bounds__(256) tree_prep_kernel(const __grid_constant__ Params p) {
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  const TreeArgs& a = p.a;
  const int b = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (b < a.batch) {
    __shared__ int parent[V4KV_MAX_TREE_NODES];
    __shared__ int depth[V4KV_MAX_TREE_NODES];
    const TreeSeq s = tree_seq(a.cu_nodes, b, a.total_nodes, a.max_nodes, t == 0 ? a.dev_status : nullptr);
    if (t == 0 && a.seq_lens[b] > a.max_len) flag(a.dev_status, V4KV_DEV_OVERFLOW);
    if (t < s.n) parent[t] = tree_parent(a.parents, s.first, t, a.dev_status);
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
      p.w.anc[s.first + t] = make_uint4(m[0], m[1], m[2], m[3]);
      p.w.depth[s.first + t] = d;
      depth[t] = d;
    }
    __syncthreads();
    const int L = seq_len(a, b), pairs = min(kPairs, a.rope.rope_dim / 2);
    if (lane < pairs)
      for (int i = warp; i < s.n; i += 8) {
        float c, sn;
        rope_cs(a.rope, lane, (long long)L + depth[i], &c, &sn);
        p.w.rope[(size_t)(s.first + i) * kPairs + lane] = make_float2(c, sn);
      }
    return;
  }
  __shared__ long long csum[8];
  __shared__ int tsum[8];
  long long ccarry = 0;
  int tcarry = 0;
  for (int base = 0; base < a.batch; base += 256) {
    const int bb = base + t;
    long long cost = 0;
    int tiles = 0;
    if (bb < a.batch) {
      const SeqPlan q = plan_of(p, bb, nullptr);
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
  for (int c = t; c <= p.grid; c += 256) {
    int4 rec = make_int4(tcarry, a.batch, 0, 0);
    if (c < p.grid && ccarry > 0) {
      const long long target = (long long)c * ccarry / p.grid;
      int lo = 0, hi = a.batch - 1;  // the last sequence that begins at or before the target
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (p.w.cost[m] <= target) lo = m; else hi = m - 1;
      }
      const SeqPlan q = plan_of(p, lo, nullptr);
      const int uc = unit_cost(p, q), n = q.te + q.tr;
      const long long off = target - p.w.cost[lo];
      const int u = (int)(off / uc), k = tile_at_cost(p, q, (int)(off % uc));
      rec = make_int4(p.w.tiles[lo] + u * n + k, lo, u, k);
    }
    p.w.rec[c] = rec;
  }
}

namespace {

size_t up(size_t x) { return (x + 255) / 256 * 256; }

size_t layout(TreeWs* w, uint8_t* base, int batch, int total_nodes, int grid) {
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
  x.cost = reinterpret_cast<long long*>(take(((size_t)batch + 1) * 8));
  x.tiles = reinterpret_cast<int32_t*>(take(((size_t)batch + 1) * 4));
  x.rec = reinterpret_cast<int4*>(take(((size_t)grid + 1) * sizeof(int4)));
  x.part_o = reinterpret_cast<float*>(take((size_t)grid * 2 * kR * kD * 4));
  x.part_ml = reinterpret_cast<float2*>(take((size_t)grid * 2 * kR * sizeof(float2)));
  if (w) *w = x;
  return at;
}

}  // namespace

size_t tree_workspace_bytes(int batch, int, int total_nodes, int, int num_sms) {
  return layout(nullptr, nullptr, batch, total_nodes, num_sms);
}

cudaError_t launch_tree_attention(const TreeArgs& a, void* workspace, int num_sms, cudaStream_t stream) {
  Params p{};
  p.a = a;
  p.grid = num_sms;
  p.per_node = a.topk != nullptr || a.heads % kR == 0;
  p.hc = (a.heads + kR - 1) / kR;
  layout(&p.w, static_cast<uint8_t*>(workspace), a.batch, a.total_nodes, p.grid);
  cudaError_t e = cudaFuncSetAttribute(tree_attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_prep_kernel, dim3(a.batch + 1), dim3(256), 0, stream, p);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_attend_kernel, dim3(p.grid), dim3(kThreads), kSmemBytes, stream, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(tree_merge_kernel, dim3(p.grid, kR / 8), dim3(256), 0, stream, p);
}

}  // namespace v4kv
