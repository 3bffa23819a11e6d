// Decode attention of drafted-token trees over the paged, compressed cache.
//
// For node i of a sequence with L cached tokens, at position pos = L + depth:
//   s_hj = sm_scale q_h . v_j,  p = softmax_j(s),  o_h = sum_j p_hj v_j
// over the entries j < floor(max(0, pos + 1 - W) / r) (or the node's top-k),
// the cached tokens [max(0, pos + 1 - W), L) and the node's ancestors with
// itself; then the inverse RoPE at pos, and bf16.
//
// One warp per (node, head): a lane holds 16 of the 512 dims of q and of the
// running sum, the score is one warp reduction per item and the softmax keeps
// its running maximum and sum (fp32), so each item is read once per head.
#include "tree.cuh"

namespace v4kv {

namespace {

constexpr int kWarps = 8;

struct Node {
  int first, n, i, b, L, depth;
};

__device__ __forceinline__ void load_bf16(const uint16_t* p, float* v) {
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = bf16_bits_to_float(p[e]);
}

__device__ __forceinline__ void load_item(const PoolArgs& pool, size_t slot, int lane, float* v) {
  if (pool.dtype == V4KV_FP8_E4M3) {
    const uint8_t* p = static_cast<const uint8_t*>(pool.data) + slot * 512 + 16 * lane;
    const float s = pool.scales[slot];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = e4m3_to_float(p[e]) * s;
  } else {
    load_bf16(static_cast<const uint16_t*>(pool.data) + slot * 512 + 16 * lane, v);
  }
}

}  // namespace

__global__ void __launch_bounds__(kWarps * 32) tree_attend_kernel(TreeArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x;  // node
  __shared__ Node node_sh;
  if (threadIdx.x == 0) {
    // the last sequence that begins at or before the row
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (a.cu_nodes[m] <= row) lo = m; else hi = m - 1;
    }
    const TreeSeq s = tree_seq(a.cu_nodes, lo, a.total_nodes, a.max_nodes, a.dev_status);
    Node nd;
    nd.first = s.first;
    nd.n = s.n;
    nd.b = lo;
    nd.i = row - s.first;
    int L = a.seq_lens[lo];
    if (L > a.max_len) {
      flag(a.dev_status, V4KV_DEV_OVERFLOW);
      L = a.max_len;
    }
    nd.L = max(0, L);
    nd.depth = -1;
    if (nd.i >= 0 && nd.i < nd.n)
      for (int p = nd.i; p >= 0; p = tree_parent(a.parents, nd.first, p, a.dev_status)) ++nd.depth;
    node_sh = nd;
  }
  __syncthreads();
  const Node nd = node_sh;
  const int h = blockIdx.y * kWarps + warp;
  if (nd.depth < 0 || h >= a.heads) return;
  float q[16], o[16], v[16];
  const size_t at = ((size_t)row * a.heads + h) * 512 + 16 * lane;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    q[e] = (a.q_dtype == V4KV_FP32 ? static_cast<const float*>(a.q)[at + e]
                                   : bf16_bits_to_float(static_cast<const uint16_t*>(a.q)[at + e])) *
           a.sm_scale * 1.4426950408889634f;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  auto item = [&]() {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) s = fmaf(q[e], v[e], s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), c = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = fmaf(l, c, p);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = fmaf(o[e], c, p * v[e]);
  };
  const long long end = (long long)nd.L + nd.depth + 1;
  const int w0 = (int)max(0LL, end - a.window_len);
  const int n_sel = a.topk ? a.k : w0 / a.ratio;
  const int stored = (nd.L + a.ratio - 1) / a.ratio;
  for (int it = 0; it < n_sel; ++it) {
    const int j = a.topk ? a.topk[(size_t)row * a.k + it] : it;
    if (j < 0) continue;
    if (j >= stored) {
      flag(a.dev_status, V4KV_DEV_BAD_INDEX);
      continue;
    }
    const int pg = page_of(a.main.block_table + (size_t)nd.b * a.main.max_blocks, a.main.max_blocks, j,
                           a.main.spb, a.main.num_pages, a.dev_status);
    if (pg < 0) continue;
    load_item(a.main, (size_t)pg * a.main.spb + j % a.main.spb, lane, v);
    item();
  }
  for (int t = min(w0, nd.L); t < nd.L; ++t) {
    const int pg = page_of(a.window.block_table + (size_t)nd.b * a.window.max_blocks, a.window.max_blocks,
                           t, a.window.spb, a.window.num_pages, a.dev_status);
    if (pg < 0) continue;
    load_item(a.window, (size_t)pg * a.window.spb + t % a.window.spb, lane, v);
    item();
  }
  for (int p = nd.i; p >= 0; p = tree_parent(a.parents, nd.first, p, a.dev_status)) {
    load_bf16(a.k_tree + (size_t)(nd.first + p) * 512 + 16 * lane, v);
    item();
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const int d = 16 * lane + e - a.rope.rope_offset;
    float x = o[e] * inv, y = o[e + 1] * inv;
    if (d >= 0 && d + 1 < a.rope.rope_dim) {
      float c, s;
      rope_cs(a.rope, d >> 1, end - 1, &c, &s);
      rope_apply(x, y, c, -s);
    }
    a.out[at + e] = float_to_bf16_bits(x);
    a.out[at + e + 1] = float_to_bf16_bits(y);
  }
}

size_t tree_workspace_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_tree_attention(const TreeArgs& a, void*, int, cudaStream_t stream) {
  tree_attend_kernel<<<dim3(a.total_nodes, (a.heads + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace v4kv
