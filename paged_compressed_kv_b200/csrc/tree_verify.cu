// Verification of drafted tokens and the packing of the accepted rows.
//
// v4kv_tree_verify. Walking from the root, the children of the last accepted
// node are asked in index order. What is left of the target's row p after c
// refusals is r = max(p - C q, 0) with C = R_0 + .. + R_(c-1), R_0 = 1 and
// R_c = sum(r): clamping commutes with further subtraction, so one running
// factor C replaces the c stored vectors. A refused guess (no draft) only
// removes its token. So a row is read as a whole only where a draft was
// refused and another child is still to be asked (R is needed), and once at
// the node where the path ends (the next token's draw); every accept test
// reads one value of p and q, all of them fetched up front.
//
// Bound: one row of p (and q) per sequence, 4 bytes a value, from HBM; for few
// sequences the latency of the walk and of the exchange between blocks. A
// cluster of 8 blocks takes each sequence, an eighth of the vocabulary each,
// so that a single sequence's row is fetched by 8 SMs at once; the partial
// sums cross through distributed shared memory. Sums are fp64: with 10^5
// values whose prefix sum is compared with a given number, fp32 sums would
// change the drawn token for about one draw in a hundred.
#include <cooperative_groups.h>

#include "tc.cuh"
#include "tree.cuh"

namespace cg = cooperative_groups;

namespace v4kv {

namespace {

constexpr int kCluster = 8;          // blocks per sequence
constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;

__device__ __forceinline__ float value_at(const void* base, int dtype, size_t i) {
  return dtype == V4KV_FP32 ? static_cast<const float*>(base)[i]
                            : bf16_bits_to_float(static_cast<const uint16_t*>(base)[i]);
}

// four consecutive values from a 16-byte (fp32) or 8-byte (bf16) aligned address
__device__ __forceinline__ float4 value4_at(const void* base, int dtype, size_t i) {
  if (dtype == V4KV_FP32) return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}

// One row as a sequence of groups of four values; the first group may begin
// before the row (`lead` values of it belong to the row above), so that every
// group is aligned whatever the row's offset.
struct Row {
  const void *p, *q;      // bases of the arrays (q null: no draft)
  int pt, qt;             // types
  size_t at;              // element offset of the row
  int lead, vocab, groups;
  size_t limit;           // elements of the arrays (groups reaching past it load singly)
  double C;               // r = max(p - C q, 0)
  const int* gone;        // without a draft: refused tokens
  int n_gone;
};

__device__ __forceinline__ void group_weights(const Row& r, int g, double* w) {
  const long long e0 = 4LL * g - r.lead;  // row index of the group's first value
  float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
  if (e0 >= 0 && r.at + e0 + 4 <= r.limit) {
    const float4 a = value4_at(r.p, r.pt, r.at + e0);
    p[0] = a.x; p[1] = a.y; p[2] = a.z; p[3] = a.w;
    if (r.q) {
      const float4 b = value4_at(r.q, r.qt, r.at + e0);
      q[0] = b.x; q[1] = b.y; q[2] = b.z; q[3] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = e0 + i >= 0 && e0 + i < r.vocab;
      p[i] = in ? value_at(r.p, r.pt, r.at + e0 + i) : 0.f;
      if (r.q && in) q[i] = value_at(r.q, r.qt, r.at + e0 + i);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double x = r.q ? __dsub_rn((double)p[i], __dmul_rn(r.C, (double)q[i])) : (double)p[i];
    w[i] = (e0 + i >= 0 && e0 + i < r.vocab && x > 0.0) ? x : 0.0;
  }
  for (int k = 0; k < r.n_gone; ++k) {
    const long long d = r.gone[k] - e0;
    if (d >= 0 && d < 4) w[d] = 0.0;
  }
}

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct VerifyShared {
  double part[2][kCluster];   // the blocks' sums (each block writes its slot in all blocks)
  double warp_part[kVWarps];
  float p[V4KV_MAX_TREE_NODES], q[V4KV_MAX_TREE_NODES], u[V4KV_MAX_TREE_NODES];
  int parent[V4KV_MAX_TREE_NODES], token[V4KV_MAX_TREE_NODES];
  int gone[V4KV_MAX_TREE_NODES];
  short path[V4KV_MAX_TREE_NODES];
  // the walk's state, written by thread 0
  int now, next_child, n_path, n_gone, task;
  double R, C;
};

enum { kSumRow = 0, kDraw = 1 };

}  // namespace

// grid (kCluster * batch), clusters of kCluster blocks
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kVThreads)
    tree_verify_kernel(VerifyArgs a) {
  __shared__ VerifyShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x % kCluster, b = blockIdx.x / kCluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  int32_t* st = rank == 0 ? a.dev_status : nullptr;
  const TreeSeq s = tree_seq(a.cu_nodes, b, a.total_nodes, a.max_nodes, tid == 0 ? st : nullptr);
  if (s.n <= 0) {  // the whole cluster leaves
    if (rank == 0) {
      for (int i = tid; i < a.max_nodes; i += kVThreads) a.path_out[(size_t)b * a.max_nodes + i] = -1;
      if (tid == 0) {
        a.n_path_out[b] = 0;
        a.next_token[b] = -1;
      }
    }
    return;
  }
  if (tid < s.n) {
    int parent = tree_parent(a.parents, s.first, tid, st);
    const int x = a.tokens[s.first + tid];
    const bool ok = x >= 0 && x < a.vocab;
    if (!ok && tid > 0) flag(st, V4KV_DEV_BAD_INDEX);
    float p = 0.f, q = 1.f;
    if (parent >= 0 && ok) {
      const size_t at = (size_t)(s.first + parent) * a.row_stride + x;
      p = value_at(a.target, a.target_dtype, at);
      if (a.draft) q = value_at(a.draft, a.draft_dtype, at);
    }
    sh.parent[tid] = ok ? parent : -1;  // a child that cannot be accepted is never asked
    sh.token[tid] = x;
    sh.p[tid] = p;
    sh.q[tid] = q;
    sh.u[tid] = a.accept_u[s.first + tid];
  }
  if (tid == 0) {
    sh.now = 0;
    sh.next_child = 1;
    sh.n_path = 1;
    sh.n_gone = 0;
    sh.path[0] = 0;
    sh.R = 1.0;
    sh.C = 0.0;
  }
  __syncthreads();

  for (int exchange = 0;;) {
    // thread 0 of every block makes the same walk until a row is needed
    if (tid == 0) {
      int now = sh.now, c = sh.next_child, n_gone = sh.n_gone, task = kDraw;
      double R = sh.R, C = sh.C;
      bool stop = false;
      while (!stop) {
        while (c < s.n && sh.parent[c] != now) ++c;
        if (c >= s.n) break;  // no child is left: draw the next token
        double have = __dsub_rn((double)sh.p[c], a.draft ? __dmul_rn(C, (double)sh.q[c]) : 0.0);
        if (!(have > 0.0)) have = 0.0;
        for (int k = 0; k < n_gone; ++k)
          if (sh.gone[k] == sh.token[c]) have = 0.0;
        const double need = __dmul_rn(__dmul_rn((double)sh.u[c], (double)sh.q[c]), R);
        if (need < have) {
          now = c;
          sh.path[sh.n_path++] = (short)c;
          R = 1.0;
          C = 0.0;
          n_gone = 0;
        } else if (a.draft) {
          C = __dadd_rn(C, R);
          // R is needed only if another child is to be asked
          int d = c + 1;
          while (d < s.n && sh.parent[d] != now) ++d;
          if (d < s.n) {
            task = kSumRow;
            stop = true;
          }
        } else {
          R = __dsub_rn(R, have);
          sh.gone[n_gone++] = sh.token[c];
        }
        ++c;
      }
      sh.now = now;
      sh.next_child = c;
      sh.n_gone = n_gone;
      sh.R = R;
      sh.C = C;
      sh.task = task;
    }
    __syncthreads();
    Row r;
    r.p = a.target;
    r.q = a.draft;
    r.pt = a.target_dtype;
    r.qt = a.draft_dtype;
    r.at = (size_t)(s.first + sh.now) * a.row_stride;
    r.lead = (int)(r.at & 3);
    r.vocab = a.vocab;
    r.groups = (a.vocab + r.lead + 3) / 4;
    r.limit = (size_t)(a.total_nodes - 1) * a.row_stride + a.vocab;
    r.C = sh.C;
    r.gone = sh.gone;
    r.n_gone = sh.n_gone;
    const int task = sh.task;
    // each warp of the cluster takes a run of consecutive groups
    const int per = (r.groups + kCluster * kVWarps - 1) / (kCluster * kVWarps);
    const int g0 = min(r.groups, (rank * kVWarps + warp) * per), g1 = min(r.groups, g0 + per);
    double total = 0.0, before = 0.0;
    int owner = 0;  // the block whose part the target falls in
    double target = 0.0;
    // the draw falls back to the whole row when nothing is left of it
    for (int attempt = 0; attempt < 2; ++attempt, ++exchange) {
      double sum = 0.0;
#pragma unroll 4
      for (int g = g0 + lane; g < g1; g += 32) {
        double w[4];
        group_weights(r, g, w);
        sum += (w[0] + w[1]) + (w[2] + w[3]);
      }
      sum = warp_sum_d(sum);
      if (lane == 0) sh.warp_part[warp] = sum;
      __syncthreads();
      // Two tables in turn: a block writes a table again two exchanges later,
      // behind a barrier that every block reached after reading it.
      double* part = sh.part[exchange & 1];
      if (tid < kCluster) {
        double t = 0.0;
        for (int w = 0; w < kVWarps; ++w) t += sh.warp_part[w];
        *cluster.map_shared_rank(part + rank, tid) = t;
      }
      cluster.sync();
      total = 0.0;
      for (int k = 0; k < kCluster; ++k) total += part[k];
      target = __dmul_rn((double)a.sample_u[b], total);
      double run = 0.0;
      owner = -1;
      for (int k = 0; k < kCluster && (owner < 0 || run <= target); ++k) {
        // the first part that ends above the target; rounding may put the
        // target at the total, then the last part with a positive value
        if (part[k] > 0.0) {
          owner = k;
          before = run;
        }
        run += part[k];
      }
      if (task == kSumRow || total > 0.0 || (r.C == 0.0 && r.n_gone == 0)) break;
      r.C = 0.0;
      r.n_gone = 0;
    }
    if (task == kSumRow) {
      ++exchange;
      if (tid == 0) sh.R = total;
      continue;
    }
    // the draw: the first value whose prefix sum exceeds the target
    const bool fine = total > 0.0 && isfinite(total);
    if (fine && rank == owner) {
      int w_own = -1;
      double start = before, run = before;
      for (int w = 0; w < kVWarps && (w_own < 0 || run <= target); ++w) {
        if (sh.warp_part[w] > 0.0) {
          w_own = w;
          start = run;
        }
        run += sh.warp_part[w];
      }
      if (warp == w_own) {
        int found = -1, last = -1;
        run = start;
        for (int g = g0; g < g1 && found < 0; g += 32) {
          double w[4] = {0.0, 0.0, 0.0, 0.0};
          if (g + lane < g1) group_weights(r, g + lane, w);
          const double own = (w[0] + w[1]) + (w[2] + w[3]);
          double incl = own;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          double pre = run + (incl - own);
          int pick = -1, pos = -1;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            pre += w[i];
            if (w[i] > 0.0) {
              pos = 4 * (g + lane) - r.lead + i;
              if (pick < 0 && pre > target) pick = pos;
            }
          }
          const unsigned hit = __ballot_sync(0xffffffffu, pick >= 0);
          if (hit) found = __shfl_sync(0xffffffffu, pick, __ffs(hit) - 1);
          const unsigned any = __ballot_sync(0xffffffffu, pos >= 0);
          if (any) last = __shfl_sync(0xffffffffu, pos, 31 - __clz(any));
          run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) a.next_token[b] = found >= 0 ? found : last;
      }
    }
    if (rank == 0) {
      const int n = sh.n_path;
      for (int i = tid; i < a.max_nodes; i += kVThreads)
        a.path_out[(size_t)b * a.max_nodes + i] = i < n ? sh.path[i] : -1;
      if (tid == 0) {
        a.n_path_out[b] = n;
        if (!fine) {
          a.next_token[b] = -1;
          flag(st, V4KV_DEV_BAD_PROB);
        }
      }
    }
    return;
  }
}

// v4kv_tree_gather. grid (batch, ceil(max_nodes / kGWarps)), a warp per path
// position: the accepted rows are a few KB each, so the kernel is one launch
// latency plus one chain of loads (path index, row). Every block sums the
// counts of the sequences before its own itself, which saves a launch.
namespace {
constexpr int kGWarps = 8;
}

__global__ void __launch_bounds__(kGWarps * 32) tree_gather_kernel(GatherArgs a) {
  __shared__ int warp_part[kGWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x, i = blockIdx.y * kGWarps + warp;
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  int32_t* st = blockIdx.y == 0 ? a.dev_status : nullptr;
  auto count = [&](int k) { return min(max(a.n_path[k], 0), a.max_nodes); };
  int sum = 0;
  for (int k = tid; k < b; k += kGWarps * 32) sum += count(k);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) warp_part[warp] = sum;
  __syncthreads();
  int first = 0;
#pragma unroll
  for (int w = 0; w < kGWarps; ++w) first += warp_part[w];
  const int n = count(b);
  if (blockIdx.y == 0 && tid == 0) {
    a.cu_out[b] = min(first, a.capacity);
    if (b == a.batch - 1) a.cu_out[a.batch] = min(first + n, a.capacity);
    if (n != a.n_path[b] || first + n > a.capacity) flag(st, V4KV_DEV_OVERFLOW);
  }
  if (i >= n || first + i >= a.capacity) return;
  const TreeSeq s = tree_seq(a.cu_nodes, b, a.total_nodes, a.max_nodes, lane == 0 ? a.dev_status : nullptr);
  const int node = a.path[(size_t)b * a.max_nodes + i];
  const bool ok = node >= 0 && node < s.n;
  if (!ok && lane == 0) flag(a.dev_status, V4KV_DEV_BAD_INDEX);
  const size_t src = (size_t)s.first + (ok ? node : 0), dst = (size_t)first + i;
  const uint4* x = reinterpret_cast<const uint4*>(a.x + src * a.dim);
  uint4* xo = reinterpret_cast<uint4*>(a.x_out + dst * a.dim);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int c = lane; c < a.dim / 8; c += 32) xo[c] = ok ? x[c] : zero;
  if (a.gate_dim == 1) {
    if (lane == 0) a.gate_out[dst] = ok ? a.gate[src] : 0.f;
  } else {
    const uint4* g = reinterpret_cast<const uint4*>(a.gate + src * a.dim);
    uint4* go = reinterpret_cast<uint4*>(a.gate_out + dst * a.dim);
    for (int c = lane; c < a.dim / 4; c += 32) go[c] = ok ? g[c] : zero;
  }
}

cudaError_t launch_tree_verify(const VerifyArgs& a, cudaStream_t stream) {
  return launch_pdl(tree_verify_kernel, dim3((unsigned)a.batch * kCluster), dim3(kVThreads), 0, stream, a);
}

cudaError_t launch_tree_gather(const GatherArgs& a, cudaStream_t stream) {
  return launch_pdl(tree_gather_kernel, dim3(a.batch, (a.max_nodes + kGWarps - 1) / kGWarps),
                    dim3(kGWarps * 32), 0, stream, a);
}

}  // namespace v4kv
