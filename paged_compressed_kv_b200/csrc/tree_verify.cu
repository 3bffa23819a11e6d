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
// Bound: one row of p (and of q, where a draft was refused) per sequence, 4
// bytes a value, from HBM: 5 us for 33 MB. In fact the chain of a sequence: the
// launch, the walk, a row's fetch and its exchange between blocks, once for each
// refused draft that has a sibling and once for the draw. Measured in calls in a row
// (and as graph replays): 10.7 us (7.8) for one chain of 5 nodes and 32001 values, 28 us
// (28) for 32 trees and 131072 values, 17 us (15.5) for 64 trees of guesses; bf16
// probabilities take as long. A cluster of 8 blocks takes each sequence, an eighth of
// the vocabulary each, so that a single sequence's row is fetched by 8 SMs at once,
// all of a warp's loads in flight together; the partial sums cross through
// distributed shared memory. Sums are fp64: with 10^5 values whose prefix sum is
// compared with a given number, fp32 sums would change the drawn token for about
// one draw in a hundred.
#include <cooperative_groups.h>

#include "tc.cuh"
#include "tree.cuh"

namespace cg = cooperative_groups;

namespace v4kv {

namespace {

constexpr int kCluster = 8;          // blocks per sequence at most
constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;

__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(uint16_t x) { return bf16_bits_to_float(x); }

// four values from an address aligned to four of them
__device__ __forceinline__ float4 four_at(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 four_at(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}

// What is left of a row: r = max(p - C q, 0), less the refused guesses. Values
// that are not positive count as 0. `head` values come before the first group
// of four that is aligned, `groups` such groups follow, then the row's last
// values.
template <typename T>
struct Row {
  const T *p, *q;  // q null: r = p
  int vocab, head, groups;
  double C;
  const int* gone;
  int n_gone;

  __device__ __forceinline__ double left(float pv, float qv, bool with_q) const {
    double x = (double)fmaxf(pv, 0.f);
    if (with_q) {
      x = fma(-C, (double)fmaxf(qv, 0.f), x);
      if (__double2hiint(x) < 0) x = 0.0;
    }
    return x;
  }
  __device__ __forceinline__ bool is_gone(int e) const {
    bool hit = false;
    for (int i = 0; i < n_gone; ++i) hit |= gone[i] == e;
    return hit;
  }
  __device__ __forceinline__ double at(int e) const {
    return is_gone(e) ? 0.0 : left(value_of(p[e]), q ? value_of(q[e]) : 0.f, q != nullptr);
  }
  __device__ __forceinline__ void group(int g, const float4& pv, const float4& qv, double* w, bool with_q) const {
    w[0] = left(pv.x, qv.x, with_q);
    w[1] = left(pv.y, qv.y, with_q);
    w[2] = left(pv.z, qv.z, with_q);
    w[3] = left(pv.w, qv.w, with_q);
    for (int i = 0; i < n_gone; ++i) {
      const int d = gone[i] - head - 4 * g;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (d == k) w[k] = 0.0;
    }
  }
  __device__ __forceinline__ double group_sum(int g, const float4& pv, const float4& qv, bool with_q) const {
    double w[4];
    group(g, pv, qv, w, with_q);
    return (w[0] + w[1]) + (w[2] + w[3]);
  }
};

constexpr int kFlight = 4;  // groups a lane has in flight

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct VerifyShared {
  double part[2][kCluster];   // the blocks' sums (each block writes its slot in all blocks)
  double warp_part[kVWarps];
  double sub_part[kVWarps];   // of the run that the draw falls in
  float p[V4KV_MAX_TREE_NODES], q[V4KV_MAX_TREE_NODES], u[V4KV_MAX_TREE_NODES];
  int parent[V4KV_MAX_TREE_NODES], token[V4KV_MAX_TREE_NODES];
  int gone[V4KV_MAX_TREE_NODES];
  short path[V4KV_MAX_TREE_NODES];
  // the walk's state, written by thread 0
  int now, next_child, n_path, n_gone, task;
  double R, C;
};

enum { kSumRow = 0, kDraw = 1 };

// The cluster barrier in two halves: a block's shared memory may be written from
// another one only once it is known to run, which every block says at entry and
// asks before its first such write, with the walk in between.
__device__ __forceinline__ void cluster_here() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_all_here() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

}  // namespace

// A cluster of blocks per sequence, grid (blocks x batch). The code is kept short
// (loops, one type per instance): a launch runs it once, and fetching it is a good
// part of a small call.
template <typename T>
__global__ void __launch_bounds__(kVThreads, 2)
    tree_verify_kernel(VerifyArgs a) {
  __shared__ VerifyShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), b = blockIdx.x / nc;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster_here();
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  int32_t* st = rank == 0 ? a.dev_status : nullptr;
  const TreeSeq s = tree_seq(a.cu_nodes, b, a.total_nodes, a.max_nodes, tid == 0 ? st : nullptr);
  if (s.n <= 0) {  // the whole cluster leaves
    cluster_all_here();
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
      p = value_of(static_cast<const T*>(a.target)[at]);
      if (a.draft) q = value_of(static_cast<const T*>(a.draft)[at]);
    }
    sh.parent[tid] = ok ? parent : -1;  // a child that cannot be accepted is never asked
    sh.token[tid] = x;
    sh.p[tid] = p;
    sh.q[tid] = fmaxf(q, 0.f);  // NaN too
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
    const size_t at = (size_t)(s.first + sh.now) * a.row_stride;
    Row<T> r;
    r.p = static_cast<const T*>(a.target) + at;
    r.q = a.draft && sh.C != 0.0 ? static_cast<const T*>(a.draft) + at : nullptr;  // nothing was refused: r = p
    r.vocab = a.vocab;
    r.head = min(a.vocab, (int)((4 - (at & 3)) & 3));
    r.groups = (a.vocab - r.head) / 4;
    r.C = sh.C;
    r.gone = sh.gone;
    r.n_gone = sh.n_gone;
    const int task = sh.task;
    // each warp of the cluster takes a run of consecutive groups, the first one
    // the values before them too, the last one the values behind them
    const int run_id = rank * kVWarps + warp;
    const int per = (r.groups + nc * kVWarps - 1) / (nc * kVWarps);
    const int g0 = min(r.groups, run_id * per), g1 = min(r.groups, g0 + per);
    // the lane's odd value, if any: lanes 0 .. 2 of the first and last warps
    int odd = -1;
    if (run_id == 0 && lane < r.head) odd = lane;
    const int back = r.head + 4 * r.groups;
    if (run_id == nc * kVWarps - 1 && lane >= 4 && back + lane - 4 < r.vocab) odd = back + lane - 4;
    double total = 0.0, before = 0.0;
    int owner = 0;  // the block whose part the target falls in
    double target = 0.0;
    // the draw falls back to the whole row when nothing is left of it
    for (int attempt = 0; attempt < 2; ++attempt, ++exchange) {
      double sum = odd >= 0 ? r.at(odd) : 0.0;
      // 32 values of a lane in flight, of p alone or of p and q
      if (!r.q) {
#pragma unroll 1
        for (int g = g0 + lane; g - lane < g1; g += 64 * kFlight) {
          float4 pv[2 * kFlight];
#pragma unroll
          for (int k = 0; k < 2 * kFlight; ++k) pv[k] = four_at(r.p + r.head + 4 * (size_t)min(g + 32 * k, g1 - 1));
#pragma unroll
          for (int k = 0; k < 2 * kFlight; ++k)
            if (g + 32 * k < g1) sum += r.group_sum(g + 32 * k, pv[k], pv[k], false);
        }
      } else {
#pragma unroll 1
        for (int g = g0 + lane; g - lane < g1; g += 32 * kFlight) {
          float4 pv[kFlight], qv[kFlight];
#pragma unroll
          for (int k = 0; k < kFlight; ++k) pv[k] = four_at(r.p + r.head + 4 * (size_t)min(g + 32 * k, g1 - 1));
#pragma unroll
          for (int k = 0; k < kFlight; ++k) qv[k] = four_at(r.q + r.head + 4 * (size_t)min(g + 32 * k, g1 - 1));
#pragma unroll
          for (int k = 0; k < kFlight; ++k)
            if (g + 32 * k < g1) sum += r.group_sum(g + 32 * k, pv[k], qv[k], true);
        }
      }
      sum = warp_sum_d(sum);
      if (lane == 0) sh.warp_part[warp] = sum;
      __syncthreads();
      if (exchange == 0) cluster_all_here();
      // Two tables in turn: a block writes a table again two exchanges later,
      // behind a barrier that every block reached after reading it.
      double* part = sh.part[exchange & 1];
      if (tid < nc) {
        double t = 0.0;
        for (int w = 0; w < kVWarps; ++w) t += sh.warp_part[w];
        *cluster.map_shared_rank(part + rank, tid) = t;
      }
      cluster.sync();
      total = 0.0;
      for (int k = 0; k < nc; ++k) total += part[k];
      target = __dmul_rn((double)a.sample_u[b], total);
      double run = 0.0;
      owner = -1;
      for (int k = 0; k < nc && (owner < 0 || run <= target); ++k) {
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
      r.q = nullptr;
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
      // Each warp sums a part of the run again, and the draw goes on in the part that
      // the target falls in: in one warp's hands a run takes up to 16 steps (64
      // sequences of 131072 values 22.3 us, 15.5 so; 7.3 and 7.8 for one of 32001).
      const int own_id = rank * kVWarps + w_own;
      const int o0 = min(r.groups, own_id * per), o1 = min(r.groups, o0 + per);
      const int sub = (o1 - o0 + kVWarps - 1) / kVWarps;
      const int s0 = min(o1, o0 + warp * sub), s1 = min(o1, s0 + sub);
      const bool head = own_id == 0 && warp == 0, tail = own_id == nc * kVWarps - 1 && warp == kVWarps - 1;
      odd = head && lane < r.head ? lane : tail && lane >= 4 && back + lane - 4 < r.vocab ? back + lane - 4 : -1;
      double sum = odd >= 0 ? r.at(odd) : 0.0;
#pragma unroll 1
      for (int g = s0 + lane; g < s1; g += 32) {
        const float4 pv = four_at(r.p + r.head + 4 * (size_t)g);
        float4 qv = pv;
        if (r.q) qv = four_at(r.q + r.head + 4 * (size_t)g);
        sum += r.group_sum(g, pv, qv, r.q != nullptr);
      }
      sum = warp_sum_d(sum);
      if (lane == 0) sh.sub_part[warp] = sum;
      __syncthreads();
      int w_sub = -1;
      run = start;
      for (int w = 0; w < kVWarps && (w_sub < 0 || run <= target); ++w) {
        if (sh.sub_part[w] > 0.0) {
          w_sub = w;
          start = run;
        }
        run += sh.sub_part[w];
      }
      if (warp == w_sub) {
        // 32 groups at a time: their prefix sums over the lanes, then the group
        // that ends above the target. The row's first values come before the
        // first step, its last ones after the last.
        int found = -1, last = -1;
        run = start;
        const int steps = (s1 - s0 + 31) / 32;
        float4 pn = make_float4(0.f, 0.f, 0.f, 0.f), qn = pn;
        auto fetch = [&](int i) {
          if (i < 0 || i >= steps) return;
          const size_t e = r.head + 4 * (size_t)min(s0 + 32 * i + lane, s1 - 1);
          pn = four_at(r.p + e);
          if (r.q) qn = four_at(r.q + e);
        };
        fetch(0);
#pragma unroll 1
        for (int i = head ? -1 : 0; i < steps + tail && found < 0; ++i) {
          const int g = s0 + 32 * i + lane;
          const bool inner = i >= 0 && i < steps;
          const bool mine = inner ? g < s1 : odd >= 0 && (odd < r.head) == (i < 0);
          const int first = inner ? r.head + 4 * g : odd;
          double w[4] = {0.0, 0.0, 0.0, 0.0};
          if (inner) {
            r.group(g, pn, qn, w, r.q != nullptr);
            fetch(i + 1);
          } else if (mine) {
            w[0] = r.at(odd);
          }
          const double own = mine ? (w[0] + w[1]) + (w[2] + w[3]) : 0.0;
          double incl = own;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          const unsigned any = __ballot_sync(0xffffffffu, own > 0.0);
          const unsigned over = __ballot_sync(0xffffffffu, own > 0.0 && run + incl > target);
          if (any) {
            // the first lane that ends above the target, else the last with a value
            const int at_lane = over ? __ffs(over) - 1 : 31 - __clz(any);
            double pre = run + (incl - own);
            int pick = -1, pos = -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              pre += w[k];
              if (w[k] > 0.0) {
                pos = first + k;
                if (pick < 0 && pre > target) pick = pos;
              }
            }
            last = __shfl_sync(0xffffffffu, pos, at_lane);
            if (over) found = __shfl_sync(0xffffffffu, pick >= 0 ? pick : pos, at_lane);
          }
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
// counts of the sequences before its own itself, which saves a launch: 4.2 us in a
// graph (9.3 as a call) for one sequence as for 128.
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

// Blocks per sequence: 8 while the batch then fits the GPU at two blocks per SM
// (one sequence's row is fetched by 8 SMs), 4 or 2 for larger ones, so that one
// wave does. 64 sequences, 131072 values: 25.0 us at 8 blocks (two waves),
// 16 us at 4.
cudaError_t launch_tree_verify(const VerifyArgs& a, int num_sms, cudaStream_t stream) {
  int nc = kCluster;
  while (nc > 2 && (long long)a.batch * nc > 2LL * num_sms) nc /= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)a.batch * nc);
  cfg.blockDim = dim3(kVThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nc;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, a.target_dtype == V4KV_FP32 ? tree_verify_kernel<float> : tree_verify_kernel<uint16_t>,
                            a);
}

cudaError_t launch_tree_gather(const GatherArgs& a, cudaStream_t stream) {
  return launch_pdl(tree_gather_kernel, dim3(a.batch, (a.max_nodes + kGWarps - 1) / kGWarps),
                    dim3(kGWarps * 32), 0, stream, a);
}

}  // namespace v4kv
