// Attention of blocks of queries over the paged INT2 cache: drafted trees, causal
// chunks (kvq_tree_attention) and cross attention (kvq_cross_attention).
//
//   q'_j = q_j R_K,h(j);   a_s = q'_j . (z_s + s_s c_s) / sqrt(128)   over the visible positions s
//   p = softmax(a);        o_rot = sum_s p_s (z_s + s_s c_s)          (rotated-V basis)
//
// Visibility.  A tree's nodes are numbered in preorder: tin(i), with size(i) nodes
// in the subtree of i.  a is i or an ancestor of i exactly when
// tin(a) <= tin(i) < tin(a) + size(a), one unsigned comparison whatever the tree's
// depth.  A chain (causal chunk) is tin(i) = i, size(i) = n - i.
//
// Launches: qb_tree_kernel (trees only) numbers the nodes, qb_rotate_kernel rotates
// the queries into the workspace (base-2 logits: scaled by log2(e) / sqrt(128)),
// qb_attend_kernel takes one warp per query row.
#include "kvq_internal.cuh"

namespace kvq {

constexpr float QB_SCALE = 0.12751742902274214f;  // log2(e) / sqrt(128)

struct QbWs {
  float* q;    // [n_total][n_q_heads][128] rotated, scaled queries
  int2* tree;  // [n_total] (tin, size)
};

static size_t qb_align(size_t x) { return (x + 255) & ~size_t(255); }

static size_t qb_layout(void* base, int n_total, int n_q_heads, QbWs* out) {
  const size_t o_q = 0, o_tree = qb_align((size_t)n_total * n_q_heads * D * sizeof(float));
  const size_t total = qb_align(o_tree + (size_t)n_total * sizeof(int2));
  if (out) {
    out->q = reinterpret_cast<float*>(static_cast<char*>(base) + o_q);
    out->tree = reinterpret_cast<int2*>(static_cast<char*>(base) + o_tree);
  }
  return total;
}

size_t query_block_workspace_bytes(int n_seqs, int n_q_heads, int n_kv_heads, int n_total, int max_q, int max_len) {
  return qb_layout(nullptr, n_total, n_q_heads, nullptr);
}

// A sequence's queries [c0, c0 + n) and cached length, checked; n = 0 where they are inconsistent.
struct QbSeq {
  int c0, n, len;
};
__device__ __forceinline__ QbSeq qb_seq(int b, const int32_t* cu_q, const int32_t* lens, int n_total, int max_q,
                                        int max_len, int mode, unsigned* err) {
  QbSeq q;
  q.c0 = cu_q[b];
  const int end = cu_q[b + 1];
  q.len = lens[b];
  q.n = end - q.c0;
  if (q.c0 < 0 || end < q.c0 || end > n_total || q.n > max_q || q.len < 0 || q.len > max_len ||
      (mode != QB_CROSS && q.n > q.len)) {
    flag_error(err, ERR_SEQ_RANGE);
    q.n = 0;
    q.len = 0;
  }
  return q;
}

__global__ void __launch_bounds__(256)
qb_tree_kernel(const int32_t* __restrict__ cu_q, const int32_t* __restrict__ lens, const int32_t* __restrict__ parents,
               int n_total, int max_q, int max_len, int2* __restrict__ tree, unsigned* err) {
  __shared__ int s_par[QB_MAX_TREE], s_size[QB_MAX_TREE], s_off[QB_MAX_TREE];
  const QbSeq q = qb_seq(blockIdx.x, cu_q, lens, n_total, max_q, max_len, QB_TREE, err);
  for (int i = threadIdx.x; i < q.n; i += blockDim.x) {
    int p = parents[q.c0 + i];
    if (p < -1 || p >= i) {
      flag_error(err, ERR_TREE);
      p = -1;
    }
    s_par[i] = p;
    s_size[i] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < q.n; i += blockDim.x)
    for (int j = i; j >= 0; j = s_par[j]) atomicAdd(&s_size[j], 1);
  __syncthreads();
  // a node's place behind its parent: 1 + the subtrees of its earlier siblings
  for (int i = threadIdx.x; i < q.n; i += blockDim.x) {
    int off = 1;
    const int p = s_par[i];
    for (int j = p + 1; j < i; ++j) off += s_par[j] == p ? s_size[j] : 0;
    s_off[i] = off;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < q.n; i += blockDim.x) {
    int tin = -1;
    for (int j = i; j >= 0; j = s_par[j]) tin += s_off[j];
    tree[q.c0 + i] = make_int2(tin, s_size[i]);
  }
}

// One warp a row (token, query head): y = x R * scale.
__global__ void __launch_bounds__(256)
qb_rotate_kernel(long long rows, int n_q_heads, int gqa, const void* __restrict__ q, int dtype, RotDev rot,
                 float* __restrict__ out) {
  __shared__ float s_x[8][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long r = (long long)blockIdx.x * 8 + warp;
  if (r >= rows) return;
  const int h = (int)(r % n_q_heads) / gqa;
  const float4 x = load4(q, (size_t)r * D + 4 * lane, dtype);
  float y[4] = {x.x, x.y, x.z, x.w};
  if (rot.kind == KVQ_ROT_SIGNED_HADAMARD) {
    const float4 sg = *reinterpret_cast<const float4*>(rot.signs + (size_t)h * D + 4 * lane);
    y[0] *= sg.x; y[1] *= sg.y; y[2] *= sg.z; y[3] *= sg.w;
    const float a0 = y[0] + y[1], a1 = y[0] - y[1], a2 = y[2] + y[3], a3 = y[2] - y[3];
    y[0] = a0 + a2; y[1] = a1 + a3; y[2] = a0 - a2; y[3] = a1 - a3;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float o = __shfl_xor_sync(0xffffffffu, y[i], d);
        y[i] = (lane & d) ? o - y[i] : y[i] + o;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] *= 0.08838834764831845f;
  } else if (rot.kind == KVQ_ROT_DENSE) {
    *reinterpret_cast<float4*>(&s_x[warp][4 * lane]) = x;
    __syncwarp();
    y[0] = y[1] = y[2] = y[3] = 0.f;
    const float* R = rot.dense + (size_t)h * D * D;
#pragma unroll 8
    for (int c = 0; c < D; ++c) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(R + c * D + 4 * lane));
      const float v = s_x[warp][c];
      y[0] = fmaf(v, w.x, y[0]); y[1] = fmaf(v, w.y, y[1]); y[2] = fmaf(v, w.z, y[2]); y[3] = fmaf(v, w.w, y[3]);
    }
  }
  *reinterpret_cast<float4*>(out + (size_t)r * D + 4 * lane) =
      make_float4(y[0] * QB_SCALE, y[1] * QB_SCALE, y[2] * QB_SCALE, y[3] * QB_SCALE);
}

__global__ void __launch_bounds__(256)
qb_attend_kernel(PageGeom g, int n_q_heads, int gqa, int n_seqs, int n_total, int max_q, int max_len, int mode,
                 const int32_t* __restrict__ cu_q, const int32_t* __restrict__ lens,
                 const int32_t* __restrict__ table, const uint8_t* __restrict__ pool, QbWs ws, float* __restrict__ out,
                 unsigned* err) {
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(r / n_q_heads), j = (int)(r % n_q_heads), h = j / gqa;
  if (t >= n_total || t >= cu_q[n_seqs]) return;
  int lo = 0, hi = n_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu_q[mid] <= t) lo = mid;
    else hi = mid;
  }
  const QbSeq q = qb_seq(lo, cu_q, lens, n_total, max_q, max_len, mode, err);
  if (t < q.c0 || t >= q.c0 + q.n) return;
  const int i = t - q.c0, base = mode == QB_CROSS ? q.len : q.len - q.n;
  const int tin = mode == QB_TREE ? ws.tree[t].x : i;
  const float4 y = *reinterpret_cast<const float4*>(ws.q + (size_t)r * D + 4 * lane);
  const int P = g.page_tokens;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < q.len; ++s) {
    if (s >= base) {
      const int a = s - base;
      const int2 ta = mode == QB_TREE ? ws.tree[q.c0 + a] : make_int2(a, q.n - a);
      if ((unsigned)(tin - ta.x) >= (unsigned)ta.y) continue;
    }
    const int page = table[(size_t)lo * g.max_blocks + s / P], slot = s % P;
    if ((unsigned)page >= (unsigned)g.num_blocks) {
      flag_error(err, ERR_BLOCK_RANGE);
      continue;
    }
    const uint8_t* rec = pool + ((size_t)page * g.n_kv_heads + h) * g.record;
    const unsigned kc = rec[32 * slot + lane], vc = rec[32 * (P + slot) + lane];
    const float2 km = __half22float2(*reinterpret_cast<const __half2*>(rec + 64 * P + 4 * slot));
    const float2 vm = __half22float2(*reinterpret_cast<const __half2*>(rec + 68 * P + 4 * slot));
    float a = y.x * fmaf(km.x, (float)(kc & 3), km.y);
    a = fmaf(y.y, fmaf(km.x, (float)((kc >> 2) & 3), km.y), a);
    a = fmaf(y.z, fmaf(km.x, (float)((kc >> 4) & 3), km.y), a);
    a = fmaf(y.w, fmaf(km.x, (float)(kc >> 6), km.y), a);
#pragma unroll
    for (int d = 16; d; d >>= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
    const float mn = fmaxf(m, a);
    const float f = exp2f(m - mn), p = exp2f(a - mn);
    m = mn;
    l = fmaf(l, f, p);
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = fmaf(p, fmaf(vm.x, (float)((vc >> (2 * c)) & 3), vm.y), o[c] * f);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<float4*>(out + (size_t)r * D + 4 * lane) = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
}

cudaError_t launch_query_block(const PageGeom& g, int n_q_heads, int n_seqs, int n_total, const void* q, int dtype,
                               const int32_t* cu_q, int max_q, const int32_t* parents, int mode, const int32_t* lens,
                               int max_len, const int32_t* table, RotDev rot_k, const uint8_t* pool, void* ws_base,
                               float* o_rot, unsigned* err, cudaStream_t s) {
  QbWs ws;
  qb_layout(ws_base, n_total, n_q_heads, &ws);
  const int gqa = n_q_heads / g.n_kv_heads;
  const long long rows = (long long)n_total * n_q_heads;
  if (mode == QB_TREE) qb_tree_kernel<<<n_seqs, 256, 0, s>>>(cu_q, lens, parents, n_total, max_q, max_len, ws.tree, err);
  qb_rotate_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(rows, n_q_heads, gqa, q, dtype, rot_k, ws.q);
  qb_attend_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(g, n_q_heads, gqa, n_seqs, n_total, max_q, max_len, mode,
                                                              cu_q, lens, table, pool, ws, o_rot, err);
  return cudaGetLastError();
}

}  // namespace kvq
