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
// Products.  Unlike the single-token decode (bound by the page stream), a block of
// n queries does 512 n gqa flop per 72 cached bytes, and above about 40 rows a KV
// head the tensor cores are the bound.  Both products therefore run on tcgen05
// with the 2-bit codes as the A operand in tensor memory and the queries as the N
// dimension (16, 32 or 64 rows: qb_rows):
//   S^T [128 tokens x N]   = C_K [128 tokens x 128 channels] Q'^T [128 x N]
//   O^T [128 channels x N] = C_V^T [128 channels x 128 tokens] W^T [128 x N]
// The codes enter centred, c - 1.5 in fp16 (exact): with mid = z + 1.5 s
//   a_s = s (q' . (c - 1.5)) + mid sum(q'),   o = sum_s (p_s s_s)(c - 1.5) + sum_s p_s mid_s
// (uncentred codes would put a large positive sum into the accumulators that the z
// term cancels, and with it the accumulators' rounding).  The fp32 operands q' and
// w = p s enter as two fp16 halves (hi, and the remainder), 22 bits together: at 64
// rows one after the other into one accumulator, the remainders first, below that
// side by side as 2 N columns.  A row's q' is scaled by a power of two that is the
// tile's or, beside rows more than 2^16 as large, its own; the remainder of w is held
// times 2^11, so that w reaches 2^-39 of the row's largest.  Each 128-token product
// starts from zero and is added up in fp32 registers, so no long sum runs through the
// tensor cores' own rounding (readouts 3 - 5e-7 off fp64).
// Softmax weights are kept as w = 2^(a + log2 s - M) directly, p = w / s: fp16 then
// holds w whatever the value scales are (a constant group, s = 0, takes the
// smallest fp16 as s: its codes are 0 and mid compensates exactly).  M is a lazy
// reference, set from the maximum of the first tile and moved only when a weight
// would pass fp16's range: one vote a tile, and most units never move it again.
//
// A CTA (one per SM, persistent over an equal slice of all work):
//   4 + 4 warps  expand the codes of a tile into tensor memory: a thread owns a token
//                (keys) or, through a transposing load, 16 channels of a field (values)
//   2 x 4 warps  softmax: a thread owns a token, each group of four warps half of the
//                rows; weights go to shared memory as the next product's B operand
//   4 warps      add up the 128-token products, load the next unit's queries, write out
//   1 warp       page copies (cp.async.bulk) and the list of units
//   1 warp       issues the MMAs
// A unit is (sequence, KV head, row tile).  Slices cut units: a unit wholly inside a
// CTA is written out at once, a cut one leaves partials (numerator, l, M) that
// qb_combine_kernel joins in slice order (results do not depend on timing).
//
// Bound: no unit is full.  16 trees of 32 drafts on 16,384 tokens, 32 / 8 heads: 360 us
// for the call, 382 TFLOP/s of attention (0.20 of the measured cuBLAS bf16 rate, twice
// that as issued), a 64 x 128 tile in 1.6 us, the tensor pipe active 36 %, the schedulers
// issuing 60 % of the time; the largest stall is the long scoreboard (3.85 warps an
// issue).  The time is in the chain of waits from role to role; which role holds the
// others up has not been measured.  The roles run side by side from one instruction
// cache, so their common path is kept short: with the expansion loops unrolled the same
// call took 414 us (then 357), with everything unrolled 1,446 us.
#include <algorithm>
#include <cstddef>

#include "quant_common.cuh"
#include "tcgen05.cuh"

namespace kvq {

constexpr float QB_SCALE = 0.12751742902274214f;  // log2(e) / sqrt(128): base-2 logits

constexpr int QB_TOK = 128;                       // tokens a tile
constexpr int QB_STAGES = 4;
constexpr int QB_STAGE_BYTES = QB_TOK * 72;
constexpr int QB_PBUF = QB_TOK * 128;             // one half of W^T: 128 rows of 128 bytes (64 fp16 columns)
constexpr int QB_UNITS = 4;                       // ring of unit descriptors
constexpr int QB_UNIT_WORK = 3;                   // what starting and ending a unit costs, in tiles (measured: 5 us and 1.6 us)
// Weights: the running maximum is put at 2^3 (further from fp16's smallest step than at 1: with the second half unscaled,
// readout error 6.5e-7 -> 4.6e-7, the same at 2^6), and again whenever a weight would pass 2^15.5.
constexpr float QB_LIFT = 3.f, QB_TRIGGER = 15.5f;
// A weight's second half is held times 2^11: up to half a step of the largest weight (2^15), and down to 2^-36 in all.
// Unscaled, weights ended at fp16's 2^-25, 2^-28 of the largest: behind a token 16 to 22 nats above 131,071 others, the
// readout was up to 7e-4 off.
constexpr int QB_LO_SHIFT = 11;
constexpr float QB_LO_UP = 2048.f, QB_LO_DOWN = 1.f / 2048.f;

constexpr int QB_APART = INT32_MIN;               // a unit's limit of open positions where its rows are far apart in size
constexpr int QB_GROUPS = 2;                      // groups of four softmax warps, half of the rows each
// Keys (4 warps), values (4), softmax, accumulation (4), copies, MMA issue and two idle warps: register shares go by four.
constexpr int QB_THREADS = 32 * (16 + 4 * QB_GROUPS);

__host__ __device__ constexpr int qb_smem_bytes(int n) {
  return 1024 + 2 * n * 512 + 2 * 2 * QB_PBUF + QB_STAGES * QB_STAGE_BYTES + n * D * 4;
}

// ---------------------------------------------------------------------------
// Workspace and the list of tiles
// ---------------------------------------------------------------------------
struct QbWs {
  float* q;          // [n_total][n_q_heads][128] rotated, scaled queries
  int2* tree;        // [n_total] (tin, size)
  long long* work;   // [n_seqs + 1] running sum of the sequences' work (tiles, and QB_UNIT_WORK a unit)
  long long* tiles;  // [n_seqs + 1] running sum of their tiles
  int4* join;        // [grid] the unit that starts in a slice and runs past its end: (first draft's row, drafts, row tile * H + head, parts); parts 0: none
  float* part;       // [2 grid][N][130]: numerator [N][128], l [N], M [N]
};

static size_t qb_align(size_t x) { return (x + 255) & ~size_t(255); }

// Rows a tile: the smallest of 16, 32, 64 that holds a sequence's rows of one KV head, else 64 (a tile of 128 tokens
// takes 1.2 us with 16 rows and 1.6 us with 64).
static int qb_rows(int max_q, int gqa) {
  const long long r = (long long)max_q * gqa;
  return r <= 16 ? 16 : r <= 32 ? 32 : 64;
}

static size_t qb_layout(void* base, int n_seqs, int n_total, int n_q_heads, int rows, int grid, QbWs* out) {
  const size_t o_tree = qb_align((size_t)n_total * n_q_heads * D * sizeof(float));
  const size_t o_work = qb_align(o_tree + (size_t)n_total * sizeof(int2));
  const size_t o_tiles = qb_align(o_work + ((size_t)n_seqs + 1) * sizeof(long long));
  const size_t o_join = qb_align(o_tiles + ((size_t)n_seqs + 1) * sizeof(long long));
  const size_t o_part = qb_align(o_join + (size_t)grid * sizeof(int4));
  if (out) {
    char* p = static_cast<char*>(base);
    out->q = reinterpret_cast<float*>(p);
    out->tree = reinterpret_cast<int2*>(p + o_tree);
    out->work = reinterpret_cast<long long*>(p + o_work);
    out->tiles = reinterpret_cast<long long*>(p + o_tiles);
    out->join = reinterpret_cast<int4*>(p + o_join);
    out->part = reinterpret_cast<float*>(p + o_part);
  }
  return qb_align(o_part + (size_t)2 * grid * rows * (D + 2) * sizeof(float));
}

size_t query_block_workspace_bytes(int n_seqs, int n_q_heads, int n_kv_heads, int n_total, int max_q, int max_len) {
  return qb_layout(nullptr, n_seqs, n_total, n_q_heads, qb_rows(max_q, n_q_heads / n_kv_heads), device_sm_count(),
                   nullptr);
}

// A sequence's queries [c0, c0 + n) and cached length, checked; n = 0 where they are inconsistent.
struct QbSeq {
  int c0, n, len;
};

struct QbArgs {
  PageGeom g;
  int n_q_heads, gqa, n_seqs, n_total, max_q, max_len, mode;
  int gqa_shift, page_shift;  // both are powers of two
  const int32_t* cu_q;
  const int32_t* lens;
  const int32_t* table;
  const uint8_t* pool;
  QbWs ws;
  float* out;
  unsigned* err;
};

__device__ __forceinline__ QbSeq qb_seq(const QbArgs& a, int b, unsigned* err) {
  QbSeq q;
  q.c0 = a.cu_q[b];
  const int end = a.cu_q[b + 1];
  q.len = a.lens[b];
  q.n = end - q.c0;
  if (q.c0 < 0 || end < q.c0 || end > a.n_total || q.n > a.max_q || q.len < 0 || q.len > a.max_len ||
      (a.mode != QB_CROSS && q.n > q.len)) {
    flag_error(err, ERR_SEQ_RANGE);
    q.n = 0;
    q.len = 0;
  }
  return q;
}

// Tiles of a sequence.  Row tile j of a causal chunk ends with draft min(n, (j + 1) c) - 1
// (c = N / gqa drafts a row tile, a power of two) and stops there:
// ceil((base + (j + 1) c) / 128) = floor((x + j + 1) / m), m = 128 / c, x = floor((base + 127) / c),
// whose sums have a closed form; trees and cross attention read every tile for each row tile.
struct QbSpan {
  int n_rt, nt, lc, lm, x;  // row tiles; tiles of the last (chain) or of every one; log2 c, log2 m
  bool chain;
  __device__ __forceinline__ long long floor_sum(long long t) const {  // sum of floor(k / m) for k = 0 .. t
    const long long q = t >> lm;
    return ((q * (q - 1) / 2) << lm) + q * (t - (q << lm) + 1);
  }
  // tiles of the row tiles before j, one KV head
  __device__ __forceinline__ long long before(int j) const {
    return chain ? floor_sum((long long)x + j) - floor_sum(x) : (long long)nt * j;
  }
  __device__ __forceinline__ int tiles(int j) const { return chain && j + 1 < n_rt ? (x + j + 1) >> lm : nt; }
  __device__ __forceinline__ long long total() const { return n_rt ? before(n_rt - 1) + nt : 0; }
};

template <int N>
__device__ __forceinline__ QbSpan qb_span(const QbArgs& a, const QbSeq& q) {
  QbSpan s;
  s.lc = 31 - __clz(N >> a.gqa_shift);
  s.lm = 7 - s.lc;
  s.n_rt = (int)(((long long)q.n * a.gqa + N - 1) / N);
  s.nt = q.len ? (q.len + QB_TOK - 1) / QB_TOK : 1;
  s.chain = a.mode == QB_CHAIN;
  s.x = (q.len - q.n + 127) >> s.lc;
  return s;
}

// Slice k of all work: [start(k), start(k + 1)), sizes equal to within one.  A unit's work is QB_UNIT_WORK, then one per
// tile; a slice has the tiles whose work lies in it.
struct QbSlices {
  long long each;
  int more;
  __device__ __forceinline__ QbSlices(long long total, int grid)
      : each(total / grid), more((int)(total - total / grid * grid)) {}
  __device__ __forceinline__ long long start(int k) const { return k * each + min(k, more); }
};

struct QbUnit {
  int b, rt, h;
  int c0, n, len;     // the sequence
  int t0, t1, nt;     // tiles [t0, t1) of nt in this slice
};

// The running sums of the sequences' work and tiles, held by a warp.  Of up to QB_FEW sequences it takes them from the
// inputs itself (a lane a run of them), without waiting for the preparation; of more, from the workspace.
constexpr int QB_FEW = 128;

template <int N>
struct QbList {
  bool few;
  int b0, b1;               // this lane's run
  long long work0, tiles0;  // before it
  long long work, tiles;    // of all

  __device__ __forceinline__ QbList(const QbArgs& a, int lane) : few(a.n_seqs <= QB_FEW) {
    if (!few) {
      work = a.ws.work[a.n_seqs];
      tiles = a.ws.tiles[a.n_seqs];
      return;
    }
    const int per = (a.n_seqs + 31) / 32;
    b0 = min(a.n_seqs, lane * per);
    b1 = min(a.n_seqs, b0 + per);
    work = tiles = 0;
    for (int b = b0; b < b1; ++b) add(a, qb_span<N>(a, qb_seq(a, b, nullptr)), work, tiles);
    work0 = -work;
    tiles0 = -tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long w = __shfl_up_sync(0xffffffffu, work, d), t = __shfl_up_sync(0xffffffffu, tiles, d);
      if (lane >= d) {
        work += w;
        tiles += t;
      }
    }
    work0 += work;
    tiles0 += tiles;
    work = __shfl_sync(0xffffffffu, work, 31);
    tiles = __shfl_sync(0xffffffffu, tiles, 31);
  }
  static __device__ __forceinline__ void add(const QbArgs& a, const QbSpan& s, long long& work, long long& tiles) {
    work += (s.total() + (long long)QB_UNIT_WORK * s.n_rt) * a.g.n_kv_heads;
    tiles += s.total() * a.g.n_kv_heads;
  }
  // The last sequence that starts at or before w (< work), and the sums before it.
  __device__ __forceinline__ int find(const QbArgs& a, long long w, int lane, long long& at_work, long long& at_tiles) const {
    if (few) {
      const int owner = 31 - __clz(__ballot_sync(0xffffffffu, b1 > b0 && work0 <= w));
      int b = b0;
      long long bw = work0, bt = tiles0;
      if (lane == owner) {
        long long nw = bw, nt = bt;
        for (int c = b0; c < b1 && nw <= w; ++c) {
          b = c;
          bw = nw;
          bt = nt;
          add(a, qb_span<N>(a, qb_seq(a, c, nullptr)), nw, nt);
        }
      }
      at_work = __shfl_sync(0xffffffffu, bw, owner);
      at_tiles = __shfl_sync(0xffffffffu, bt, owner);
      return __shfl_sync(0xffffffffu, b, owner);
    }
    int lo = 0, cnt = a.n_seqs;
    while (cnt > 1) {
      const int step = (cnt + 31) / 32, i = lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, i < cnt && a.ws.work[lo + i] <= w);
      const int k = 31 - __clz(m);
      lo += k * step;
      cnt = min(step, cnt - k * step);
    }
    at_work = a.ws.work[lo];
    at_tiles = a.ws.tiles[lo];
    return lo;
  }
};

// The unit that holds the work at `w`, by one warp: u.t0 = the first of its tiles at or after w; `in`: w inside the unit;
// `before`: the tiles of all that come before w.
template <int N>
__device__ __forceinline__ QbUnit qb_locate(const QbArgs& a, const QbList<N>& list, long long w, int lane, int& in,
                                            long long& before) {
  long long at_work, at_tiles;
  QbUnit u;
  u.b = list.find(a, w, lane, at_work, at_tiles);
  const QbSeq q = qb_seq(a, u.b, nullptr);
  const QbSpan s = qb_span<N>(a, q);
  const int H = a.g.n_kv_heads;
  const long long rem = w - at_work;
  int j0 = 0, j1 = s.n_rt;
  while (j1 - j0 > 1) {
    const int mid = (j0 + j1) >> 1;
    if ((s.before(mid) + (long long)QB_UNIT_WORK * mid) * H <= rem) j0 = mid;
    else j1 = mid;
  }
  u.rt = j0;
  u.nt = s.tiles(j0);
  const long long rest = rem - (s.before(j0) + (long long)QB_UNIT_WORK * j0) * H;  // < (nt + QB_UNIT_WORK) H < 2^31
  const unsigned each = (unsigned)(u.nt + QB_UNIT_WORK);
  u.h = (int)((unsigned)rest / each);
  in = (int)((unsigned)rest % each);
  u.t0 = max(0, in - QB_UNIT_WORK);
  u.t1 = u.nt;
  u.c0 = q.c0;
  u.n = q.n;
  u.len = q.len;
  before = at_tiles + s.before(j0) * H + (long long)u.h * u.nt + u.t0;
  return u;
}

// The unit after u, from its first tile.
template <int N>
__device__ __forceinline__ void qb_next(const QbArgs& a, QbUnit& u) {
  QbSeq q{u.c0, u.n, u.len};
  if (++u.h == a.g.n_kv_heads) {
    u.h = 0;
    if (++u.rt >= qb_span<N>(a, q).n_rt) {
      u.rt = 0;
      do {
        if (++u.b >= a.n_seqs) {
          u.nt = 0;
          return;
        }
        q = qb_seq(a, u.b, nullptr);
      } while (q.n == 0);
      u.c0 = q.c0;
      u.n = q.n;
      u.len = q.len;
    }
  }
  u.nt = qb_span<N>(a, q).tiles(u.rt);
  u.t0 = 0;
  u.t1 = u.nt;
}

// ---------------------------------------------------------------------------
// Preparation: one launch for the list of tiles (block 0), the trees' numbering (one
// block a sequence) and the rotation of the queries.
// ---------------------------------------------------------------------------
constexpr int QB_PREP_THREADS = 256;

template <int N>
__device__ __forceinline__ void qb_list_tiles(const QbArgs& a) {
  __shared__ long long s_warp[2][QB_PREP_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (a.n_seqs + QB_PREP_THREADS - 1) / QB_PREP_THREADS;
  const int b0 = min(a.n_seqs, (int)threadIdx.x * per), b1 = min(a.n_seqs, b0 + per);
  long long work = 0, tiles = 0;
  for (int b = b0; b < b1; ++b) {
    QbList<N>::add(a, qb_span<N>(a, qb_seq(a, b, a.err)), work, tiles);
  }
  long long inc_w = work, inc_t = tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long w = __shfl_up_sync(0xffffffffu, inc_w, d), t = __shfl_up_sync(0xffffffffu, inc_t, d);
    if (lane >= d) {
      inc_w += w;
      inc_t += t;
    }
  }
  if (lane == 31) {
    s_warp[0][warp] = inc_w;
    s_warp[1][warp] = inc_t;
  }
  __syncthreads();
  long long at_w = inc_w - work, at_t = inc_t - tiles;
  for (int w = 0; w < warp; ++w) {
    at_w += s_warp[0][w];
    at_t += s_warp[1][w];
  }
  for (int b = b0; b < b1; ++b) {
    a.ws.work[b] = at_w;
    a.ws.tiles[b] = at_t;
    QbList<N>::add(a, qb_span<N>(a, qb_seq(a, b, nullptr)), at_w, at_t);
  }
  if (threadIdx.x == QB_PREP_THREADS - 1) {
    a.ws.work[a.n_seqs] = at_w;
    a.ws.tiles[a.n_seqs] = at_t;
  }
}

__device__ __forceinline__ void qb_number_tree(const QbArgs& a, int b, const int32_t* __restrict__ parents,
                                               int* smem) {
  int *s_par = smem, *s_size = smem + QB_MAX_TREE, *s_off = smem + 2 * QB_MAX_TREE;
  const QbSeq q = qb_seq(a, b, nullptr);
  for (int i = threadIdx.x; i < q.n; i += blockDim.x) {
    int p = parents[q.c0 + i];
    if (p < -1 || p >= i) {
      flag_error(a.err, ERR_TREE);
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
    a.ws.tree[q.c0 + i] = make_int2(tin, s_size[i]);
  }
}

// Identity and signed Hadamard, one warp a row (token, query head): y = x R * scale.
__device__ __forceinline__ void qb_rotate_row(const QbArgs& a, long long r, const void* __restrict__ q, int dtype,
                                              const RotDev& rot, int lane) {
  const int h = (int)(r % a.n_q_heads) / a.gqa;
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
  }
  *reinterpret_cast<float4*>(a.ws.q + (size_t)r * D + 4 * lane) =
      make_float4(y[0] * QB_SCALE, y[1] * QB_SCALE, y[2] * QB_SCALE, y[3] * QB_SCALE);
}

// Dense rotations: a block takes 32 columns of one KV head's R and every `chunks`-th tile of
// its rows.  fp32 values are split into three bf16 limbs (24 bits, exact), bf16 queries
// are one; the products whose limbs count from 2^0 to 2^-16 are taken on mma.sync (m16n8k16,
// fp32 accumulation), 3 for bf16 queries and 6 for fp32, smallest first: about 2^-22 relative.
// The order of the channels in the products is free: step s gives thread t of a row the
// channels 8 (4 (s / 2) + t) + 4 (s % 2) + 0 .. 3, so that it loads its part of a row as four
// runs of 8 channels.  The rotation is a few per cent of the attention's work, so it needs no
// tensor memory; with a load per channel pair instead it was bound by the load pipe (8 x 447 x
// 16 rows: 49 us).
constexpr int QB_ROT_COLS = 32;
__host__ __device__ constexpr int qb_rot_rows(bool f32) { return f32 ? 64 : 128; }

__device__ __forceinline__ void qb_split3(float x, float y, uint32_t (&limb)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    limb[i] = *reinterpret_cast<const uint32_t*>(&h);
    x -= __low2float(h);
    y -= __high2float(h);
  }
}

__device__ __forceinline__ void qb_mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

template <bool F32>
__device__ __forceinline__ void qb_rotate_dense(const QbArgs& a, int h, int slice, int chunk, int chunks,
                                                const void* __restrict__ q, const float* __restrict__ dense,
                                                uint2 (*s_b)[8][QB_ROT_COLS / 8][32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // R's limbs as B fragments: [limb][16-channel step][8 columns][lane = 4 (column % 8) + pair]
  const float* r_in = dense + (size_t)h * D * D + QB_ROT_COLS * slice + lane;
  float2 v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = make_float2(__ldg(r_in + (2 * (warp + 8 * j)) * D), __ldg(r_in + (2 * (warp + 8 * j) + 1) * D));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int p = warp + 8 * j;  // channels 2p, 2p + 1; a lane a column
    uint32_t limb[3];
    qb_split3(v[j].x, v[j].y, limb);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      reinterpret_cast<uint32_t*>(&s_b[i][2 * (p >> 4) + ((p >> 1) & 1)][lane >> 3][4 * (lane & 7) + ((p >> 2) & 3)])[p & 1] = limb[i];
  }
  __syncthreads();
  const int rows = a.n_total << a.gqa_shift, gm = a.gqa - 1;  // n_total * n_q_heads < 2^31
  constexpr int MT = qb_rot_rows(F32) / 64, RUN = F32 ? 2 : 1;  // 16-row tiles a warp; 16-byte loads a run
  const int rg = warp & 3, cg = warp >> 2, g = lane >> 2, t = lane & 3;
  auto offset = [&](int r) { return ((size_t)(r >> a.gqa_shift) * a.n_q_heads + h * a.gqa + (r & gm)) * D; };
  for (long long r0 = (long long)chunk * 64 * MT; r0 < rows; r0 += (long long)chunks * 64 * MT) {
    size_t o[MT][2];  // rows g and g + 8 of the warp's tiles
    uint4 in[MT][2][4][RUN];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o[m][i] = offset(min((int)r0 + 16 * MT * rg + 16 * m + 8 * i + g, rows - 1));
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < RUN; ++e)
            in[m][i][c][e] = __ldg(static_cast<const uint4*>(q) + (o[m][i] + 32 * c + 8 * t) / (F32 ? 4 : 8) + e);
      }
    // the leading products in two sums of four steps, the others in a third: added in fp32 (the tensor cores truncate)
    float d[3][MT][2][4] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t x[MT][F32 ? 3 : 1][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (F32) {
            const uint4 w = in[m][i][k >> 1][k & 1];
            uint32_t lo[3], hi[3];
            qb_split3(__uint_as_float(w.x), __uint_as_float(w.y), lo);
            qb_split3(__uint_as_float(w.z), __uint_as_float(w.w), hi);
#pragma unroll
            for (int e = 0; e < 3; ++e) {
              x[m][e][i] = lo[e];
              x[m][e][2 + i] = hi[e];
            }
          } else {
            const uint4 w = in[m][i][k >> 1][0];
            x[m][0][i] = k & 1 ? w.z : w.x;
            x[m][0][2 + i] = k & 1 ? w.w : w.y;
          }
        }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        uint2 b[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) b[i] = s_b[i][k][2 * cg + n][lane];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if constexpr (F32) {
            qb_mma_bf16(d[2][m][n], x[m][2], b[0]);
            qb_mma_bf16(d[2][m][n], x[m][1], b[1]);
            qb_mma_bf16(d[2][m][n], x[m][0], b[2]);
            qb_mma_bf16(d[2][m][n], x[m][1], b[0]);
          } else {
            qb_mma_bf16(d[2][m][n], x[m][0], b[2]);
          }
          qb_mma_bf16(d[2][m][n], x[m][0], b[1]);
          qb_mma_bf16(d[k >> 2][m][n], x[m][0], b[0]);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if ((int)r0 + 16 * MT * rg + 16 * m + 8 * i + g < rows)
            *reinterpret_cast<float2*>(a.ws.q + o[m][i] + QB_ROT_COLS * slice + 16 * cg + 8 * n + 2 * t) =
                make_float2((d[0][m][n][2 * i] + (d[1][m][n][2 * i] + d[2][m][n][2 * i])) * QB_SCALE,
                            (d[0][m][n][2 * i + 1] + (d[1][m][n][2 * i + 1] + d[2][m][n][2 * i + 1])) * QB_SCALE);
  }
}

template <int N>
__global__ void __launch_bounds__(QB_PREP_THREADS)
qb_prepare_kernel(QbArgs a, const int32_t* __restrict__ parents, const void* __restrict__ q, int dtype, RotDev rot,
                  int chunks) {
  __shared__ __align__(16) uint2 s_b[3][8][QB_ROT_COLS / 8][32];
  pdl_launch_dependents();
  const int trees = a.mode == QB_TREE ? a.n_seqs : 0;
  const int block = (int)blockIdx.x - 1 - trees;
  if (blockIdx.x == 0) {
    qb_list_tiles<N>(a);
  } else if (block < 0) {
    qb_number_tree(a, blockIdx.x - 1, parents, reinterpret_cast<int*>(s_b));
  } else if (rot.kind == KVQ_ROT_DENSE) {
    const int H = a.g.n_kv_heads, h = block % H, slice = block / H % (D / QB_ROT_COLS), chunk = block / (H * (D / QB_ROT_COLS));
    if (dtype == KVQ_F32) qb_rotate_dense<true>(a, h, slice, chunk, chunks, q, rot.dense, s_b);
    else qb_rotate_dense<false>(a, h, slice, chunk, chunks, q, rot.dense, s_b);
  } else {
    const long long r = (long long)block * (QB_PREP_THREADS / 32) + (threadIdx.x >> 5);
    if (r < (long long)a.n_total * a.n_q_heads) qb_rotate_row(a, r, q, dtype, rot, threadIdx.x & 31);
  }
}

// ---------------------------------------------------------------------------
// Tensor memory wrappers of this kernel
// ---------------------------------------------------------------------------
// D[tmem] (+)= A[tmem] B[smem]^T, fp16 operands, by one thread; D enters times 2^-SHIFT.
template <int SHIFT = 0>
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, bool acc) {
  if constexpr (SHIFT == 0)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p, %5;\n}" ::"r"(d),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)acc), "n"(SHIFT)
        : "memory");
}
// One lane of a converged warp, in the form from which the compiler knows that the code
// under it runs in a single thread (its matrix operands then need no per-lane loop).
__device__ __forceinline__ bool qb_elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0;
}
// fp16 A and B, fp32 D, M = 128; B K-major or (rows of N) MN-major (bit 16).
__host__ __device__ constexpr uint32_t qb_idesc(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

#define QB_R8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// this thread's lane, 16 consecutive columns
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      QB_R8(r, 0), QB_R8(r, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&v)[8]) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), QB_R8(r, 0)
               : "memory");
}
// 16 lanes x 16 columns: thread t holds row t / 4 (and + 8), column t % 4 of every group of four columns
__device__ __forceinline__ void tmem_st16x128_x4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), QB_R8(r, 0)
               : "memory");
}
#undef QB_R8
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// This thread's scores of `n` rows, in place, each times its row's power of two; `lo` columns further on, if not 0, the
// second half's scores.  Rarely called: out of line, to stay out of the hot loop's instructions (inlined, 16 trees of 32
// drafts on 16k took 363.6 instead of 360.7 us, 4 x 512 chunk on 8k 753 instead of 750).
__device__ __noinline__ void qb_scale_back(uint32_t scores, const float* row_unscale, int n, int lo) {
  tc_fence_after();
  for (int half = 0; half <= lo; half += max(1, lo))
    for (int j = 0; j < n; j += 8) {
      float v[8];
      tmem_ld8(scores + half + j, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= row_unscale[j + k];
      tmem_st8(scores + half + j, v);
    }
  tmem_wait_st();
}

// 16 consecutive columns of this thread's lane; the load and its wait are one statement.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
template <int C>
__device__ __forceinline__ void qb_tmem_ld(uint32_t taddr, float (&v)[C]) {
  static_assert(C == 8 || C % 16 == 0, "columns");
  if constexpr (C == 8) {
    tmem_ld8(taddr, v);
  } else {
#pragma unroll
    for (int c = 0; c < C; c += 16) tmem_ld16(taddr + c, *reinterpret_cast<float(*)[16]>(v + c));
  }
}

// ---------------------------------------------------------------------------
// Expansion of 2-bit codes, both 16-bit halves of a register at once, as fp16 c - 1.5:
// a field (bits 2f, 2f + 1 of a half) masked into the mantissa of 2^k + c (exact), from
// which 2^k + 1.5 is subtracted (exact).  Fields that would straddle the exponent bits
// are taken from the byte-swapped halves (keys) or rotated (values).  Keys as plain c, a
// subnormal c 2^(bit - 24) without the subtraction, ran as fast but cost precision in the
// scores (readout error 1.6e-6 instead of 5e-7).
// ---------------------------------------------------------------------------
__host__ __device__ constexpr int qb_bit(int f) { return f == 0 ? 8 : f <= 4 ? 2 * f : 2 * f - 8; }  // 2, 4, 6 or 8
__device__ __forceinline__ uint32_t qb_swap(uint32_t x) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %1, 0x2301;" : "=r"(d) : "r"(x));
  return d;
}
// The field at bits BIT, BIT + 1 as c - 1.5.
template <int BIT>
__device__ __forceinline__ uint32_t qb_centred(uint32_t x) {
  constexpr uint32_t e = (uint32_t)(25 - BIT) << 10;  // 2^(10 - BIT): one unit of c at that bit
  constexpr uint32_t off = e + (3u << (BIT - 1));     // 2^(10 - BIT) + 1.5
  const uint32_t v = (x & (0x00030003u << BIT)) | (e | (e << 16));
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v),
                            __halves2half2(__ushort_as_half(off), __ushort_as_half(off)));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ float qb_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Maximum over the warp (of what is not NaN).
__device__ __forceinline__ float qb_warp_max(float x) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}
__device__ __forceinline__ float qb_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t qb_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// A vote of four warps at hardware barrier `id`.
__device__ __forceinline__ bool qb_vote(int id, bool p) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return any != 0;
}
// A token's constants: key scale and mid, log2 of the value scale, its reciprocal, value mid over value scale.
enum { QB_C_SK, QB_C_KMID, QB_C_LS, QB_C_INV, QB_C_ZC };

// Register shares by role (a thread; 0: as launched): keys, values, softmax, accumulation, copies and MMA issue.  The
// 24 warps are launched with 80; the 64-row tile: 4 x 40 + 4 x 48 + 8 x 128 + 4 x 96 + 4 x 40 = 1920 = 24 x 80; the 32-row
// tile: 4 x 56 + 4 x 56 + 8 x 104 + 4 x 96 + 4 x 56 = 1888.
struct QbRegisters {
  int keys, values, softmax, acc, misc;
};
__host__ __device__ constexpr QbRegisters qb_shares(int n) {
  return n == 64 ? QbRegisters{40, 48, 128, 96, 40} : n == 32 ? QbRegisters{56, 56, 104, 96, 56} : QbRegisters{0, 0, 0, 0, 0};
}

// Register shares of a group of four warps (the block's total stays what it was launched with).
template <int R, bool UP>
__device__ __forceinline__ void qb_registers() {
  if constexpr (R == 0) return;
  else if constexpr (UP) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

template <int N>
struct QbShared {  // alignas: read as 16-byte vectors
  alignas(16) float sumq[2][N];     // per row of the unit's queries: sum(q')
  alignas(16) int tin[2][N];
  alignas(16) float neg_m[2][N];    // -M, 0 at first
  alignas(16) float scale[4][N];    // factors of the accumulated numerator for tile i (i % 4), where flagged
  alignas(8) int moved[4][QB_GROUPS];            // per group: whether tile i (i % 4) moved a reference
  alignas(16) float red[QB_GROUPS][4][32];        // per group: the rows' maxima per warp
  alignas(8) float delta[QB_GROUPS][32];          // per group: how far the references moved
  alignas(16) float tok[4][5][QB_TOK];  // constants of tile i (i % 4): see QB_C_*
  alignas(16) float lsum[4][N];
  alignas(16) float zsum[4][N];
  alignas(16) QbUnit unit[QB_UNITS];
  QbUnit first;
  alignas(8) long long tiles_before[2];  // the slice's two ends
  long long work;                        // of all slices
  float unscale[2];                 // what the products of key codes and queries are scaled back by
  bool apart[2];                    // rows far apart in size: unscale is 1, and each row has its own row_unscale
  alignas(16) float row_unscale[2][N];
  uint32_t qmax[2][4], qmin[2][4];  // bits of the warps' largest and smallest row maxima (of rows that are not all zero)
  float row_z[N], row_f[N];         // of the unit being written out
  alignas(8) uint64_t full[QB_STAGES];
  uint64_t empty[QB_STAGES];
  uint64_t unit_full[QB_UNITS], unit_free[QB_UNITS];
  uint64_t q_ready[2];
  // by tile parity.  k_ready: its keys are expanded.  p_ready: its weights and values are there and the products of
  // two tiles earlier are read (softmax, expansion and accumulation warps arrive).  s_done, o_done: the tensor cores have
  // finished its scores, its readout.  They work in order - scores of i + 1, readout of i - so s_done(i) also says
  // that the readout of i - 2 is finished with its weights, and p_ready(i - 2) that the scores of i - 2 are read.
  uint64_t k_ready[2], p_ready[2], s_done[2], o_done[2];
  uint64_t lz_ready, lz_free, last;
  uint64_t group;                   // meetings of the four accumulation warps
  uint32_t tmem;
};
static_assert(offsetof(QbShared<16>, neg_m) % 16 == 0 && offsetof(QbShared<16>, tok) % 16 == 0 &&
                  offsetof(QbShared<16>, scale) % 16 == 0 && offsetof(QbShared<16>, sumq) % 16 == 0,
              "vector reads");

template <int N>
__global__ void __launch_bounds__(QB_THREADS, 1) qb_attend_kernel(QbArgs a) {
  constexpr int NG = QB_GROUPS, NH = N / NG;  // groups of softmax warps, rows of a group
  constexpr int W_ACC = 8 + 4 * NG, W_COPY = W_ACC + 4, W_MMA = W_COPY + 1;  // first warps of the roles
  // Up to 32 rows the two halves of an fp32 operand stand side by side as 2 N columns of one product, whose two results are
  // added by the reader: an MMA of few columns takes as long as its A operand (about 35 cycles), so half as many MMAs
  // run in half the time.  64 rows: one product after the other into the same columns.
  constexpr bool PAIR = N <= 32;
  constexpr uint32_t T_K = 0, T_V = 128, T_S = 256, T_O = 384;  // tensor memory columns, two buffers of 64 each
  extern __shared__ uint8_t qb_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(qb_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem;                          // [2 units][hi, lo][2 halves of 64 channels][N rows of 128 bytes]; PAIR: [units][halves][hi, lo][N]
  uint8_t* s_p = s_q + 2 * N * 512;             // [2 tiles][hi, lo][128 tokens of 128 bytes]; PAIR: [tiles][1][tokens of N hi, N lo]
  uint8_t* s_stage = s_p + 4 * QB_PBUF;
  float* s_out = reinterpret_cast<float*>(s_stage + QB_STAGES * QB_STAGE_BYTES);  // [N][128] of a finished unit
  __shared__ QbShared<N> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr unsigned FULLM = 0xffffffffu;
  constexpr int Q_LO = PAIR ? N * 128 : N * 256, Q_HALF = PAIR ? 2 * N * 128 : N * 128;  // bytes from hi to lo, from half to half
  // byte of the 16-byte chunk `c` (8 rows) of a token's hi (0) or lo (1) weights
  auto p_at = [](int part, int c, int token) {
    return PAIR ? token * 128 + (((c + part * (N / 8)) ^ (token & 7)) << 4) : part * QB_PBUF + token * 128 + ((c ^ (token & 7)) << 4);
  };

  // Up to QB_FEW sequences the list of work, the pages and their expansion need nothing of the preparation: only the
  // warps that read its queries and trees wait for it.
  if (a.n_seqs > QB_FEW) pdl_wait();
  if (tid == 32) {
    for (int i = 0; i < QB_STAGES; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 4 + 4);
    }
    for (int i = 0; i < QB_UNITS; ++i) {
      mbar_init(&sh.unit_full[i], 1);
      mbar_init(&sh.unit_free[i], 4 * NG + 4 + 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_ready[i], 4);
      mbar_init(&sh.k_ready[i], 4);
      mbar_init(&sh.s_done[i], 1);
      mbar_init(&sh.p_ready[i], 4 + 4 * NG + 4);
      mbar_init(&sh.o_done[i], 1);
    }
    mbar_init(&sh.lz_ready, 4 * NG);
    mbar_init(&sh.lz_free, 4);
    mbar_init(&sh.last, 1);
    mbar_init(&sh.group, 4);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  if (warp == 2 || warp == 3) {  // the slice's first unit and its tiles
    const QbList<N> list(a, lane);
    const QbSlices slices(list.work, gridDim.x);
    const long long w0 = slices.start(blockIdx.x), w1 = slices.start(blockIdx.x + 1);
    long long before = 0;
    if (w1 > w0) {
      int in;
      if (warp == 2) {
        const QbUnit u = qb_locate<N>(a, list, w0, lane, in, before);
        if (lane == 0) sh.first = u;
      } else if (w1 < list.work) {
        qb_locate<N>(a, list, w1, lane, in, before);
      } else {
        before = list.tiles;
      }
    }
    if (lane == 0) {
      sh.tiles_before[warp - 2] = before;
      sh.work = list.work;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = sh.tmem;
  const int n_tiles = (int)(sh.tiles_before[1] - sh.tiles_before[0]);

  // warp-uniform bounded wait, kept short (it stands in many places); a role that gives up ends, and with
  // it, in time, the others
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    int left = WAIT_LIMIT;
#pragma unroll 1
    while (!__all_sync(FULLM, mbar_try_wait(bar, parity & 1)))
      if (--left == 0) return false;
    return true;
  };
  auto gave_up = [&]() {
    if (lane == 0) flag_error(a.err, ERR_TIMEOUT);
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // the four accumulation warps meet (a bounded wait, unlike a hardware barrier)
  uint32_t round = 0;
  auto meet = [&]() {
    arrive(&sh.group);
    return wait(&sh.group, round++);
  };

  if (n_tiles > 0) {
    if (warp < 4) {
      // ---- key codes -> tensor memory, and the tokens' constants ----
      qb_registers<qb_shares(N).keys, false>();
      const uint32_t lanes = (uint32_t)(32 * warp) << 16;
      const int ps = a.page_shift, pm = (1 << ps) - 1;
      const int tok = 32 * warp + lane;
      const int k_off = (tok >> ps) * a.g.record + 32 * (tok & pm);
      const int meta_off = (tok >> ps) * a.g.record + (64 << ps) + 4 * (tok & pm);
      int i = 0;
      for (; i < n_tiles; ++i) {
        const int st = i % QB_STAGES, buf = i & 1;
        const uint8_t* stage = s_stage + st * QB_STAGE_BYTES;
        if (!wait(&sh.full[st], i / QB_STAGES)) break;
        const float2 km = __half22float2(*reinterpret_cast<const __half2*>(stage + meta_off));
        const float2 vm = __half22float2(*reinterpret_cast<const __half2*>(stage + meta_off + (4 << ps)));
        const float sv = vm.x == 0.f ? 5.9604644775390625e-08f : vm.x;
        float ls = __log2f(sv), inv = __fdividef(1.f, sv), zc = inv * fmaf(1.5f, sv, vm.y);
        if (!(fabsf(zc) <= 3.4e38f)) {  // not finite: NaN for the rows that see the token, 0 * 0 for the others
          ls = NAN;
          inv = zc = 0.f;
        }
        // the scores of tile i - 2 are done: its expanded keys may go, and the constants of tile i - 4 have been read
        if (i >= 2 && !wait(&sh.s_done[buf], (i >> 1) - 1)) break;
        float(*c)[QB_TOK] = sh.tok[i & 3];
        c[QB_C_SK][tok] = km.x;
        c[QB_C_KMID][tok] = fmaf(1.5f, km.x, km.y);
        c[QB_C_LS][tok] = ls;
        c[QB_C_INV][tok] = inv;
        c[QB_C_ZC][tok] = zc;
        tc_fence_after();
        // short loops on purpose: straight-line code runs at the speed of the instruction fetch
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const uint2 w = *reinterpret_cast<const uint2*>(stage + k_off + 8 * k);
          uint32_t r[16];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t x = e ? w.y : w.x, y = qb_swap(x);
            r[8 * e + 0] = qb_centred<qb_bit(0)>(y);
            r[8 * e + 1] = qb_centred<qb_bit(1)>(x);
            r[8 * e + 2] = qb_centred<qb_bit(2)>(x);
            r[8 * e + 3] = qb_centred<qb_bit(3)>(x);
            r[8 * e + 4] = qb_centred<qb_bit(4)>(x);
            r[8 * e + 5] = qb_centred<qb_bit(5)>(y);
            r[8 * e + 6] = qb_centred<qb_bit(6)>(y);
            r[8 * e + 7] = qb_centred<qb_bit(7)>(y);
          }
          tmem_st16(tmem + lanes + T_K + 64 * buf + 16 * k, r);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(&sh.k_ready[buf]);
        arrive(&sh.empty[st]);
      }
      if (i < n_tiles) gave_up();
    } else if (warp < 8) {
      // ---- value codes -> tensor memory ----
      qb_registers<qb_shares(N).values, false>();
      const uint32_t lanes = (uint32_t)(32 * (warp - 4)) << 16;
      const int ps = a.page_shift, pm = (1 << ps) - 1;
      // rows of the transposing loads: lane l gives row l % 8 of matrix l / 8; 16 tokens are 1152 bytes of either page size
      const int vt = (lane & 7) + ((lane >> 4) << 3), vh = (lane >> 3) & 1;
      const int v_off = (vt >> ps) * a.g.record + (32 << ps) + 32 * (vt & pm) + 16 * vh;
      // a warp's fields 2 w and 2 w + 1 are bits 4 w .. 4 w + 3: rotated to bits 4 .. 7
      const int v_rotate = (4 * (warp - 4) - 4) & 31;
      int i = 0;
      for (; i < n_tiles; ++i) {
        const int st = i % QB_STAGES, buf = i & 1;
        const uint8_t* stage = s_stage + st * QB_STAGE_BYTES;
        if (!wait(&sh.full[st], i / QB_STAGES)) break;
        if (i >= 2 && !wait(&sh.o_done[buf], (i >> 1) - 1)) break;
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {  // 32 tokens: 16 columns
          uint32_t raw[8], r[8];
          ldsm_x4_trans(smem_u32(stage + v_off + 2304 * k), *reinterpret_cast<uint32_t(*)[4]>(raw));
          ldsm_x4_trans(smem_u32(stage + v_off + 2304 * k + 1152), *reinterpret_cast<uint32_t(*)[4]>(raw + 4));
          const uint32_t ta = tmem + lanes + T_V + 64 * buf + 16 * k;
#pragma unroll
          for (int j = 0; j < 8; ++j) raw[j] = __funnelshift_r(raw[j], raw[j], v_rotate);
#pragma unroll
          for (int j = 0; j < 8; ++j) r[j] = qb_centred<4>(raw[j]);
          tmem_st16x128_x4(ta, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) r[j] = qb_centred<6>(raw[j]);
          tmem_st16x128_x4(ta + (16u << 16), r);
        }
        arrive(&sh.empty[st]);
        tmem_wait_st();
        tc_fence_before();
        arrive(&sh.p_ready[buf]);
      }
      if (i < n_tiles) gave_up();
    } else if (warp < W_ACC) {
      // ---- softmax: one token a thread, rows col0 .. col0 + NH - 1 ----
      qb_registers<qb_shares(N).softmax, true>();
      pdl_wait();
      const int group = (warp - 8) >> 2, q4 = warp & 3, col0 = group * NH;
      const uint32_t lanes = (uint32_t)(32 * q4) << 16;
      const int tok = 32 * q4 + lane;
      const bool lead = tid == 256 + 128 * group;
      float unscale = 0.f;
      const float* s_sumq = nullptr;
      const int* s_tin = nullptr;
      float* s_neg_m = nullptr;
      int un = -1, t = 0, t1 = 0, base = 0, open = 0, len = 0, c0 = 0;
      bool unset = false, fresh = false;
      uint64_t l2[NH / 2], z2[NH / 2];
      // One hardware vote a tile, so every warp makes exactly n_tiles rounds: one whose wait has run out
      // stays in step with the others and does nothing else.
      bool ok = true;
      for (int i = 0; i < n_tiles; ++i, ++t) {
        const int buf = i & 1, use = i >> 1;
        if (t == t1 && ok) {
          ++un;
          if ((ok = wait(&sh.unit_full[un % QB_UNITS], un / QB_UNITS) && wait(&sh.q_ready[un & 1], un >> 1))) {
            const QbUnit& u = sh.unit[un % QB_UNITS];
            t = u.t0;
            t1 = u.t1;
            len = u.len;
            c0 = u.c0;
            base = a.mode == QB_CROSS ? u.len : u.len - u.n;
            // positions below `open` are seen by every row of the tile (a unit with rows far apart in size: none, so that
            // every tile goes through the branch where their scores are scaled back)
            open = sh.apart[un & 1] ? QB_APART : a.mode == QB_CHAIN ? base + u.rt * (N >> a.gqa_shift) + 1 : base;
            arrive(&sh.unit_free[un % QB_UNITS]);
            unscale = sh.unscale[un & 1];
            s_sumq = sh.sumq[un & 1];
            s_tin = sh.tin[un & 1];
            s_neg_m = sh.neg_m[un & 1];
            unset = tok < NH;  // row col0 + tok has seen nothing yet, and M = 0
            fresh = true;      // some row has not
#pragma unroll
            for (int j = 0; j < NH / 2; ++j) l2[j] = z2[j] = 0ull;
          }
        }
        {
          const bool masked = (t + 1) * QB_TOK > open;
          int key_tin = 0;
          unsigned key_size = 0x7fffffffu;
          if (__builtin_expect(masked && ok, 0)) {
            if (open == QB_APART && wait(&sh.s_done[buf], use))
              qb_scale_back(tmem + lanes + T_S + 64 * buf + col0, sh.row_unscale[un & 1] + col0, NH, PAIR ? N : 0);
            const int d = t * QB_TOK + tok - base;
            if (d + base >= len) {
              key_size = 0u;
            } else if (d >= 0) {
              const int2 ts = a.mode == QB_TREE ? a.ws.tree[c0 + d] : make_int2(d, len - base - d);
              key_tin = ts.x;
              key_size = (unsigned)ts.y;
            }
          }
          if (!ok || !wait(&sh.s_done[buf], use)) {
            ok = false;
            if (qb_vote(1 + group, false)) {  // the others move their references
              qb_vote(1 + group, false);
              qb_vote(1 + group, false);
            }
            continue;
          }
          tc_fence_after();
          const float(*tc)[QB_TOK] = sh.tok[i & 3];
          const float sk = tc[QB_C_SK][tok] * unscale, kmid = tc[QB_C_KMID][tok], ls = tc[QB_C_LS][tok],
                      inv = tc[QB_C_INV][tok], zc = tc[QB_C_ZC][tok];
          const uint64_t sk2 = f2pk(sk, sk), kmid2 = f2pk(kmid, kmid), ls2 = f2pk(ls, ls), inv2 = f2pk(inv, inv),
                         zc2 = f2pk(zc, zc);
          uint8_t* weights = s_p + (2 * buf) * QB_PBUF;
          const uint32_t scores = tmem + lanes + T_S + 64 * buf + col0;
          if (lead) sh.moved[i & 3][group] = 0;
          // x: a + log2 s - M, -infinity where the row does not see the token
          float x[NH], top = -INFINITY;
          qb_tmem_ld<NH>(scores, x);
          if constexpr (PAIR) {
            float y[NH];
            qb_tmem_ld<NH>(scores + N, y);
#pragma unroll
            for (int j = 0; j < NH; ++j) x[j] += y[j];
          }
#pragma unroll
          for (int j = 0; j < NH; j += 4) {
            const float4 sq = *reinterpret_cast<const float4*>(s_sumq + col0 + j);
            const float4 nm = *reinterpret_cast<const float4*>(s_neg_m + col0 + j);
            const uint64_t u0 = f2fma(kmid2, f2pk(sq.x, sq.y), f2add(f2pk(nm.x, nm.y), ls2));
            const uint64_t u1 = f2fma(kmid2, f2pk(sq.z, sq.w), f2add(f2pk(nm.z, nm.w), ls2));
            const float2 d0 = f2up(f2fma(sk2, f2pk(x[j], x[j + 1]), u0));
            const float2 d1 = f2up(f2fma(sk2, f2pk(x[j + 2], x[j + 3]), u1));
            x[j] = d0.x; x[j + 1] = d0.y; x[j + 2] = d1.x; x[j + 3] = d1.y;
          }
          if (__builtin_expect(masked, 0)) {
#pragma unroll
            for (int j = 0; j < NH; ++j) x[j] = (unsigned)(s_tin[col0 + j] - key_tin) < key_size ? x[j] : -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < NH; j += 2) top = qb_max3(top, x[j], x[j + 1]);
          // whether any weight of the 128 tokens would pass the limit
          if (__builtin_expect(qb_vote(1 + group, top > QB_TRIGGER || fresh), 0)) {
            // the references move up to the rows' maxima over the 128 tokens
            float row_max = 0.f;
#pragma unroll
            for (int j = 0; j < NH; ++j) {
              const float m = qb_warp_max(x[j]);
              if (lane == j) row_max = m;
            }
            if (lane < NH) sh.red[group][q4][lane] = row_max;
            qb_vote(1 + group, false);
            bool some = false;
            if (tok < NH) {
              const float m = fmaxf(fmaxf(sh.red[group][0][tok], sh.red[group][1][tok]),
                                    fmaxf(sh.red[group][2][tok], sh.red[group][3][tok]));
              const float by = (unset ? m > -INFINITY : m > QB_LIFT) ? m - QB_LIFT : 0.f;
              s_neg_m[col0 + tok] -= by;
              sh.delta[group][tok] = by;
              sh.scale[i & 3][col0 + tok] = unset ? 1.f : qb_ex2(-by);  // nothing to scale yet
              if (m > -INFINITY) unset = false;
              some = unset;
              if (lead) sh.moved[i & 3][group] = 1;
            }
            fresh = qb_vote(1 + group, some);
#pragma unroll
            for (int j = 0; j < NH; j += 2) {
              const float2 f = *reinterpret_cast<const float2*>(sh.scale[i & 3] + col0 + j);
              const float2 by = *reinterpret_cast<const float2*>(sh.delta[group] + j);
              const uint64_t f2 = f2pk(f.x, f.y);
              l2[j / 2] = f2mul(l2[j / 2], f2);
              z2[j / 2] = f2mul(z2[j / 2], f2);
              x[j] -= by.x;
              x[j + 1] -= by.y;
            }
          }
#pragma unroll
          for (int j = 0; j < NH; ++j) x[j] = qb_ex2(x[j]);
#pragma unroll
          for (int j = 0; j < NH; j += 8) {  // two fp16 halves of every weight
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float w0 = x[j + 2 * k], w1 = x[j + 2 * k + 1];
              hi[k] = qb_half2(w0, w1);
              const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi[k]));
              const float2 r = f2up(f2mul(f2sub(f2pk(w0, w1), f2pk(back.x, back.y)), f2pk(QB_LO_UP, QB_LO_UP)));
              lo[k] = qb_half2(r.x, r.y);
            }
            const int c = (col0 + j) >> 3;
            *reinterpret_cast<uint4*>(weights + p_at(0, c, tok)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(weights + p_at(1, c, tok)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          tc_fence_before();
          fence_proxy_async();
          arrive(&sh.p_ready[buf]);
#pragma unroll
          for (int j = 0; j < NH; j += 2) {
            const uint64_t w2 = f2pk(x[j], x[j + 1]);
            l2[j / 2] = f2fma(w2, inv2, l2[j / 2]);
            z2[j / 2] = f2fma(w2, zc2, z2[j / 2]);
          }
        }
        if (t + 1 < t1) continue;
        // the unit's l and sum p mid over the warp's 32 tokens: every thread leaves its NH values where its weights of
        // the next tile will go, and adds one row up
        if ((i > 0 && !(ok = wait(&sh.o_done[(i - 1) & 1], (i - 1) >> 1))) || (un && !(ok = wait(&sh.lz_free, un - 1))))
          continue;
        uint8_t* mine = s_p + 2 * ((i + 1) & 1) * QB_PBUF;
        // a chunk's two places (hi and lo) hold 8 rows of fp32
        auto at = [&](int row, int token) { return mine + p_at((row >> 2) & 1, (col0 + row) >> 3, token); };
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
          for (int j = 0; j < NH; j += 4) {
            const float2 p = f2up(pass ? z2[j / 2] : l2[j / 2]), q = f2up(pass ? z2[j / 2 + 1] : l2[j / 2 + 1]);
            *reinterpret_cast<float4*>(at(j, tok)) = make_float4(p.x, p.y, q.x, q.y);
          }
          __syncwarp();
          if (lane < NH) {
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
            for (int k = 0; k < 32; k += 4)
#pragma unroll
              for (int e = 0; e < 4; ++e) sum[e] += reinterpret_cast<const float*>(at(lane, 32 * q4 + k + e))[lane & 3];
            (pass ? sh.zsum : sh.lsum)[q4][col0 + lane] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
          }
          __syncwarp();
        }
        arrive(&sh.lz_ready);
      }
      if (!ok) gave_up();
    } else if (warp < W_COPY) {
      // ---- accumulation: one channel a thread ----
      qb_registers<qb_shares(N).acc, true>();
      pdl_wait();
      const int q4 = warp & 3, wt = tid - 32 * W_ACC;
      const uint32_t lanes = (uint32_t)(32 * q4) << 16;
      constexpr int TPR = 128 / N;  // threads a query row
      const int row = wt / TPR, part = wt % TPR, gs = a.gqa_shift, gm = (1 << gs) - 1;
      // channel 8 g + f is in tensor-memory lane 16 f + g: this thread's channels 4 lane .. 4 lane + 3 are 16 lanes apart
      const int from = 64 * (lane & 1) + (lane >> 1);
      QbUnit u{};
      int i = 0;
      bool done = false;
      int4 join = make_int4(0, 0, 0, 0);
      arrive(&sh.p_ready[0]);  // nothing to read before tiles 0 and 1
      arrive(&sh.p_ready[1]);
      // round un: the queries of unit un + 1 into their buffer, then unit un
      for (int un = -1;; ++un) {
        if (!wait(&sh.unit_full[(un + 1) % QB_UNITS], (un + 1) / QB_UNITS)) break;
        const QbUnit next = sh.unit[(un + 1) % QB_UNITS];
        arrive(&sh.unit_free[(un + 1) % QB_UNITS]);
        if (next.t1 > next.t0) {
          const int R = next.rt * N + row, tk = R >> gs, buf = (un + 1) & 1;
          const bool valid = tk < next.n;
          const float* src =
              a.ws.q + ((size_t)(next.c0 + (valid ? tk : 0)) * a.n_q_heads + next.h * a.gqa + (R & gm)) * D + part * N;
          // all of a thread's loads at once: with a round trip per load this took 8 us a unit
          float v[N];
#pragma unroll
          for (int j = 0; j < N; j += 4) {
            const float4 x = valid ? *reinterpret_cast<const float4*>(src + j) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[j] = x.x; v[j + 1] = x.y; v[j + 2] = x.z; v[j + 3] = x.w;
          }
          float m = 0.f, s = 0.f;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            s += v[j];
            const float w = fabsf(v[j]);
            m = w < INFINITY ? fmaxf(m, w) : m;  // of the finite ones
          }
#pragma unroll
          for (int d = 1; d < TPR; d <<= 1) {
            s += __shfl_xor_sync(FULLM, s, d);
            m = fmaxf(m, __shfl_xor_sync(FULLM, m, d));  // the row's
          }
          // non-negative floats are in the order of their bits
          uint32_t top = __reduce_max_sync(FULLM, __float_as_uint(m));
          uint32_t low = __reduce_min_sync(FULLM, m > 0.f ? __float_as_uint(m) : 0x7f7fffffu);
          if (lane == 0) {
            sh.qmax[buf][q4] = top;
            sh.qmin[buf][q4] = low;
          }
          if (!meet()) break;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            top = max(top, sh.qmax[buf][k]);
            low = min(low, sh.qmin[buf][k]);
          }
          // One power of two for the tile puts its largest row at 2^13 .. 2^14.  fp16's step is 2^-24 at least, so a row keeps
          // the 22 bits of its two halves down to 2^-16 of the largest.  Where some row is smaller, each has a power of its
          // own, and its scores are scaled back by it, so that no row's precision depends on another's size (multiplied into
          // every score of every tile, the rows' own powers cost 11 % of a long call: 357 -> 395 us on 16 trees of 32 drafts on 16k).
          const bool apart = (int)(top >> 23) - (int)(low >> 23) > 16;
          const uint32_t of = apart ? __float_as_uint(m) : top;
          const int e = of ? min(100, 13 - ((int)(of >> 23) - 127)) : 0;  // -114 for the largest finite row
          const float scale = __uint_as_float((uint32_t)(127 + e) << 23);
          uint8_t* dst = s_q + buf * N * 512 + row * 128;
#pragma unroll
          for (int j = 0; j < N; j += 16) {
            // K order of the expanded keys: channels f and 8 + f of a 16-channel word side by side
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int f = 0; f < 8; ++f) {
              const float x = v[j + f] * scale, y = v[j + 8 + f] * scale;
              hi[f] = qb_half2(x, y);
              const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi[f]));
              lo[f] = qb_half2(x - back.x, y - back.y);
            }
            const int w = (part * N + j) >> 4;  // 16-channel word
            uint8_t* d = dst + (w >> 2) * Q_HALF;
            const int c0 = ((2 * (w & 3)) ^ (row & 7)) << 4, c1 = ((2 * (w & 3) + 1) ^ (row & 7)) << 4;
            *reinterpret_cast<uint4*>(d + c0) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(d + c1) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
            *reinterpret_cast<uint4*>(d + Q_LO + c0) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            *reinterpret_cast<uint4*>(d + Q_LO + c1) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
          }
          if (part == 0) {
            sh.sumq[buf][row] = s;
            sh.neg_m[buf][row] = 0.f;
            sh.tin[buf][row] =
                !valid ? 0 : a.mode == QB_TREE ? a.ws.tree[next.c0 + tk].x : a.mode == QB_CHAIN ? tk : 0;
          }
          const float back = __uint_as_float((uint32_t)(127 - e) << 23);
          if (part == 0) sh.row_unscale[buf][row] = back;
          if (wt == 0) {
            sh.unscale[buf] = apart ? 1.f : back;
            sh.apart[buf] = apart;
          }
          fence_proxy_async();
          arrive(&sh.q_ready[buf]);
        }
        if (un >= 0) {
          float acc[N];
#pragma unroll
          for (int j = 0; j < N; ++j) acc[j] = 0.f;
          bool ok = true;
          for (int t = u.t0; t < u.t1; ++t, ++i) {
            const int buf = i & 1, use = i >> 1;
            if (!(ok = wait(&sh.o_done[buf], use))) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < NG; ++c) {
              float o[NH];
              qb_tmem_ld<NH>(tmem + lanes + T_O + 64 * buf + c * NH, o);
              if constexpr (PAIR) {
                float low[NH];
                qb_tmem_ld<NH>(tmem + lanes + T_O + 64 * buf + N + c * NH, low);
#pragma unroll
                for (int j = 0; j < NH; ++j) o[j] = fmaf(low[j], QB_LO_DOWN, o[j]);
              }
              if (sh.moved[i & 3][c]) {
#pragma unroll
                for (int j = 0; j < NH; ++j) acc[c * NH + j] *= sh.scale[i & 3][c * NH + j];
              }
#pragma unroll
              for (int j = 0; j < NH; j += 2) {
                const float2 s = f2up(f2add(f2pk(acc[c * NH + j], acc[c * NH + j + 1]), f2pk(o[j], o[j + 1])));
                acc[c * NH + j] = s.x;
                acc[c * NH + j + 1] = s.y;
              }
            }
            tc_fence_before();
            arrive(&sh.p_ready[buf]);  // for tile i + 2
          }
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < N; ++j) s_out[j * D + wt] = acc[j];
          if (!wait(&sh.lz_ready, un)) break;
          const bool whole = u.t0 == 0 && u.t1 == u.nt;
          if (u.t0 == 0 && !whole) {  // the following slices hold the other nt - t1 tiles
            const QbSlices slices(sh.work, gridDim.x);
            int parts = 1;
            while (slices.start(blockIdx.x + 1 + parts) - slices.start(blockIdx.x + 1) < u.nt - u.t1) ++parts;
            join = make_int4(u.c0, u.n, u.rt * a.g.n_kv_heads + u.h, 1 + parts);
          }
          float* part_out = a.ws.part + (size_t)(2 * blockIdx.x + (u.t0 == 0 ? 1 : 0)) * N * (D + 2);
          if (wt < N) {
            const float l = (sh.lsum[0][wt] + sh.lsum[1][wt]) + (sh.lsum[2][wt] + sh.lsum[3][wt]);
            const float z = (sh.zsum[0][wt] + sh.zsum[1][wt]) + (sh.zsum[2][wt] + sh.zsum[3][wt]);
            sh.row_z[wt] = z;
            sh.row_f[wt] = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
            if (!whole) {
              part_out[N * D + wt] = l;
              part_out[N * D + N + wt] = -sh.neg_m[un & 1][wt];
            }
          }
          arrive(&sh.lz_free);
          if (!meet()) break;
          const int rows = min(N, (u.n << gs) - u.rt * N);
          float* out = a.out + ((size_t)u.c0 * a.n_q_heads + u.h * a.gqa) * D + 4 * lane;
#pragma unroll 2
          for (int j = q4; j < rows; j += 4) {
            const float *o = s_out + j * D + from, z = sh.row_z[j], f = sh.row_f[j];
            const float4 y = make_float4((o[0] + z) * f, (o[16] + z) * f, (o[32] + z) * f, (o[48] + z) * f);
            const int R = u.rt * N + j;
            float* to = whole ? out + ((size_t)(R >> gs) * a.n_q_heads + (R & gm)) * D : part_out + j * D + 4 * lane;
            *reinterpret_cast<float4*>(to) = y;
          }
          if (!meet()) break;  // the staging rows may be written again
        }
        if (next.t1 == next.t0) {
          done = true;
          break;
        }
        u = next;
      }
      if (!done) gave_up();
      if (wt == 0) a.ws.join[blockIdx.x] = join;
    } else if (warp == W_COPY) {
      qb_registers<qb_shares(N).misc, false>();
      // ---- page copies, and the list of units one ahead of them ----
      QbUnit u = sh.first, ahead;
      long long left = n_tiles;
      auto publish = [&](int un, QbUnit v, long long room) {
        if (room <= 0) v.t0 = v.t1 = 0;
        else if (v.t1 - v.t0 > room) v.t1 = v.t0 + (int)room;
        bool ok = true;
        if (un >= QB_UNITS) ok = wait(&sh.unit_free[un % QB_UNITS], un / QB_UNITS - 1);
        if (lane == 0) sh.unit[un % QB_UNITS] = v;
        arrive(&sh.unit_full[un % QB_UNITS]);
        return ok;
      };
      bool ok = publish(0, u, left);
      const int pages = QB_TOK / a.g.page_tokens;
      int i = 0;
      for (int un = 0; ok && left > 0; ++un) {
        if (u.t1 - u.t0 > left) u.t1 = u.t0 + (int)left;
        left -= u.t1 - u.t0;
        ahead = u;
        if (left > 0) qb_next<N>(a, ahead);
        if (!(ok = publish(un + 1, ahead, left))) break;
        const int32_t* row = a.table + (size_t)u.b * a.g.max_blocks;
        auto page_of = [&](int t) {  // this lane's page of tile t, -1 where there is none
          const int p = t * pages + lane;
          return t < u.t1 && lane < pages && (long long)p * a.g.page_tokens < u.len ? row[p] : -1;
        };
        auto expected = [&](int t) { return lane < pages && (long long)(t * pages + lane) * a.g.page_tokens < u.len; };
        int id = page_of(u.t0);
        for (int t = u.t0; t < u.t1; ++t, ++i) {
          const int st = i % QB_STAGES;
          const int id_next = page_of(t + 1);
          const bool want = expected(t), good = want && (unsigned)id < (unsigned)a.g.num_blocks;
          if (want && !good) flag_error(a.err, ERR_BLOCK_RANGE);
          if (i >= QB_STAGES && !(ok = wait(&sh.empty[st], i / QB_STAGES - 1))) break;
          const int n = __popc(__ballot_sync(FULLM, good));
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], n * a.g.record);
          __syncwarp();
          if (good)
            bulk_g2s(s_stage + st * QB_STAGE_BYTES + lane * a.g.record,
                     a.pool + ((size_t)id * a.g.n_kv_heads + u.h) * a.g.record, a.g.record, &sh.full[st]);
          id = id_next;
        }
        u = ahead;
      }
      if (!ok) {  // no copy in flight when the CTA ends
        gave_up();
        for (int k = max(0, i - QB_STAGES); k < i; ++k) mbar_wait_bounded(&sh.full[k % QB_STAGES], (k / QB_STAGES) & 1);
      }
    } else if (warp > W_MMA) {
      qb_registers<qb_shares(N).misc, false>();
    } else {
      qb_registers<qb_shares(N).misc, false>();
      // ---- MMA issue ----
      constexpr int COLS = PAIR ? 2 * N : N, PARTS = PAIR ? 1 : 2;
      constexpr uint32_t I_QK = qb_idesc(COLS, false), I_PV = qb_idesc(COLS, true);
      int un = -1, left = 0;
      uint64_t q = 0;
      bool ok = true;
      for (int i = 0; i <= n_tiles; ++i) {  // the scores of tile i, then the readout of tile i - 1
        if (i < n_tiles) {
          const int buf = i & 1, use = i >> 1;
          if (left == 0) {
            ++un;
            if (!(ok = wait(&sh.unit_full[un % QB_UNITS], un / QB_UNITS) && wait(&sh.q_ready[un & 1], un >> 1))) break;
            left = sh.unit[un % QB_UNITS].t1 - sh.unit[un % QB_UNITS].t0;
            arrive(&sh.unit_free[un % QB_UNITS]);
            q = sw128_desc(s_q + (un & 1) * N * 512);
          }
          --left;
          if (!(ok = wait(&sh.k_ready[buf], use))) break;
          tc_fence_after();
          if (qb_elect()) {
            const uint32_t ak = tmem + T_K + 64 * buf, d = tmem + T_S + 64 * buf;
#pragma unroll 1
            for (int p = 0; p < PARTS; ++p)  // (lo, then hi:) 4 steps of 16 channels in each of two halves
#pragma unroll
              for (int k = 0; k < 8; ++k)
                tc_mma_f16_ts(d, ak + 8 * k, q + ((PAIR || p ? 0 : Q_LO) + (k >> 2) * Q_HALF) / 16 + (k & 3) * 2, I_QK, p + k > 0);
            tc_commit(&sh.s_done[buf]);
          }
          __syncwarp();
        }
        if (i > 0) {
          const int buf = (i - 1) & 1, use = (i - 1) >> 1;
          if (!(ok = wait(&sh.p_ready[buf], use))) break;
          tc_fence_after();
          if (qb_elect()) {
            const uint64_t hi = sw128_desc(s_p + (2 * buf) * QB_PBUF), lo = sw128_desc(s_p + (2 * buf + 1) * QB_PBUF);
            const uint32_t av = tmem + T_V + 64 * buf, d = tmem + T_O + 64 * buf;
#pragma unroll 1
            for (int p = 0; p < PARTS; ++p)
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (k == 0 && p) tc_mma_f16_ts<QB_LO_SHIFT>(d, av, hi, I_PV, true);
                else tc_mma_f16_ts(d, av + 8 * k, (PAIR || p ? hi : lo) + k * (2048 >> 4), I_PV, p + k > 0);
            tc_commit(&sh.o_done[buf]);
          }
          __syncwarp();
        }
      }
      if (!ok) {  // let the tensor cores finish before their memory is freed
        gave_up();
        if (qb_elect()) tc_commit(&sh.last);
        __syncwarp();
        mbar_wait_bounded(&sh.last, 0);
      }
    }
  }
  if (n_tiles == 0 && tid == 0) a.ws.join[blockIdx.x] = make_int4(0, 0, 0, 0);
  pdl_wait();  // also of a CTA without tiles: what follows this grid follows the preparation
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Units cut by slices.  Block k joins the unit that starts in slice k and runs past its
// end: its partial there (slot 2k + 1) and slots 2j of the following slices, in order.
constexpr int QB_JOIN_ROWS = 8;  // a warp a row

template <int N>
__global__ void __launch_bounds__(32 * QB_JOIN_ROWS) qb_combine_kernel(QbArgs a) {
  const int lane = threadIdx.x & 31, r = blockIdx.y * QB_JOIN_ROWS + (threadIdx.x >> 5), k = blockIdx.x;
  pdl_wait();
  const int4 join = a.ws.join[k];
  const int parts = join.w, rt = join.z / a.g.n_kv_heads, h = join.z % a.g.n_kv_heads;
  const int R = rt * N + r, tk = R >> a.gqa_shift;
  if (parts == 0 || tk >= join.y) return;
  const float* first = a.ws.part + (size_t)(2 * k + 1) * N * (D + 2);
  const float* rest = a.ws.part + (size_t)(2 * k) * N * (D + 2);  // + 2 j slots: slice k + j
  const size_t step = (size_t)2 * N * (D + 2);
  // eight parts at a time, their loads in flight together, into a running sum (a part without visible tokens, l = 0, has
  // no reference)
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < parts; j0 += 8) {
    float pm[8], pl[8];
    float4 v[8];
    float top = m;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = j0 + j < parts;
      const float* p = j0 + j ? rest + (in ? j0 + j : 1) * step : first;
      pl[j] = in ? p[N * D + r] : 0.f;
      pm[j] = p[N * D + N + r];
      v[j] = *reinterpret_cast<const float4*>(p + r * D + 4 * lane);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, pl[j] != 0.f ? pm[j] : -INFINITY);
    const float f0 = l != 0.f ? exp2f(m - top) : 0.f;
    m = top;
    l *= f0;
    o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (pl[j] == 0.f) continue;
      const float f = exp2f(pm[j] - m);
      o.x = fmaf(v[j].x, f, o.x); o.y = fmaf(v[j].y, f, o.y); o.z = fmaf(v[j].z, f, o.z); o.w = fmaf(v[j].w, f, o.w);
      l = fmaf(pl[j], f, l);
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<float4*>(a.out + ((size_t)(join.x + tk) * a.n_q_heads + h * a.gqa + (R & (a.gqa - 1))) * D + 4 * lane) =
      make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

template <typename K, typename... A>
static cudaError_t qb_launch_pdl(K kernel, dim3 grid, int block, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int N>
static cudaError_t qb_launch(const QbArgs& a, const int32_t* parents, const void* q, int dtype, RotDev rot, int grid,
                             cudaStream_t s) {
  static std::atomic<unsigned long long> attr{0};  // per device
  cudaError_t e = smem_limit_once(attr, qb_attend_kernel<N>, qb_smem_bytes(N));
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.n_total * a.n_q_heads;
  long long blocks = (rows + QB_PREP_THREADS / 32 - 1) / (QB_PREP_THREADS / 32);
  int chunks = 1;
  if (rot.kind == KVQ_ROT_DENSE) {  // at most three blocks an SM (their registers), one wave, each with R's limbs split once
    const int per_chunk = a.g.n_kv_heads * (D / QB_ROT_COLS);
    const int tile = qb_rot_rows(dtype == KVQ_F32);
    const long long tiles = ((long long)a.n_total * a.gqa + tile - 1) / tile, most = 3 * grid / per_chunk;
    chunks = (int)std::max<long long>(1, std::min(tiles, most));
    blocks = (long long)per_chunk * chunks;
  }
  blocks += 1 + (a.mode == QB_TREE ? a.n_seqs : 0);
  qb_prepare_kernel<N><<<(unsigned)blocks, QB_PREP_THREADS, 0, s>>>(a, parents, q, dtype, rot, chunks);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = qb_launch_pdl(qb_attend_kernel<N>, dim3(grid), QB_THREADS, qb_smem_bytes(N), s, a)) != cudaSuccess) return e;
  return qb_launch_pdl(qb_combine_kernel<N>, dim3(grid, N / QB_JOIN_ROWS), 32 * QB_JOIN_ROWS, 0, s, a);
}

cudaError_t launch_query_block(const PageGeom& g, int n_q_heads, int n_seqs, int n_total, const void* q, int dtype,
                               const int32_t* cu_q, int max_q, const int32_t* parents, int mode, const int32_t* lens,
                               int max_len, const int32_t* table, RotDev rot_k, const uint8_t* pool, void* ws_base,
                               float* o_rot, unsigned* err, cudaStream_t s) {
  const int gqa = n_q_heads / g.n_kv_heads, rows = qb_rows(max_q, gqa), grid = device_sm_count();
  QbArgs a{g, n_q_heads, gqa, n_seqs, n_total, max_q, max_len, mode, __builtin_ctz(gqa), __builtin_ctz(g.page_tokens),
           cu_q, lens, table, pool, {}, o_rot, err};
  qb_layout(ws_base, n_seqs, n_total, n_q_heads, rows, grid, &a.ws);
  return rows == 16   ? qb_launch<16>(a, parents, q, dtype, rot_k, grid, s)
         : rows == 32 ? qb_launch<32>(a, parents, q, dtype, rot_k, grid, s)
                      : qb_launch<64>(a, parents, q, dtype, rot_k, grid, s);
}

}  // namespace kvq
