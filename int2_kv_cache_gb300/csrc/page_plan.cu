// Page plans and tree commits: the bookkeeping of a serving step, on the device.
//
// kvq_plan_pages turns the requests' old and new lengths into block-table entries,
// free-page ring updates, cu_new and the slot of every new token.  With
// p(x) = ceil(x / P), sequence b takes max(0, p(new) - p(old)) pages, gives
// max(0, p(old) - p(new)) back and has max(0, new - old) new tokens; three
// exclusive prefix sums over the sequences place them all:
//   page i of the taken list of b   = ring[(head + take_at[b] + i) mod num_blocks]
//   page i of the given list of b  -> ring[(tail + give_at[b] + i) mod num_blocks]
//   token t of b at pos = old + t - cu_new[b] has slot page(pos / P) * P + pos % P
// The taken and the given ring entries never overlap (tail - head + given <=
// num_blocks is checked), so every item is independent once the sums exist.
// Bound: latency (a 256-request step moves a few KB).  Up to PLAN_SMALL sequences
// every CTA forms the prefix sums itself in shared memory and the plan is one
// launch; above, a one-CTA scan leaves them in the workspace for a second launch
// (8,191 requests took 34 us in two launches).
//
// kvq_tree_commit moves the 72-byte records of the accepted drafts down to the
// first drafts' slots: no arithmetic, so the cache bytes are those that were
// attended.  One warp owns a (sequence, KV head): it loads up to 32 records into
// registers before it stores any, and as accepted[i] >= i with both increasing,
// no store of an earlier batch can hit a later batch's source.
#include <algorithm>

#include "kvq_internal.cuh"

namespace kvq {

constexpr int PLAN_SMALL = 16384;       // 3 arrays of 4 bytes: 192 KB of shared memory
constexpr int PLAN_THREADS = 256;       // up to PLAN_FEW sequences, and in the second launch of two
constexpr int PLAN_MANY_THREADS = 1024;
constexpr int PLAN_FEW = 1024;

struct PlanSums {
  long long tok, take, give;
};

__device__ __forceinline__ PlanSums plan_add(const PlanSums& a, const PlanSums& b) {
  return PlanSums{a.tok + b.tok, a.take + b.take, a.give + b.give};
}

// One sequence's counts; bad lengths count nothing and clear `ok`.
__device__ __forceinline__ PlanSums plan_counts(int o, int n, int page_shift, long long max_tokens, bool& ok) {
  if (o < 0 || n < 0 || o > max_tokens || n > max_tokens) {
    ok = false;
    return PlanSums{0, 0, 0};
  }
  const int mask = (1 << page_shift) - 1;
  const int p0 = (int)(((unsigned)o + mask) >> page_shift), p1 = (int)(((unsigned)n + mask) >> page_shift);
  return PlanSums{n > o ? n - o : 0, p1 > p0 ? p1 - p0 : 0, p0 > p1 ? p0 - p1 : 0};
}

// Block-wide exclusive scan of one PlanSums per thread; returns the total.
template <int THREADS>
__device__ __forceinline__ PlanSums plan_scan(PlanSums v, PlanSums& excl, PlanSums* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  PlanSums inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    PlanSums o;
    o.tok = __shfl_up_sync(0xffffffffu, inc.tok, d);
    o.take = __shfl_up_sync(0xffffffffu, inc.take, d);
    o.give = __shfl_up_sync(0xffffffffu, inc.give, d);
    if (lane >= d) inc = plan_add(inc, o);
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  PlanSums before{0, 0, 0}, total{0, 0, 0};
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before = total;
    total = plan_add(total, s_warp[w]);
  }
  excl = PlanSums{before.tok + inc.tok - v.tok, before.take + inc.take - v.take, before.give + inc.give - v.give};
  return total;
}

// Whether the plan can be carried out as a whole.
__device__ __forceinline__ bool plan_feasible(const PlanSums& t, long long head, long long tail, int num_blocks,
                                              int max_new) {
  return head >= 0 && tail >= head && tail - head <= num_blocks && t.take <= tail - head &&
         tail - head + t.give <= num_blocks && t.tok <= max_new;
}

// The sequence whose half-open prefix range holds item i: pre[b] <= i < pre[b + 1].
template <typename T>
__device__ __forceinline__ int plan_find(const T* pre, int n, long long i) {
  int lo = 0, hi = n;  // pre[lo] <= i < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct PlanArgs {
  int n_seqs, page_shift, num_blocks, max_blocks, max_new;
  const int32_t* old_lens;
  const int32_t* new_lens;
  int32_t* table;
  int32_t* ring;
  const long long* ring_in;
  long long* ring_out;
  int32_t* cu_new;
  long long* slots;
  unsigned* err;
};

__device__ __forceinline__ int plan_wrap(long long i, int num_blocks) {
  return (int)(i >= num_blocks ? i - num_blocks : i);
}

// The plan's items, grid-strided over blockIdx.x; blockIdx.y is their kind, so that the kinds' chains of loads run
// beside one another.  tok / take / give: prefix arrays of n_seqs + 1.
enum { PLAN_TOKENS = 0, PLAN_TAKES = 1, PLAN_GIVES = 2, PLAN_KINDS = 3 };

template <typename T>
__device__ __forceinline__ void plan_tokens(const PlanArgs& a, const T* tok, const T* take, const int* old_lens,
                                            const PlanSums& total, bool ok, long long head, long long tail) {
  const long long i0 = (long long)blockIdx.x * blockDim.x + threadIdx.x, step = (long long)gridDim.x * blockDim.x;
  if (i0 == 0) {
    a.ring_out[0] = ok ? head + total.take : head;
    a.ring_out[1] = ok ? tail + total.give : tail;
  }
  for (long long b = i0; b <= a.n_seqs; b += step) a.cu_new[b] = ok ? (int32_t)tok[b] : 0;
  const int mask = (1 << a.page_shift) - 1, hm = ok ? (int)(head % a.num_blocks) : 0;
  for (long long t = i0; t < a.max_new; t += step) {
    long long slot = -1;
    if (ok && t < total.tok) {
      const int b = plan_find(tok, a.n_seqs, t);
      const int old = old_lens[b];
      const int pos = old + (int)(t - tok[b]);
      const int p0 = (int)(((unsigned)old + mask) >> a.page_shift), pi = pos >> a.page_shift;
      const int page = pi < p0 ? a.table[(size_t)b * a.max_blocks + pi]
                               : a.ring[plan_wrap((long long)hm + take[b] + (pi - p0), a.num_blocks)];
      if ((unsigned)page < (unsigned)a.num_blocks) slot = ((long long)page << a.page_shift) + (pos & mask);
      else flag_error(a.err, ERR_BLOCK_RANGE);
    }
    a.slots[t] = slot;
  }
}

template <typename T>
__device__ __forceinline__ void plan_takes(const PlanArgs& a, const T* take, const int* old_lens, long long count,
                                           long long head) {
  const int mask = (1 << a.page_shift) - 1, hm = (int)(head % a.num_blocks);
  for (long long k = (long long)blockIdx.x * blockDim.x + threadIdx.x; k < count; k += (long long)gridDim.x * blockDim.x) {
    const int page = a.ring[plan_wrap(hm + k, a.num_blocks)];
    const int b = plan_find(take, a.n_seqs, k);
    const int p0 = (int)(((unsigned)old_lens[b] + mask) >> a.page_shift);
    if ((unsigned)page >= (unsigned)a.num_blocks) flag_error(a.err, ERR_BLOCK_RANGE);
    a.table[(size_t)b * a.max_blocks + p0 + (int)(k - take[b])] = page;
  }
}

template <typename T>
__device__ __forceinline__ void plan_gives(const PlanArgs& a, const T* give, const int* new_lens, long long count,
                                           long long tail) {
  const int mask = (1 << a.page_shift) - 1, tm = (int)(tail % a.num_blocks);
  for (long long k = (long long)blockIdx.x * blockDim.x + threadIdx.x; k < count; k += (long long)gridDim.x * blockDim.x) {
    const int b = plan_find(give, a.n_seqs, k);
    const int p1 = (int)(((unsigned)new_lens[b] + mask) >> a.page_shift);
    const int page = a.table[(size_t)b * a.max_blocks + p1 + (int)(k - give[b])];
    if ((unsigned)page >= (unsigned)a.num_blocks) flag_error(a.err, ERR_BLOCK_RANGE);
    a.ring[plan_wrap(tm + k, a.num_blocks)] = page;
  }
}

// One launch: every CTA holds what its kind of item needs in shared memory: the sums in 32 bits (those of a plan that
// can be carried out fit: tokens <= max_new, pages <= num_blocks; of another only the verdict, taken in 64 bits, is used)
// and the lengths.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) plan_small_kernel(PlanArgs a) {
  extern __shared__ int s_pre[];
  __shared__ PlanSums s_warp[THREADS / 32];
  const int kind = blockIdx.y;
  int *s_items = s_pre, *s_lens = s_pre + a.n_seqs + 1, *s_take = s_pre + 2 * (a.n_seqs + 1);
  constexpr int PER = THREADS == PLAN_THREADS ? PLAN_FEW / PLAN_THREADS : PLAN_SMALL / PLAN_MANY_THREADS;
  const int per = (a.n_seqs + THREADS - 1) / THREADS;
  const int b0 = min(a.n_seqs, (int)threadIdx.x * per), b1 = min(a.n_seqs, b0 + per);
  const long long max_tokens = (long long)a.max_blocks << a.page_shift;
  const long long head = a.ring_in[0], tail = a.ring_in[1];
  int o[PER], n[PER];  // a thread's run of sequences, its loads in flight together
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    o[i] = b0 + i < b1 ? a.old_lens[b0 + i] : 0;
    n[i] = b0 + i < b1 ? a.new_lens[b0 + i] : 0;
  }
  PlanSums mine{0, 0, 0};
  bool ok = true;
#pragma unroll
  for (int i = 0; i < PER; ++i) mine = plan_add(mine, plan_counts(o[i], n[i], a.page_shift, max_tokens, ok));
  PlanSums at;
  const PlanSums total = plan_scan<THREADS>(mine, at, s_warp);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (b0 + i < b1) {
      s_items[b0 + i] = (int)(kind == PLAN_TOKENS ? at.tok : kind == PLAN_TAKES ? at.take : at.give);
      s_lens[b0 + i] = kind == PLAN_GIVES ? n[i] : o[i];
      if (kind == PLAN_TOKENS) s_take[b0 + i] = (int)at.take;
    }
    at = plan_add(at, plan_counts(o[i], n[i], a.page_shift, max_tokens, ok));
  }
  if (threadIdx.x == 0) s_items[a.n_seqs] = (int)(kind == PLAN_TOKENS ? total.tok : kind == PLAN_TAKES ? total.take : total.give);
  ok = __syncthreads_and(ok) && plan_feasible(total, head, tail, a.num_blocks, a.max_new);
  if (kind == PLAN_TOKENS) {
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) flag_error(a.err, ERR_PLAN);
    plan_tokens(a, s_items, s_take, s_lens, total, ok, head, tail);
  } else if (ok && kind == PLAN_TAKES) {
    plan_takes(a, s_items, s_lens, total.take, head);
  } else if (ok) {
    plan_gives(a, s_items, s_lens, total.give, tail);
  }
}

// Workspace of the two-launch plan: three prefix arrays of n_seqs + 1, then 0 / 1 (feasible).
size_t plan_workspace_bytes(int n_seqs) { return ((size_t)3 * (n_seqs + 1) + 1) * sizeof(long long); }

__global__ void __launch_bounds__(PLAN_MANY_THREADS) plan_scan_kernel(PlanArgs a, long long* ws) {
  __shared__ PlanSums s_warp[PLAN_MANY_THREADS / 32];
  long long *tok = ws, *take = ws + a.n_seqs + 1, *give = ws + 2 * ((size_t)a.n_seqs + 1);
  const long long max_tokens = (long long)a.max_blocks << a.page_shift;
  const int per = (a.n_seqs + PLAN_MANY_THREADS - 1) / PLAN_MANY_THREADS;
  const int b0 = min(a.n_seqs, (int)threadIdx.x * per), b1 = min(a.n_seqs, b0 + per);
  bool ok = true;
  PlanSums mine{0, 0, 0};
  for (int b = b0; b < b1; ++b)
    mine = plan_add(mine, plan_counts(a.old_lens[b], a.new_lens[b], a.page_shift, max_tokens, ok));
  PlanSums at;
  const PlanSums total = plan_scan<PLAN_MANY_THREADS>(mine, at, s_warp);
  for (int b = b0; b < b1; ++b) {
    tok[b] = at.tok;
    take[b] = at.take;
    give[b] = at.give;
    at = plan_add(at, plan_counts(a.old_lens[b], a.new_lens[b], a.page_shift, max_tokens, ok));
  }
  ok = __syncthreads_and(ok) && plan_feasible(total, a.ring_in[0], a.ring_in[1], a.num_blocks, a.max_new);
  if (threadIdx.x == 0) {
    tok[a.n_seqs] = total.tok;
    take[a.n_seqs] = total.take;
    give[a.n_seqs] = total.give;
    ws[3 * ((size_t)a.n_seqs + 1)] = ok;
    if (!ok) flag_error(a.err, ERR_PLAN);
  }
}

__global__ void __launch_bounds__(PLAN_THREADS) plan_expand_kernel(PlanArgs a, const long long* ws) {
  const long long *tok = ws, *take = ws + a.n_seqs + 1, *give = ws + 2 * ((size_t)a.n_seqs + 1);
  const bool ok = ws[3 * ((size_t)a.n_seqs + 1)] != 0;
  const PlanSums total{tok[a.n_seqs], take[a.n_seqs], give[a.n_seqs]};
  if (blockIdx.y == PLAN_TOKENS) plan_tokens(a, tok, take, a.old_lens, total, ok, a.ring_in[0], a.ring_in[1]);
  else if (ok && blockIdx.y == PLAN_TAKES) plan_takes(a, take, a.old_lens, total.take, a.ring_in[0]);
  else if (ok) plan_gives(a, give, a.new_lens, total.give, a.ring_in[1]);
}

cudaError_t launch_plan_pages(const PageGeom& g, int n_seqs, const int32_t* old_lens, const int32_t* new_lens,
                              int32_t* table, int32_t* ring, const int64_t* ring_in, int64_t* ring_out, int max_new,
                              int32_t* cu_new, int64_t* slots, void* ws, unsigned* err, cudaStream_t s) {
  const PlanArgs a{n_seqs, g.page_tokens == 16 ? 4 : 3, g.num_blocks, g.max_blocks, max_new, old_lens, new_lens,
                   table, ring, reinterpret_cast<const long long*>(ring_in), reinterpret_cast<long long*>(ring_out),
                   cu_new, reinterpret_cast<long long*>(slots), err};
  const long long items = max_new > n_seqs ? max_new : n_seqs + 1;
  const int sms = device_sm_count();
  auto blocks = [&](int threads, int most) { return dim3((unsigned)std::min<long long>((items + threads - 1) / threads, most), PLAN_KINDS); };
  const int smem = 3 * (n_seqs + 1) * (int)sizeof(int);
  if (n_seqs <= PLAN_FEW) {
    plan_small_kernel<PLAN_THREADS><<<blocks(PLAN_THREADS, 2 * sms), PLAN_THREADS, smem, s>>>(a);
  } else if (n_seqs <= PLAN_SMALL) {
    static std::atomic<unsigned long long> attr{0};  // per device
    const cudaError_t e = smem_limit_once(attr, plan_small_kernel<PLAN_MANY_THREADS>, 3 * (PLAN_SMALL + 1) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    plan_small_kernel<PLAN_MANY_THREADS><<<blocks(PLAN_MANY_THREADS, std::max(1, sms / PLAN_KINDS)), PLAN_MANY_THREADS, smem, s>>>(a);
  } else {
    plan_scan_kernel<<<1, PLAN_MANY_THREADS, 0, s>>>(a, static_cast<long long*>(ws));
    plan_expand_kernel<<<blocks(PLAN_THREADS, 4 * sms), PLAN_THREADS, 0, s>>>(a, static_cast<const long long*>(ws));
  }
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Commit of an accepted path
// ---------------------------------------------------------------------------
constexpr int COMMIT_WARPS = 8;

__global__ void __launch_bounds__(32 * COMMIT_WARPS)
tree_commit_kernel(PageGeom g, int page_shift, int max_accept, int n_total, const int32_t* __restrict__ cu_q,
                   const int32_t* __restrict__ accepted, const int32_t* __restrict__ n_accepted,
                   const long long* __restrict__ slots, const int32_t* __restrict__ lens,
                   int32_t* __restrict__ new_lens, uint8_t* __restrict__ pool, unsigned* err) {
  const int b = blockIdx.x, h = blockIdx.y * COMMIT_WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int c0 = cu_q[b], n = cu_q[b + 1] - c0, len = lens[b], na = n_accepted[b];
  const bool shape_ok = c0 >= 0 && n >= 0 && c0 + (long long)n <= n_total && n <= len;
  bool ok = shape_ok && na >= 0 && na <= max_accept && na <= n;
  const int32_t* acc = accepted + (size_t)b * max_accept;
  if (ok) {
    bool mine = true;
    for (int i = lane; i < na; i += 32) mine = mine && acc[i] < n && acc[i] > (i ? acc[i - 1] : -1);
    ok = __all_sync(0xffffffffu, mine);
  }
  if (h == 0 && lane == 0) {
    new_lens[b] = shape_ok ? len - n + (ok ? na : 0) : (len > 0 ? len : 0);
    if (!ok) flag_error(err, ERR_TREE);
  }
  if (!ok || h >= g.n_kv_heads) return;
  const long long n_slots = (long long)g.num_blocks << page_shift;
  const int P = 1 << page_shift, part = lane & 7;
  // parts 0, 1: key codes; 2, 3: value codes; 4, 5: their (scale, zero); 6, 7: none
  const int width = part < 4 ? 32 : 4, base = part < 4 ? (part >> 1) * 32 * P + (part & 1) * 16 : 64 * P + (part - 4) * 4 * P;
  const int mask = P - 1;
  auto at = [&](long long slot) {
    return pool + ((size_t)(slot >> page_shift) * g.n_kv_heads + h) * g.record + base + width * (int)(slot & mask);
  };
  for (int i0 = 0; i0 < na; i0 += 32) {
    uint4 v[8];
    uint8_t* to[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + 4 * u + (lane >> 3);
      to[u] = nullptr;
      if (i >= na || acc[i] == i) continue;
      const long long src = slots[c0 + acc[i]], dst = slots[c0 + i];
      if (src < 0 || src >= n_slots || dst < 0 || dst >= n_slots) {
        flag_error(err, ERR_BLOCK_RANGE);
        continue;
      }
      if (part >= 6) continue;
      to[u] = at(dst);
      if (part < 4) v[u] = *reinterpret_cast<const uint4*>(at(src));
      else v[u].x = *reinterpret_cast<const uint32_t*>(at(src));
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (!to[u]) continue;
      if (part < 4) *reinterpret_cast<uint4*>(to[u]) = v[u];
      else *reinterpret_cast<uint32_t*>(to[u]) = v[u].x;
    }
    __syncwarp();
  }
}

cudaError_t launch_tree_commit(const PageGeom& g, int n_seqs, int n_total, int max_accept, const int32_t* cu_q,
                               const int32_t* accepted, const int32_t* n_accepted, const int64_t* slots,
                               const int32_t* lens, int32_t* new_lens, uint8_t* pool, unsigned* err, cudaStream_t s) {
  const dim3 grid(n_seqs, (g.n_kv_heads + COMMIT_WARPS - 1) / COMMIT_WARPS);
  tree_commit_kernel<<<grid, 32 * COMMIT_WARPS, 0, s>>>(g, g.page_tokens == 16 ? 4 : 3, max_accept, n_total, cu_q,
                                                        accepted, n_accepted,
                                                        reinterpret_cast<const long long*>(slots), lens, new_lens, pool,
                                                        err);
  return cudaGetLastError();
}

}  // namespace kvq
