// The paged INT2 cache read back: for every asked token and KV head
//   k = (z + s c) R_K^T + mu,   v = (z + s c) R_V^T
// (the write stored x = (k - mu) R_K and v R_V; R is orthogonal, so R^T takes it back).
//
// Rotated roles run on the tensor cores (read_rot_kernel): with centred codes, exact in
// fp16,
//   y_c = s sum_d (code_d - 1.5) R[c][d] + (z + 1.5 s) sum_d R[c][d] + mu_c
// is a [128 tokens x 128] x [128 x 128] product whose A operand comes from 32 bytes of
// codes a row, so scale and zero are applied to the accumulators.  A dense R enters as
// two fp16 limbs (hi, and the remainder) of R 2^e, e putting its largest element at
// 2^13 to 2^14: 22 bits and more, as fp32 has to be met.  A Hadamard matrix is +-1, exact in
// one limb with the signs; 1 / sqrt(128) is a factor of the result.
// The order of the channels inside the product is free as long as codes and R agree on
// it: a 32-bit word's fields f of both halves (channels 16 w + f and 16 w + 8 + f) go
// side by side, which makes a register of the operand out of one mask and one FMA.
//
// A CTA of 256 threads (two an SM) has one role and head, R staged once, and every n-th
// 128-token tile, so that all heads' rows of a token go out at about the same time (a run of
// tiles each: 1 us more, Hadamard 5).  A thread owns half of a token's row from its codes to
// its stores, so that pages, scales and zeros never leave its registers and the codes go
// straight into tensor memory.  A tile's product runs while its threads expand the next
// tile's codes (two A buffers), load those of the one after, and, once its accumulators are
// in registers, finish and store them beside the next product: through shared memory by bulk
// tensor copies, or, where a tile has rows that keep their content, by the threads (a
// thread's own row, 32 bytes at a time, filled the load-store pipe: 102 us where the copies
// take 85).
// Bound: HBM, 72 bytes in and 512 (bf16) or 1,024 out a token and head; the dense product is
// 2 x 4.2 MFLOP a tile, below the time of its bytes.  65,536 tokens of 8 heads in bf16 take
// 74.6 us dense (4.1 TB/s: its warps wait for tensor memory, pages and one another at the tile's
// barrier), 67 Hadamard, 59 identity (read_plain_kernel); in fp32 32,768 tokens dense 57.
// Its sequence kept from tile to tile saves a search a row (81 and 72); row sums and means read from
// shared memory are 5 of the 75, the table's latency 7.  Not kept: warps of their own for expansion and output, one
// CTA an SM (86 to 101 us dense); the pages looked up a tile earlier (87).
#include <algorithm>

#include "quant_common.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"

namespace kvq {

constexpr int RC_THREADS = 256;
constexpr int RC_TILE = 128 * 128 * 2;  // a limb of R: two K halves of 128 rows of 128 bytes
constexpr uint32_t RC_COLUMNS = 256;     // tensor memory: the accumulator, then two buffers of 64 columns of codes
constexpr int RC_HALF = RC_TILE / 2;

struct RcRole {
  RotDev rot;
  const float* mu;
  void* out;
  int codes_off, meta_off;
};

struct RcArgs {
  PageGeom g;
  int n_seqs, n_total, n_roles, page_shift;
  const int32_t* cu;
  const int32_t* start;
  const int32_t* table;
  const uint8_t* pool;
  RcRole role[2];
  unsigned* err;
  CUtensorMap out[2];  // [n_total][H][128] in boxes of 128 rows of one head, 128 bytes wide
};

// The sequence whose rows a thread reads: rows [lo, hi), the first at position `start`.
struct RcSeq {
  int b = 0, lo = 0, hi = 0, start = 0;
};
// The page id and slot of row t; false (row left as it was) for a row of no sequence or, flagged, a bad position.
__device__ __forceinline__ bool rc_page(const RcArgs& a, int t, RcSeq& q, int* id, int* slot) {
  if (t < q.lo || t >= q.hi) {
    if (t < __ldg(a.cu) || t >= __ldg(a.cu + a.n_seqs)) return false;
    int b = 0, end = a.n_seqs;  // cu[b] <= t < cu[end]
    while (end - b > 1) {
      const int mid = (b + end) >> 1;
      if (__ldg(a.cu + mid) <= t) b = mid; else end = mid;
    }
    q = RcSeq{b, __ldg(a.cu + b), __ldg(a.cu + b + 1), __ldg(a.start + b)};
  }
  const long long pos = (long long)q.start + (t - q.lo), page = pos >> a.page_shift;
  if (pos < 0 || page >= a.g.max_blocks) {
    flag_error(a.err, ERR_POS_RANGE);
    return false;
  }
  *id = __ldg(a.table + (size_t)q.b * a.g.max_blocks + page);
  *slot = (int)pos & ((1 << a.page_shift) - 1);
  return true;
}
// The page's record of a head, nullptr, flagged, for a bad id.
__device__ __forceinline__ const uint8_t* rc_record(const RcArgs& a, int id, int h) {
  if ((unsigned)id >= (unsigned)a.g.num_blocks) {
    flag_error(a.err, ERR_BLOCK_RANGE);
    return nullptr;
  }
  return a.pool + ((size_t)id * a.g.n_kv_heads + h) * a.g.record;
}

__device__ __forceinline__ uint32_t rc_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 codes of a word -> 8 registers of two centred fp16 (fields f of the low and the high half).  A field at bit 2 p of
// 16 with the exponent of 1024 above it is 1024 + c 4^p; p = 1 .. 4 keep 1024 4^-p + 1.5 representable.
__device__ __forceinline__ void rc_expand(uint32_t w, uint32_t (&r)[8]) {
  const uint32_t src[8] = {w << 2, w, w, w, w, w >> 6, w >> 6, w >> 6};
  constexpr int P[8] = {1, 1, 2, 3, 4, 2, 3, 4};
#pragma unroll
  for (int f = 0; f < 8; ++f) {
    const int p = P[f];
    const uint32_t v = (src[f] & (0x00030003u << (2 * p))) | 0x64006400u;
    const float inv = 1.f / (float)(1 << (2 * p));
    const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&v), __float2half2_rn(inv),
                              __float2half2_rn(-(1024.f * inv + 1.5f)));
    r[f] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

// 32 consecutive columns of this thread's lane.
__device__ __forceinline__ void rc_tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// fp16 A and B (both K-major), fp32 D, 128 x 128.
constexpr uint32_t RC_IDESC = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

__host__ __device__ constexpr int rc_smem(bool dense) { return 1024 + RC_TILE * (dense ? 3 : 2); }  // R's limbs, the rows on their way out

// D[tmem] (+)= A[tmem] B[smem]^T, by one thread.
__device__ __forceinline__ void rc_mma(uint32_t d, uint32_t a, uint64_t b_desc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(RC_IDESC), "r"((uint32_t)accumulate)
      : "memory");
}
// 8 columns of this thread's lane.
__device__ __forceinline__ void rc_tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void rc_store_box(const CUtensorMap* map, int channel, int head, int row, const void* src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(channel),
               "r"(head), "r"(row), "r"(smem_u32(src))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The copies of this thread have read their shared memory.
__device__ __forceinline__ void rc_copies_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
// The four warps of a half meet; whether any of them says so.
__device__ __forceinline__ bool rc_any(int half, bool p) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"((uint32_t)p), "r"(1 + half)
      : "memory");
  return any != 0;
}

template <bool DENSE, bool F32>
__global__ void __launch_bounds__(RC_THREADS, 2) read_rot_kernel(const __grid_constant__ RcArgs a) {
  extern __shared__ uint8_t rc_raw[];
  uint8_t* sB = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(rc_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(16) float s_sum[D];  // sum_d R[c][d]
  __shared__ __align__(16) float s_mu[D];
  __shared__ float s_max[RC_THREADS / 32];
  __shared__ __align__(8) uint64_t s_bar;
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int r = tid & 127, half = tid >> 7;  // the thread's row, and which 64 of its channels
  uint8_t* sO = sB + RC_TILE * (DENSE ? 2 : 1) + half * RC_HALF;  // the half's rows on their way out
  const int H = a.g.n_kv_heads;
  // the block's role and head; its tiles are first, first + step ..
  const int tiles = (a.n_total + 127) / 128, rhs = a.n_roles * H, step = gridDim.x / rhs;
  const int rh = blockIdx.x % rhs, first = blockIdx.x / rhs, n = (tiles - first + step - 1) / step;
  const int h = rh % H;
  const RcRole& ro = a.role[rh / H];
  if (tid == 0) {
    mbar_init(&s_bar, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, RC_COLUMNS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem, lanes = (uint32_t)(32 * (warp & 3)) << 16;

  struct Row {
    uint4 codes;
    uint32_t meta;
    bool ok;
  };
  RcSeq seq;
  auto fetch = [&](int i) {  // of the i-th tile
    Row x{make_uint4(0, 0, 0, 0), 0, false};
    const int t = (first + i * step) * 128 + r;
    if (i >= n || t >= a.n_total) return x;
    int id, slot;
    const uint8_t* rec = rc_page(a, t, seq, &id, &slot) ? rc_record(a, id, h) : nullptr;
    x.ok = rec;
    if (x.ok) {
      x.codes = __ldg(reinterpret_cast<const uint4*>(rec + ro.codes_off + GROUP_BYTES * slot) + half);
      x.meta = __ldg(reinterpret_cast<const uint32_t*>(rec + ro.meta_off) + slot);
    }
    return x;
  };
  auto expand = [&](const Row& x, int buf) {
    const uint32_t w[4] = {x.codes.x, x.codes.y, x.codes.z, x.codes.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t v[8];
      rc_expand(w[j], v);
      rc_tmem_st8(tmem + lanes + 128 + 64 * buf + 32 * half + 8 * j, v);
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
  };
  float down = 1.f;  // what the products are scaled back by
  auto stage = [&]() {  // the head's R, with its row sums and the mean
    if constexpr (DENSE) {
      // a warp a row, a lane four channels; warp w has rows 16 w and on
      const int c0 = 16 * warp, lane = tid & 31;
      const float4* R = reinterpret_cast<const float4*>(ro.rot.dense + (size_t)h * D * D) + c0 * (D / 4) + lane;
      float4 x[16];
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __ldg(R + i * (D / 4));
#pragma unroll
      for (int i = 0; i < 16; ++i)
        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(x[i].x), fabsf(x[i].y)), fmaxf(fabsf(x[i].z), fabsf(x[i].w))));
      mx = warp_max(mx);
      if (lane == 0) s_max[warp] = mx;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < RC_THREADS / 32; ++i) mx = fmaxf(mx, s_max[i]);
      // R 2^e: its largest element in [2^13, 2^14)
      const int e = mx > 0.f && mx < INFINITY ? min(100, max(-100, 13 - ilogbf(mx))) : 0;
      const float up = exp2f((float)e);
      down = exp2f((float)-e);
      // Lanes m = 0 .. 3 of a 16-channel word have channels 4 m and on.  Channels k and k + 8 go side by side: lane m and lane
      // m ^ 2 exchange theirs, then lanes 0 and 1 write the word's two chunks of the first limb, lanes 2 and 3 those of the remainder.
      const bool rest = lane & 2;
      const int chunk = 2 * (lane >> 2) + (lane & 1);
      uint8_t* to = sB + (rest ? RC_TILE : 0) + (chunk >> 3) * RC_HALF;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int c = c0 + i;
        const float sum = warp_sum((x[i].x + x[i].y) + (x[i].z + x[i].w));
        if (lane == 0) s_sum[c] = sum;
        const float own[4] = {x[i].x * up, x[i].y * up, x[i].z * up, x[i].w * up};
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float other = __shfl_xor_sync(0xffffffffu, own[k], 2);
          const float lo = rest ? other : own[k], hi = rest ? own[k] : other;
          w[k] = rc_half2(lo, hi);
          const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          if (rest) w[k] = rc_half2(lo - hf.x, hi - hf.y);
        }
        *reinterpret_cast<uint4*>(to + c * 128 + (((chunk & 7) ^ (c & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {  // sign_c H: row 0 is the only one whose sum is not zero
      const float sign = __ldg(ro.rot.signs + (size_t)h * D + r);
      const uint32_t flip = sign < 0.f ? 0x80008000u : 0u;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = 64 * half + 16 * (c / 2) + 4 * (c % 2) + i;
          w[i] = flip ^ (((__popc(r & k) & 1) ? 0xbc00u : 0x3c00u) | ((__popc(r & (k + 8)) & 1) ? 0xbc000000u : 0x3c000000u));
        }
        *reinterpret_cast<uint4*>(sB + half * RC_HALF + r * 128 + ((c ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (half == 0) s_sum[r] = r == 0 ? sign * 11.313708498984761f : 0.f;
      down = 0.08838834764831845f;
    }
    if (tid < D) s_mu[tid] = ro.mu ? __ldg(ro.mu + (size_t)h * D + tid) : 0.f;
    fence_proxy_async();  // the tensor cores read R through the async proxy
  };
  auto issue = [&](int buf) {  // thread 0
    tc_fence_after();
    const uint64_t bd = sw128_desc(sB);
#pragma unroll
    for (int limb = DENSE ? 1 : 0; limb >= 0; --limb)  // the remainder first
#pragma unroll
      for (int k = 0; k < 8; ++k)
        rc_mma(tmem, tmem + 128 + 64 * buf + 8 * k,
               bd + (uint64_t)(limb * (RC_TILE >> 4) + (k >> 2) * (RC_HALF >> 4) + 2 * (k & 3)), k > 0 || (DENSE && limb == 0));
    tc_commit(&s_bar);
  };

  Row cur{}, nxt{};
  if (n > 0) {
    cur = fetch(0);
    stage();
    nxt = fetch(1);
    expand(cur, 0);
    tc_fence_before();
    __syncthreads();
    if (tid == 0) issue(0);
  }
  for (int i = 0; i < n; ++i) {
    const uint32_t meta_next = nxt.meta;
    const bool ok_next = nxt.ok;
    // while the product runs: the codes of the next tile into the other buffer, those of the one after on their way
    expand(nxt, (i + 1) & 1);
    nxt = fetch(i + 2);
    const bool done = mbar_wait_bounded(&s_bar, i & 1);
    tc_fence_after();
    float acc[64];
    rc_tmem_ld32(tmem + lanes + 64 * half, *reinterpret_cast<float(*)[32]>(acc));
    rc_tmem_ld32(tmem + lanes + 64 * half + 32, *reinterpret_cast<float(*)[32]>(acc + 32));
    tc_fence_before();
    if (__syncthreads_or(!done)) {
      if (tid == 0) flag_error(a.err, ERR_TIMEOUT);
      break;
    }
    if (i + 1 < n && tid == 0) issue((i + 1) & 1);
    // ---- scale, zero, mean; the row's 64 channels out ----
    const __half2 sz = *reinterpret_cast<const __half2*>(&cur.meta);
    const float sc = __low2float(sz), mid = fmaf(1.5f, sc, __high2float(sz));
    const float sd = sc * down;
    const uint64_t sd2 = f2pk(sd, sd), mid2 = f2pk(mid, mid);
    const int t0 = (first + i * step) * 128, t = t0 + r;
    const size_t out = ((size_t)t * H + h) * D + 64 * half;
    constexpr int ROUNDS = F32 ? 2 : 1, WIDTH = 64 / ROUNDS;  // 128 bytes of a row a round
#pragma unroll
    for (int round = 0; round < ROUNDS; ++round) {
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < WIDTH; j += 4) {
        const int c = round * WIDTH + j;
        float4 s4 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (DENSE || c == 0) s4 = *reinterpret_cast<const float4*>(s_sum + 64 * half + c);
        float4 m4 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ro.mu) m4 = *reinterpret_cast<const float4*>(s_mu + 64 * half + c);
        const uint64_t s2[2] = {f2pk(s4.x, s4.y), f2pk(s4.z, s4.w)}, m2[2] = {f2pk(m4.x, m4.y), f2pk(m4.z, m4.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint64_t x2 = f2pk(acc[c + 2 * e], acc[c + 2 * e + 1]);
          const float2 y = f2up(f2fma(sd2, x2, f2fma(mid2, s2[e], m2[e])));
          if constexpr (F32) {
            w[j + 2 * e] = __float_as_uint(y.x);
            w[j + 2 * e + 1] = __float_as_uint(y.y);
          } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(y.x, y.y);
            w[j / 2 + e] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
      }
      if (r == 0) rc_copies_read();
      if (rc_any(half, !cur.ok && t < a.n_total)) {
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(ro.out) + (out + round * WIDTH) * (F32 ? 4 : 2));
        if (cur.ok) {
#pragma unroll
          for (int c = 0; c < 8; ++c) p[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(sO + r * 128 + ((c ^ (r & 7)) << 4)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        fence_proxy_async();
        rc_any(half, false);
        if (r == 0) rc_store_box(&a.out[rh / H], 64 * half + round * WIDTH, h, t0, sO);
      }
    }
    cur.meta = meta_next;
    cur.ok = ok_next;
  }
  if (r == 0) rc_copies_read();  // shared memory goes with the block
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, RC_COLUMNS);
}

// 32 bytes to a 32-byte boundary (wide) or a 16-byte one.
__device__ __forceinline__ void rc_store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A role without a rotation.  A warp has `tokens` tokens (32 at most), each looked up once by a lane, and writes their rows in
// the order of memory: 8 lanes a (token, head), 16 channels a lane, four of them at once.  The mean stands in shared memory
// in the order in which a warp reads it (read from global memory beside the stores it took 20 of 74 us).  A 2-bit field
// masked in place under the right exponent is 2^(23 - bit) + c as fp32, exactly.  65,536 tokens of 8 heads: 59.4 us in bf16,
// 5.2 TB/s (a lane one, two, four (token, head)s ahead 61.5, 59.4, 60.5 us; two, four, eight tokens a warp 67.6, 59.4, 58.0, in
// fp32 with half the tokens 49.1, 49.4, 58.1).
constexpr int RC_HEADS = 32;  // heads a block at most

template <bool F32>
__global__ void __launch_bounds__(RC_THREADS) read_plain_kernel(const __grid_constant__ RcArgs a, int tokens, bool wide) {
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int AHEAD = 2;  // (token, head)s of a lane whose loads are in flight
  __shared__ float4 s_mean[RC_HEADS][4][8];
  const int H = a.g.n_kv_heads, lane = threadIdx.x & 31, w = lane & 7, sub = lane >> 3, parts = (H + RC_HEADS - 1) / RC_HEADS;
  const RcRole& ro = a.role[blockIdx.y / parts];
  const int h0 = blockIdx.y % parts * RC_HEADS, heads = min(RC_HEADS, H - h0);
  const long long t0 = ((long long)blockIdx.x * (RC_THREADS / 32) + (threadIdx.x >> 5)) * tokens;
  const int n = (int)max(0ll, min((long long)tokens, a.n_total - t0));
  const uint8_t* rec = nullptr;
  int id, slot = 0;
  RcSeq seq;
  if (lane < n && rc_page(a, (int)t0 + lane, seq, &id, &slot)) rec = rc_record(a, id, h0);
  if (ro.mu) {
    for (int i = threadIdx.x; i < heads * 32; i += RC_THREADS)
      s_mean[i >> 5][i & 3][(i >> 2) & 7] = __ldg(reinterpret_cast<const float4*>(ro.mu + (size_t)h0 * D) + i);
    __syncthreads();
  }
  // this lane's (token, head)s: sub, sub + 4 ..
  const int step_t = 4 / heads, step_h = 4 - step_t * heads;
  int tok = sub / heads, h = sub - tok * heads;
  auto next = [&](int& t, int& i) {
    t += step_t;
    i += step_h;
    if (i >= heads) {
      i -= heads;
      ++t;
    }
  };
  const bool mean = ro.mu != nullptr;
  for (int p0 = 0; p0 < n * heads; p0 += 4 * AHEAD) {
    uint32_t codes[AHEAD], meta[AHEAD];
    int at[AHEAD];  // head, -1: nothing to write
    int row[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const uint8_t* r = reinterpret_cast<const uint8_t*>(__shfl_sync(FULL, (unsigned long long)rec, tok & 31));
      const int s = __shfl_sync(FULL, slot, tok & 31);
      at[i] = tok < n && r ? h : -1;
      row[i] = tok;
      codes[i] = meta[i] = 0;
      if (at[i] >= 0) {
        r += (size_t)h * a.g.record;
        codes[i] = __ldg(reinterpret_cast<const uint32_t*>(r + ro.codes_off + GROUP_BYTES * s) + w);
        meta[i] = __ldg(reinterpret_cast<const uint32_t*>(r + ro.meta_off) + s);
      }
      next(tok, h);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (at[i] < 0) continue;
      const __half2 sz = *reinterpret_cast<const __half2*>(&meta[i]);
      const float s = __low2float(sz), z = __high2float(sz);
      const uint64_t s2 = f2pk(s, s);
      const size_t out = ((size_t)(t0 + row[i]) * H + h0 + at[i]) * D + 16 * w;
      constexpr int RUN = F32 ? 8 : 16;  // channels in 32 bytes
#pragma unroll
      for (int c = 0; c < 16; c += RUN) {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < RUN; j += 4) {
          float4 m4 = make_float4(0.f, 0.f, 0.f, 0.f);
          if (mean) m4 = s_mean[at[i]][(c + j) / 4][w];
          const uint64_t m2[2] = {f2pk(m4.x, m4.y), f2pk(m4.z, m4.w)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int bit = 2 * (c + j + 2 * e), b = bit < 20 ? bit : bit - 16;  // of the first of two fields
            const uint32_t x = bit < 20 ? codes[i] : codes[i] >> 16;
            const uint32_t lo = (x & (3u << b)) | ((150u - b) << 23), hi = (x & (12u << b)) | ((148u - b) << 23);
            const uint64_t k = f2add(f2pk(__uint_as_float(lo), __uint_as_float(hi)),
                                     f2pk(-(float)(1 << (23 - b)), -(float)(1 << (21 - b))));
            const float2 y = f2up(f2add(f2fma(s2, k, f2pk(z, z)), m2[e]));
            if constexpr (F32) {
              v[j + 2 * e] = __float_as_uint(y.x);
              v[j + 2 * e + 1] = __float_as_uint(y.y);
            } else {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(y.x, y.y);
              v[j / 2 + e] = *reinterpret_cast<const uint32_t*>(&b2);
            }
          }
        }
        rc_store32(static_cast<uint8_t*>(ro.out) + (out + c) * (F32 ? 4 : 2), v, wide);
      }
    }
  }
}

// The output of a role as a tensor of boxes.
static bool rc_map(CUtensorMap* map, const RcArgs& a, const void* out, bool f32) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t row = D * (f32 ? 4 : 2), H = (cuuint64_t)a.g.n_kv_heads;
  const cuuint64_t dims[3] = {D, H, (cuuint64_t)a.n_total}, strides[2] = {row, row * H};
  const cuuint32_t box[3] = {f32 ? 32u : 64u, 1, 128}, one[3] = {1, 1, 1};
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(out), dims,
             strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool DENSE, bool F32>
static cudaError_t rc_launch_rot(RcArgs& a, cudaStream_t s) {
  for (int i = 0; i < a.n_roles; ++i)
    if (!rc_map(&a.out[i], a, a.role[i].out, F32)) return cudaErrorNotSupported;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = smem_limit_once(done, read_rot_kernel<DENSE, F32>, rc_smem(DENSE));
  if (e != cudaSuccess) return e;
  // the same number of blocks for each head of each role, side by side, so that all heads' rows of a token go out at about
  // the same time (rounded down: two roles of 32 heads take 256 of 304 places, of 80 heads 160)
  const int rhs = a.n_roles * a.g.n_kv_heads, tiles = (a.n_total + 127) / 128;
  const int grid = rhs * std::min(tiles, std::max(1, 2 * device_sm_count() / rhs));
  read_rot_kernel<DENSE, F32><<<grid, RC_THREADS, rc_smem(DENSE), s>>>(a);
  return cudaGetLastError();
}

template <bool F32>
static cudaError_t rc_launch_plain(const RcArgs& a, cudaStream_t s) {
  // four tokens a warp unless that leaves SMs idle
  const int tokens = a.n_total >= 4 * (RC_THREADS / 32) * 2 * device_sm_count() ? 4 : 1;
  const long long blocks = ((long long)a.n_total + tokens * (RC_THREADS / 32) - 1) / (tokens * (RC_THREADS / 32));
  const dim3 grid((unsigned)blocks, (unsigned)(a.n_roles * ((a.g.n_kv_heads + RC_HEADS - 1) / RC_HEADS)));
  // 32-byte stores where both outputs allow them: of two 16-byte ones side by side each takes half of
  // every 32-byte sector (65,536 tokens of 8 heads, an earlier kernel: 92 against 171 us in fp32, 73 against 80 in bf16)
  uintptr_t low = 0;
  for (int i = 0; i < a.n_roles; ++i) low |= reinterpret_cast<uintptr_t>(a.role[i].out);
  read_plain_kernel<F32><<<grid, RC_THREADS, 0, s>>>(a, tokens, (low & 31) == 0);
  return cudaGetLastError();
}

cudaError_t launch_read_cache(const PageGeom& g, int n_seqs, int n_total, const int32_t* cu, const int32_t* start,
                              const int32_t* table, RotDev rot_k, RotDev rot_v, const float* mu_k, const uint8_t* pool,
                              void* k, void* v, int dtype, unsigned* err, cudaStream_t s) {
  const int P = g.page_tokens;
  const RcRole role[2] = {{rot_k, mu_k, k, 0, 64 * P}, {rot_v, nullptr, v, 32 * P, 68 * P}};
  const bool f32 = dtype == KVQ_F32;
  // one launch a kind of rotation
  for (int kind : {KVQ_ROT_DENSE, KVQ_ROT_SIGNED_HADAMARD, KVQ_ROT_IDENTITY}) {
    RcArgs a{g, n_seqs, n_total, 0, P == 16 ? 4 : 3, cu, start, table, pool, {}, err, {}};
    for (const RcRole& r : role)
      if (r.out && r.rot.kind == kind) a.role[a.n_roles++] = r;
    if (!a.n_roles) continue;
    cudaError_t e;
    if (kind == KVQ_ROT_DENSE) e = f32 ? rc_launch_rot<true, true>(a, s) : rc_launch_rot<true, false>(a, s);
    else if (kind == KVQ_ROT_SIGNED_HADAMARD) e = f32 ? rc_launch_rot<false, true>(a, s) : rc_launch_rot<false, false>(a, s);
    else e = f32 ? rc_launch_plain<true>(a, s) : rc_launch_plain<false>(a, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kvq
