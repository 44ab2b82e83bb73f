// Decode attention with capped scores, a distance bias, a sliding window and a prefix
// (kvq_decode_attention_score): one query a sequence over the paged INT2 cache.
//
//   q' = q R_K;  a_s = q'.(z_s + s_s c_s) / sqrt(128);  a_s <- cap tanh(a_s / cap) - slope |t - s|
//   over the visible s:  p = softmax(a),  o = sum_s p_s (z_s + s_s c_s)      (rotated-V basis)
//
// Only what is visible is read: a sequence's list holds the 64-token entries of its
// prefix and of its window.  As in kvq_decode_attention, the whole batch's list is cut
// into one equal slice a warp, whatever the lengths; a warp streams its entries through
// shared memory (three stages of 64 tokens, one bulk copy a page), runs both products
// as mma.sync on the packed 2-bit codes and leaves a partial softmax for every
// (sequence, KV head) that its slice touches, which ds_combine_kernel joins in slice
// order (results do not depend on timing).
//
// Products.  A 2-bit field masked in place at bit p of a 16-bit word is the fp16
// subnormal c 2^(p - 24): one logical operation for two codes, the power of two taken up
// by the query or by the output.  The tensor cores align a product by the exponent that
// its operands are written with, 2^-14 for every subnormal, so a field at bit p loses
// 10 - p bits of their adder (measured: 128-term sums off by 1.3e-6 with p = 0 .. 8,
// 2e-8 with normal operands).  Keys are therefore shifted to bits 4, 6 and 8 (two shifts a
// word), values, whose sums run on over a whole slice, to 7 and 9 (five): readouts of 1,000
// tokens 4.6e-6 -> 9e-7 off fp64, of 16,384 5.4e-6 -> 2.7e-6, for 2 us of 60 there (all
// values at bit 9: 2.5e-6, 2 us more; keys at 7 and 9 change nothing).  Queries and weights
// enter as two fp16 halves side by side in two columns (22 bits).  Values enter as (c, w)
// and (3 - c, -w) in turn, so that the common part of the sums cancels between
// neighbouring tiles instead of growing.  The tensor cores truncate what they add up: every
// 256 tokens the sums go to fp32 sums in tensor memory, which nothing else here uses (at 16,384
// tokens 2.7e-6 -> 1.2e-6 off, 59.5 -> 61.8 us; every 512 tokens 1.7e-6, 61.5 us).  The weights
// change from a lane a token to a lane a column by matrix transposes (shuffles and selections
// instead: 2 us more).  A weight times its value scale has to fit fp16: the reference that scores
// are taken from moves when it does not (scales over 512), and lies below the maximum where all
// scales are tiny (weight_lift); looking at it in every chunk costs 0.7 of 60 us on the
// device (1.3 of 63.7 a call).
//
// Bound: a warp's chain of products, fields and weights, four warps a scheduler (58 % of the
// issue slots; without the work the call took 39 us, without the copies alone 61, without
// both 23): 16 x 16,384 tokens, 32 / 8 heads in 61.1 us, 2.5 TB/s of cache.  A
// cap adds 9 operations a score, and 6 more only where a warp's scores pass 0.8 of it:
// 63.7 us.  Ragged lengths and windows cost nothing but their entries: 64 sequences of up to
// 8,192 tokens, 40 / 10 heads, 64 + 1,024 seen, 31.1 us.
#include <type_traits>

#include "async_copy.cuh"
#include "quant_common.cuh"
#include "score.cuh"
#include "tcgen05.cuh"

namespace kvq {

constexpr float DS_LOG2E = 1.4426950408889634f;
constexpr int DS_STAGES = 3;
constexpr float DS_TAU = 6.f;        // a reference maximum moves once a score passes it by 2^6
constexpr float DS_LO = 2048.f;      // second halves are held times 2^11
// Scores are taken over the cap, if there is one: in units 2^k of it for a row whose scale would pass 2^60 of it, as scores
// that fp32 can tell from 0 are then far past the cap either way.  Without a cap rows over 2^59 have theirs in units of 2^64,
// and say so by a negative scale.  Neither a score's terms nor their scale then pass fp32.
constexpr float DS_FAR = 0x1p64f;
constexpr int DS_PART = D + 4;       // acc[128], m (base 2), l, 2 unused
constexpr int DS_PREP_THREADS = 256;

__host__ __device__ constexpr int ds_tiles(int gqa) { return (gqa + 3) / 4; }           // MMA column tiles, 2 columns a head
__host__ __device__ constexpr int ds_max_warps(int gqa) { return gqa >= 8 ? 12 : 16; }  // of an SM's one block (registers)
constexpr int DS_FLUSH = 4;  // entries after which a warp's sums go to tensor memory
// Tensor memory columns of a block of `warps` warps: 32 for each column tile of the warps that share a quarter of its lanes.
__host__ __device__ constexpr int ds_columns(int gqa, int warps) {
  const int need = warps / 4 * 32 * ds_tiles(gqa);
  return need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : 256;
}
constexpr int DS_WARP_SMEM = DS_STAGES * 64 * 72;

// How far a half word's field f (bits 2 f, 2 f + 1) is shifted up, and the bit at which it is then masked: 4, 6 or 8 for
// keys, 7 or 9 for values, 9 for all of them where few warps are at work (fine).
__host__ __device__ constexpr int ds_key_shift(int f) { return f < 2 ? 6 : f < 5 ? 0 : -6; }
__host__ __device__ constexpr int ds_value_shift(int f, bool fine) {
  return fine || f == 0 ? 9 - 2 * f : f <= 2 ? 5 : f <= 4 ? 1 : f <= 6 ? -3 : -5;
}
__host__ __device__ constexpr int ds_key_bit(int f) { return 2 * f + ds_key_shift(f); }
__host__ __device__ constexpr int ds_value_bit(int f, bool fine) { return 2 * f + ds_value_shift(f, fine); }

struct DsWs {
  float* part;      // [warps + units][gqa][132]: the partial of warp w for unit u at w + u
  uint32_t* qfrag;  // [units][16 * tiles][32]
  float2* qsum;     // [units][gqa] (scale of the products, sum of q'), in the row's units: see DS_FAR
  int2* span;       // [units] the slices that meet the unit
};

static size_t ds_align(size_t x) { return (x + 255) & ~size_t(255); }

static size_t ds_layout(void* base, int units, int gqa, int warps, DsWs* out) {
  const size_t o_frag = ds_align((size_t)(warps + units) * gqa * DS_PART * sizeof(float));
  const size_t o_sum = ds_align(o_frag + (size_t)units * 16 * ds_tiles(gqa) * 32 * sizeof(uint32_t));
  const size_t o_span = ds_align(o_sum + (size_t)units * gqa * sizeof(float2));
  if (out) {
    char* p = static_cast<char*>(base);
    out->part = reinterpret_cast<float*>(p);
    out->qfrag = reinterpret_cast<uint32_t*>(p + o_frag);
    out->qsum = reinterpret_cast<float2*>(p + o_sum);
    out->span = reinterpret_cast<int2*>(p + o_span);
  }
  return ds_align(o_span + (size_t)units * sizeof(int2));
}

struct DsArgs {
  PageGeom g;
  int n_seqs, n_q_heads, max_len;
  const int32_t* lens;
  const int32_t* table;
  const uint8_t* pool;
  ScoreDev score;
  DsWs ws;
  float* out;
  unsigned* err;
};

// What a sequence's query sees: positions [0, prefix) and [lo, len), as 64-token entries: the first n_pre of them, then,
// `jump` further on, the rest of n.
struct DsView {
  int len, prefix, lo, n_pre, jump, n;
  __device__ __forceinline__ int first_token(int i) const { return 64 * (i < n_pre ? i : i + jump); }
};
__device__ __forceinline__ DsView ds_view(const DsArgs& a, int b, unsigned* err = nullptr) {
  DsView v{__ldg(a.lens + b), 0, 0, 0, 0, 0};
  if (v.len < 0 || v.len > a.max_len) {
    flag_error(err, ERR_SEQ_RANGE);
    v.len = 0;
  }
  if (a.score.prefix) v.prefix = min(max(__ldg(a.score.prefix + b), 0), v.len);
  v.lo = max(0, v.len - a.score.window);
  v.n_pre = (v.prefix + 63) >> 6;
  const int first = max(v.n_pre, v.lo >> 6);
  v.jump = first - v.n_pre;
  v.n = v.n_pre + max(0, ((v.len + 63) >> 6) - first);
  return v;
}

__device__ __forceinline__ uint32_t ds_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// floor(log2 x) of a normal x (of a subnormal one -127), and 2^e, e in -126 .. 127.
__device__ __forceinline__ int ds_exponent(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }
__device__ __forceinline__ float ds_pow2(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }
__device__ __forceinline__ float ds_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ds_tmem_st8(uint32_t taddr, const float (&v)[8]) {  // 8 columns of this thread's lane
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void ds_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A field of both halves of four words, in place for the product.
template <bool COMPLEMENT>
__device__ __forceinline__ void ds_field(int shift, int bit, const uint32_t (&w)[4], uint32_t (&a)[4]) {
  const uint32_t mask = 0x00030003u << bit;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t src = shift >= 0 ? w[x] << shift : w[x] >> -shift;
    a[x] = COMPLEMENT ? ~src & mask : src & mask;
  }
}
__device__ __forceinline__ uint32_t ds_transpose(uint32_t x) {  // an 8 x 8 matrix of 16-bit elements, a row's pair a lane
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

// ---------------------------------------------------------------------------
// The queries: rotated, scaled to base-2 scores, as the B operand of q'.c; one CTA a KV
// head and run of sequences (a dense R stays in registers).
// ---------------------------------------------------------------------------
template <int G, bool DENSE>
__global__ void __launch_bounds__(DS_PREP_THREADS) ds_prepare_kernel(const __grid_constant__ DsArgs a, const void* q,
                                                                     int dtype, RotDev rot, int seqs_per_cta) {
  constexpr int NT = ds_tiles(G), NW = DS_PREP_THREADS / 32;
  pdl_launch_dependents();  // the decode kernel lists its work and starts its copies meanwhile
  __shared__ __align__(16) float qv[G][D];
  __shared__ __align__(16) float red[DENSE ? NW : 1][G][D];
  __shared__ int s_exp[G];
  const int h = blockIdx.x, H = a.g.n_kv_heads, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr float SCALE = DS_LOG2E * INV_SQRT_D;
  float4 r[16];  // warp w: rows 16 w .. of R, lane: columns 4 l ..
  if (DENSE) {
    const float4* R = reinterpret_cast<const float4*>(rot.dense + (size_t)h * D * D) + lane;
#pragma unroll
    for (int c = 0; c < 16; ++c) r[c] = __ldg(R + (16 * warp + c) * (D / 4));
  }
  for (int si = 0; si < seqs_per_cta; ++si) {
    const int b = blockIdx.y * seqs_per_cta + si;
    if (b >= a.n_seqs) break;
    const int u = b * H + h;
    __syncthreads();  // the last sequence's rows have been read
    const size_t row0 = ((size_t)b * a.n_q_heads + h * G) * D;
    if (DENSE) {
      for (int i = tid; i < G * D; i += DS_PREP_THREADS) qv[i / D][i % D] = load1(q, row0 + i, dtype);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < G; ++j) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float x = qv[j][16 * warp + c];
          y.x = fmaf(x, r[c].x, y.x); y.y = fmaf(x, r[c].y, y.y); y.z = fmaf(x, r[c].z, y.z); y.w = fmaf(x, r[c].w, y.w);
        }
        reinterpret_cast<float4*>(red[warp][j])[lane] = y;
      }
      __syncthreads();
      for (int i = tid; i < G * D; i += DS_PREP_THREADS) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) y += red[w][i / D][i % D];
        qv[i / D][i % D] = y * SCALE;
      }
    } else {
      for (int j = warp; j < G; j += NW) {
        float4 x = rotate_vec_warp(load4(q, row0 + (size_t)j * D + 4 * lane, dtype), rot, h, lane, false);
        reinterpret_cast<float4*>(qv[j])[lane] = make_float4(x.x * SCALE, x.y * SCALE, x.z * SCALE, x.w * SCALE);
      }
    }
    __syncthreads();
    for (int j = warp; j < G; j += NW) {
      const float4 v = reinterpret_cast<const float4*>(qv[j])[lane];
      const float mx = warp_max(fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
      // the largest |q'| 2^e in [2^9, 2^10): 2^4 more at the lowest field stays in fp16
      const int e = mx > 0.f && mx < INFINITY ? min(100, 9 - ds_exponent(mx)) : 0;  // -119 for the largest finite row
      const bool far = a.score.cap == 0.f && e < -50;
      const float unit = a.score.cap > 0.f ? a.score.inv_cap * ds_pow2(min(0, 60 - 16 + e - ds_exponent(a.score.inv_cap)))
                         : far             ? 1.f / DS_FAR
                                           : 1.f;
      const float tot = warp_sum((v.x * unit + v.y * unit) + (v.z * unit + v.w * unit));
      if (lane == 0) {
        s_exp[j] = e;
        const int half = (16 - e) / 2;  // 2^(16 - e) alone may pass fp32
        const float scale = unit * ds_pow2(half) * ds_pow2(16 - e - half);
        a.ws.qsum[(size_t)u * G + j] = make_float2(far ? -scale : scale, tot);
      }
    }
    __syncthreads();
    // Word (nt, s, r) of lane (g, t): column g is head j = 4 nt + g / 2, its first half (g even) or remainder times 2^11,
    // of q'_j 2^(e + 8 - bit(s)) at channels 32 t + 16 r + s and 8 on.
    uint32_t* fr = a.ws.qfrag + (size_t)u * NT * 16 * 32;
    for (int i = tid; i < NT * 16 * 32; i += DS_PREP_THREADS) {
      const int w = i >> 5, L = i & 31, nt = w >> 4, s = (w & 15) >> 1, rr = w & 1, g = L >> 2, t = L & 3;
      const int j = 4 * nt + (g >> 1);
      float v0 = 0.f, v1 = 0.f;
      if (j < G) {
        const float f = ds_pow2(s_exp[j] + 8 - ds_key_bit(s));
        const float x0 = qv[j][32 * t + 16 * rr + s] * f, x1 = qv[j][32 * t + 16 * rr + 8 + s] * f;
        const float2 hf = __half22float2(__floats2half2_rn(x0, x1));
        v0 = g & 1 ? (x0 - hf.x) * DS_LO : hf.x;
        v1 = g & 1 ? (x1 - hf.y) * DS_LO : hf.y;
      }
      fr[i] = ds_half2(v0, v1);
    }
    if (tid == 0) a.ws.span[u] = make_int2(1, 0);
    if (__ldg(a.lens + b) == 0)
      for (int i = tid; i < G * D; i += DS_PREP_THREADS) a.out[row0 + i] = 0.f;
  }
}

// ---------------------------------------------------------------------------
// The decode: blocks of `nw` warps, a slice of the batch's entries each.
// ---------------------------------------------------------------------------
template <int G, int P, bool FINE>
__global__ void __launch_bounds__(ds_max_warps(G) * 32, 1) ds_split_kernel(const __grid_constant__ DsArgs a) {
  constexpr int NT = ds_tiles(G), MAXW = ds_max_warps(G);
  constexpr int REC = 72 * P, PPE = 64 / P;  // bytes a page record, pages an entry
  constexpr int EPF = 32 / PPE;              // entries whose pages the warp's lanes hold
  constexpr int STAGE = 64 * 72, CHUNK = 32 * 72;
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t ds_smem[];
  __shared__ __align__(8) uint64_t bars[MAXW][DS_STAGES];
  __shared__ uint8_t s_pages[MAXW][DS_STAGES];  // which pages of the staged entry were copied
  __shared__ int s_before[MAXW * 32], s_warp[MAXW];
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gi = lane >> 2, ti = lane & 3;
  const int nw = blockDim.x >> 5, H = a.g.n_kv_heads;
  uint8_t* stages = ds_smem + warp * DS_STAGES * STAGE;

  // ---- the batch's list: sequence b holds H n_b entries, those of its KV heads one after another ----
  const int per = (a.n_seqs + (int)blockDim.x - 1) / (int)blockDim.x;
  const int b0 = min(a.n_seqs, tid * per), b1 = min(a.n_seqs, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += ds_view(a, b, blockIdx.x == 0 ? a.err : nullptr).n;
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_warp[warp] = inc;
  if (warp == 0) {
    tmem_alloc(&s_tmem, ds_columns(G, nw));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int total = 0;
  for (int w = 0; w < nw; ++w) {
    if (w == warp) s_before[tid] = total + inc - mine;
    total += s_warp[w];
  }
  __syncthreads();
  total *= H;
  const int n_warps = gridDim.x * nw, each = (total + n_warps - 1) / n_warps;
  const int gw = blockIdx.x * nw + warp;
  const long long start = (long long)gw * each;
  const int g0 = (int)min((long long)total, start);
  const int n = min(total, g0 + each) - g0;

  // a place in the list: sequence b, KV head h, whose entries are [first, end)
  struct Place {
    int b, h, first, end;
    DsView v;
  } at{};
  if (n > 0) {
    // the last thread whose run starts at or before g0, then the sequence in its run
    int lo = 0, cnt = blockDim.x;
    while (cnt > 1) {
      const int half = cnt >> 1;
      if ((long long)s_before[lo + half] * H <= g0) { lo += half; cnt -= half; } else cnt = half;
    }
    int base = s_before[lo];
    const int e1 = min(a.n_seqs, (lo + 1) * per);
    for (int b = lo * per; b < e1; b += 32) {
      const int x = b + lane < e1 ? ds_view(a, b + lane).n : 0;
      int s = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL, s, o);
        if (lane >= o) s += y;
      }
      const unsigned past = __ballot_sync(FULL, (long long)(base + s) * H > g0);
      if (past) {
        const int k = __ffs(past) - 1;
        at.b = b + k;
        base += __shfl_sync(FULL, s - x, k);
        break;
      }
      base += __shfl_sync(FULL, s, 31);
    }
    at.v = ds_view(a, at.b);
    at.h = (g0 - base * H) / at.v.n;
    at.first = base * H + at.h * at.v.n;
    at.end = at.first + at.v.n;
  }
  auto walk = [&](Place& p, int i) {  // on to list entry i
    while (i >= p.end) {
      if (++p.h == H) {
        p.h = 0;
        do p.v = ds_view(a, ++p.b);
        while (p.v.n == 0);
      }
      p.first = p.end;
      p.end += p.v.n;
    }
  };
  Place ahead = at;  // of the copies

  // Lane l holds the record of page l % PPE of entry i0 + l / PPE: -2 none that is seen, -1 a bad id.
  int rec = -2;
  auto pages = [&](int i0) {
    Place p = ahead;
    const int i = i0 + lane / PPE;
    rec = -2;
    if (i < n) {
      walk(p, g0 + i);
      const int t0 = p.v.first_token(g0 + i - p.first) + lane % PPE * P;
      if (t0 < p.v.len && (t0 < p.v.prefix || t0 + P > p.v.lo)) {
        const int id = __ldg(a.table + (size_t)p.b * a.g.max_blocks + t0 / P);
        rec = (unsigned)id < (unsigned)a.g.num_blocks ? id * H + p.h : -1;
      }
    }
  };
  int issued = 0;
  auto issue = [&](int i) {
    issued = i + 1;
    const int st = i % DS_STAGES;
    walk(ahead, g0 + i);
    if (i % EPF == 0) pages(i);
    const bool own = lane / PPE == i % EPF, ok = own && rec >= 0;
    const unsigned okm = __ballot_sync(FULL, ok), bad = __ballot_sync(FULL, own && rec == -1);
    const uint32_t bits = okm >> (i % EPF * PPE) & ((1u << PPE) - 1u);
    uint64_t* bar = &bars[warp][st];
    if (lane == 0) {
      if (bad) flag_error(a.err, ERR_BLOCK_RANGE);
      s_pages[warp][st] = (uint8_t)bits;
      mbar_arrive_expect_tx(bar, (uint32_t)__popc(bits) * REC);
    }
    __syncwarp();
    if (ok) {
      fence_proxy_async();
      bulk_g2s(stages + st * STAGE + lane % PPE * REC, a.pool + (size_t)rec * REC, REC, bar);
    }
  };
  if (n > 0) {
    if (lane == 0) {
      for (int s = 0; s < DS_STAGES; ++s) mbar_init(&bars[warp][s], 1);
      fence_mbar_init();
    }
    __syncwarp();
    for (int i = 0; i < DS_STAGES && i < n; ++i) issue(i);
  }
  pdl_wait();               // the queries
  pdl_launch_dependents();  // the combine may be scheduled as blocks retire
  const uint32_t tmem = s_tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 32 * NT * (warp >> 2);

  // ---- a segment: the warp's entries of one (sequence, KV head) ----
  uint32_t bq[NT][8][2];
  float qs[NT], qt[NT], slope[NT], m[NT], thr[NT], lp[NT], zp[NT], acc[NT][8][4];
  float behind[NT];      // what the sums in tensor memory are scaled by by now
  bool flushed = false;  // whether there are any
  int unit = -1, first = 0, end = 0;
  const float cap = a.score.cap;
  unsigned far = 0;  // bit nt: the units of the lane's row there are DS_FAR
  auto begin = [&](const Place& p) {
    unit = p.b * H + p.h;
    first = p.first;
    end = p.end;
    const uint32_t* fr = a.ws.qfrag + (size_t)unit * NT * 16 * 32 + lane;
    far = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        bq[nt][s][0] = __ldg(fr + (nt * 16 + 2 * s) * 32);
        bq[nt][s][1] = __ldg(fr + (nt * 16 + 2 * s + 1) * 32);
      }
      const int j = 4 * nt + ti;
      const float2 c = j < G ? __ldg(a.ws.qsum + (size_t)unit * G + j) : make_float2(0.f, 0.f);
      qs[nt] = fabsf(c.x);
      qt[nt] = c.y;
      far |= c.x < 0.f ? 1u << nt : 0u;
      slope[nt] = a.score.slopes && j < G ? score_slope(__ldg(a.score.slopes + p.h * G + j)) : 0.f;
      m[nt] = 0.f;
      thr[nt] = -INFINITY;
      lp[nt] = zp[nt] = 0.f;
      behind[nt] = 1.f;
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[nt][f][0] = acc[nt][f][1] = acc[nt][f][2] = acc[nt][f][3] = 0.f;
    }
  };
  // the sums to those in tensor memory (last: these back instead)
  auto flush = [&](bool last) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int f = 0; f < 8; f += 2) {
        const uint32_t at = tmem + 32 * nt + 4 * f;
        float v[8] = {};
        if (flushed) tmem_ld8(at, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[k] = fmaf(v[k], behind[nt], acc[nt][f + k / 4][k % 4]);
          acc[nt][f + k / 4][k % 4] = last ? v[k] : 0.f;
        }
        if (!last) ds_tmem_st8(at, v);
      }
      behind[nt] = 1.f;
    }
    if (!last) asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    flushed = true;
  };
  auto finish = [&]() {
    if (flushed) flush(true);
    flushed = false;
    float* out = a.ws.part + (size_t)(gw + unit) * G * DS_PART;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        lp[nt] += __shfl_xor_sync(FULL, lp[nt], o);
        zp[nt] += __shfl_xor_sync(FULL, zp[nt], o);
      }
      const int j = 4 * nt + ti;
      if (j < G) {
        float o[16];
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          const float up = (float)(1 << (24 - ds_value_bit(f, FINE)));
          o[f] = fmaf(fmaf(acc[nt][f][1], 1.f / DS_LO, acc[nt][f][0]), up, zp[nt]);      // channel 8 g + f
          o[8 + f] = fmaf(fmaf(acc[nt][f][3], 1.f / DS_LO, acc[nt][f][2]), up, zp[nt]);  // channel 64 + 8 g + f
        }
        float4* dst = reinterpret_cast<float4*>(out + j * DS_PART);
        dst[2 * gi] = make_float4(o[0], o[1], o[2], o[3]);
        dst[2 * gi + 1] = make_float4(o[4], o[5], o[6], o[7]);
        dst[16 + 2 * gi] = make_float4(o[8], o[9], o[10], o[11]);
        dst[16 + 2 * gi + 1] = make_float4(o[12], o[13], o[14], o[15]);
        if (gi == 0) *reinterpret_cast<float2*>(out + j * DS_PART + D) = make_float2(m[nt], lp[nt]);
      }
    }
    if (lane == 0 && gw == first / each) a.ws.span[unit] = make_int2(gw, (end - 1) / each);
  };

  // bytes inside a staged chunk of row r of 16-token tile u, P tokens a record (16 tokens are 1,152 bytes either way)
  auto row = [](int u, int r) { return u * 1152 + (P == 16 ? 0 : (r >> 3) * REC); };
  auto in_page = [](int r) { return P == 16 ? r : r & 7; };
  const int v_row = 8 * (lane >> 4) + (lane & 7);
  const uint32_t v_off = row(0, v_row) + 32 * P + 32 * in_page(v_row) + 16 * ((lane >> 3) & 1);

  // 32 tokens from tok0 on.  ALL: every one is seen and was copied.
  auto chunk = [&](auto all_tag, const uint8_t* st, int tok0, const DsView& v, int bits) {
    constexpr bool ALL = decltype(all_tag)::value;
    bool seen[4];
    float x[NT][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = k >> 1, r = gi + 8 * (k & 1), s = tok0 + 16 * u + r;
      seen[k] = ALL || (s < v.len && (s < v.prefix || s >= v.lo) && (bits >> (P == 16 ? u : 2 * u + (r >> 3)) & 1));
    }
    // ---- scores in base 2 ----
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint2 k0 = *reinterpret_cast<const uint2*>(st + row(u, gi) + 32 * in_page(gi) + 8 * ti);
      const uint2 k1 = *reinterpret_cast<const uint2*>(st + row(u, gi + 8) + 32 * in_page(gi + 8) + 8 * ti);
      // rows g, g + 8 of channels 32 t .. + 15, then of the next 16
      const uint32_t w[4] = {k0.x, k1.x, k0.y, k1.y};
      float d[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.f;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        uint32_t f[4];
        ds_field<false>(ds_key_shift(s), ds_key_bit(s), w, f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) ds_mma(d[nt], f, bq[nt][s][0], bq[nt][s][1]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = gi + 8 * e;
        const float2 km = __half22float2(*reinterpret_cast<const __half2*>(st + row(u, r) + 64 * P + 4 * in_page(r)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          x[nt][2 * u + e] = fmaf(km.x * qs[nt], fmaf(d[nt][2 * e + 1], 1.f / DS_LO, d[nt][2 * e]), km.y * qt[nt]);
      }
    }
    if (cap > 0.f) {
      float z = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) z = fmaxf(z, x[nt][k] * x[nt][k]);
      if (__any_sync(FULL, z > CAP_FIT)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[nt][k] = cap * tanh_any(x[nt][k]);
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const uint64_t y = f2pk(x[nt][k], x[nt][k + 1]), z2 = f2mul(y, y);
            const float2 t = f2up(f2fma(f2mul(y, z2), tanh_fit2(z2), y));
            x[nt][k] = cap * t.x;
            x[nt][k + 1] = cap * t.y;
          }
      }
    } else if (far) {  // scores beyond fp32's largest are equal
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float y = x[nt][k] * (far >> nt & 1 ? DS_FAR : 1.f);
          x[nt][k] = fabsf(y) > 0x1p126f ? copysignf(0x1p126f, y) : y;
        }
    }
    if (a.score.slopes) {
      const int far = v.len - 1 - tok0 - gi;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float dist = (float)(far - 8 * k);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[nt][k] = fmaf(-slope[nt], dist, x[nt][k]);
      }
    }
    if (!ALL) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[nt][k] = seen[k] ? x[nt][k] : -INFINITY;
    }
    // value scales, negated in tile 1, and what a weight adds to every channel: z, and 3 s in tile 1
    float vs[4], vz[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = gi + 8 * (k & 1);
      const float2 vm = __half22float2(*reinterpret_cast<const __half2*>(st + row(k >> 1, r) + 68 * P + 4 * in_page(r)));
      vs[k] = k >> 1 ? -vm.x : vm.x;
      vz[k] = k >> 1 ? fmaf(3.f, vm.x, vm.y) : vm.y;
    }
    // ---- weights ----
    uint32_t bp[NT][2][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float top = max3(x[nt][0], x[nt][1], fmaxf(x[nt][2], x[nt][3]));
      float p[4], w[4];  // 2^(x - ref), the same times the value scale; the largest of these
      auto weigh = [&](float ref) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          p[k] = ds_ex2(x[nt][k] - ref);
          w[k] = p[k] * vs[k];
          if (!ALL) {
            p[k] = seen[k] ? p[k] : 0.f;
            w[k] = seen[k] ? w[k] : 0.f;
          }
        }
        return max3(fabsf(w[0]), fabsf(w[1]), fmaxf(fabsf(w[2]), fabsf(w[3])));
      };
      const float high = weigh(m[nt]);
      const bool rises = top > thr[nt], over = high > WEIGHT_HIGH;
      if (__any_sync(FULL, rises || over)) {
        const unsigned column = 0x11111111u << ti;  // of heads: 32 tokens
        const unsigned up = __ballot_sync(FULL, rises) & column, far = __ballot_sync(FULL, over) & column;
        float mx = top, most = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) most = fmaxf(most, x[nt][k] + lg2_approx(fabsf(vs[k])));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
          most = fmaxf(most, __shfl_xor_sync(FULL, most, o));
        }
        if (up | far) {
          const float ref = up ? mx : thr[nt] - DS_TAU, now = ref - weight_lift(most - ref);
          const float scale = thr[nt] == -INFINITY ? 0.f : ds_ex2(m[nt] - now);
          m[nt] = now;
          thr[nt] = ref + DS_TAU;
          behind[nt] *= scale;
          lp[nt] *= scale;
          zp[nt] *= scale;
#pragma unroll
          for (int f = 0; f < 8; ++f) {
            acc[nt][f][0] *= scale; acc[nt][f][1] *= scale; acc[nt][f][2] *= scale; acc[nt][f][3] *= scale;
          }
        }
        weigh(m[nt]);
      }
      uint32_t pk[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float z = p[k] * vz[k];
        if (!ALL) z = seen[k] ? z : 0.f;
        lp[nt] += p[k];
        zp[nt] += z;
        const float hf = __half2float(__float2half_rn(w[k]));
        pk[k] = ds_half2(w[k], (w[k] - hf) * DS_LO);
      }
      // lane (g, t) has token g of head 4 nt + t, first half and remainder; the product wants columns g, tokens 2 t, 2 t + 1
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) bp[nt][u][e] = ds_transpose(pk[2 * u + e]);
    }
    // ---- readout ----
    const uint32_t va = smem_u32(st) + v_off;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t w[4];
      ldsm_x4_trans(va + u * 1152, w);
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        uint32_t c[4];
        if (u) ds_field<true>(ds_value_shift(f, FINE), ds_value_bit(f, FINE), w, c);
        else ds_field<false>(ds_value_shift(f, FINE), ds_value_bit(f, FINE), w, c);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) ds_mma(acc[nt][f], c, bp[nt][u][0], bp[nt][u][1]);
      }
    }
  };

  int i = 0, since = 0;
  for (; i < n; ++i) {
    const int st = i % DS_STAGES;
    if (!__all_sync(FULL, mbar_wait_bounded(&bars[warp][st], (i / DS_STAGES) & 1))) break;
    walk(at, g0 + i);
    if (at.b * H + at.h != unit) {
      if (unit >= 0) finish();
      begin(at);
      since = 0;
    }
    const int bits = s_pages[warp][st], tok = at.v.first_token(g0 + i - at.first);
#pragma unroll 1
    for (int sub = 0; sub < 2; ++sub) {
      const int t0 = tok + 32 * sub, have = bits >> (sub * (PPE / 2)) & ((1 << (PPE / 2)) - 1);
      if (have == 0) continue;
      const uint8_t* s = stages + st * STAGE + sub * CHUNK;
      const bool all = t0 + 32 <= at.v.len && (t0 + 32 <= at.v.prefix || t0 >= at.v.lo) && have == (1 << (PPE / 2)) - 1;
      if (all) chunk(std::true_type{}, s, t0, at.v, have);
      else chunk(std::false_type{}, s, t0, at.v, have);
    }
    __syncwarp();
    if (i + DS_STAGES < n) issue(i + DS_STAGES);
    if (++since == DS_FLUSH) {
      flush(false);
      since = 0;
    }
  }
  if (i < n) {
    if (lane == 0) flag_error(a.err, ERR_TIMEOUT);
    for (; i < issued; ++i) mbar_wait_bounded(&bars[warp][i % DS_STAGES], (i / DS_STAGES) & 1);  // no copy in flight at the end
  } else if (n > 0) {
    finish();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(s_tmem, ds_columns(G, nw));
  }
}

// The partials of a unit, joined in slice order: a block a (unit, query head), warp w the slots w, w + nw ..., the warps'
// states in warp order.
constexpr int DS_MAX_JOIN = 32;

template <int G>
__global__ void __launch_bounds__(DS_MAX_JOIN * 32) ds_combine_kernel(const __grid_constant__ DsArgs a) {
  __shared__ float s_m[DS_MAX_JOIN], s_l[DS_MAX_JOIN];
  __shared__ __align__(16) float s_o[DS_MAX_JOIN][D];
  pdl_launch_dependents();
  pdl_wait();
  const int u = blockIdx.x, j = blockIdx.y, nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int2 span = __ldcg(a.ws.span + u);
  const int slots = span.y - span.x + 1;
  if (slots <= 0) return;  // nothing cached (zeros are written) or a bad length
  const size_t step = (size_t)G * DS_PART;
  const float* base = a.ws.part + ((size_t)(span.x + u) * G + j) * DS_PART;
  float M = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t0 = warp; t0 < slots; t0 += 4 * nw) {
    float2 ml[4];
    float4 x[4];
    float top = M;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = t0 + k * nw;
      ml[k] = make_float2(0.f, 0.f);
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < slots) {
        ml[k] = __ldcg(reinterpret_cast<const float2*>(base + t * step + D));
        x[k] = __ldcg(reinterpret_cast<const float4*>(base + t * step) + lane);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[k].y != 0.f ? ml[k].x : -INFINITY);
    const float f0 = l != 0.f ? exp2f(M - top) : 0.f;
    M = top;
    l *= f0;
    o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (ml[k].y == 0.f) continue;  // a part that saw nothing
      const float f = exp2f(ml[k].x - M);
      l = fmaf(f, ml[k].y, l);
      o.x = fmaf(f, x[k].x, o.x); o.y = fmaf(f, x[k].y, o.y); o.z = fmaf(f, x[k].z, o.z); o.w = fmaf(f, x[k].w, o.w);
    }
  }
  const int b = u / a.g.n_kv_heads, h = u % a.g.n_kv_heads;
  float4* dst = reinterpret_cast<float4*>(a.out + ((size_t)b * a.n_q_heads + h * G + j) * D);
  if (nw > 1) {
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = l;
    }
    reinterpret_cast<float4*>(s_o[warp])[lane] = o;
    __syncthreads();
    if (warp > 0) return;
    float top = -INFINITY;
    for (int w = 0; w < nw; ++w) top = fmaxf(top, s_l[w] != 0.f ? s_m[w] : -INFINITY);
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < nw; ++w) {
      if (s_l[w] == 0.f) continue;
      const float f = exp2f(s_m[w] - top);
      const float4 x = reinterpret_cast<const float4*>(s_o[w])[lane];
      l = fmaf(f, s_l[w], l);
      o.x = fmaf(f, x.x, o.x); o.y = fmaf(f, x.y, o.y); o.z = fmaf(f, x.z, o.z); o.w = fmaf(f, x.w, o.w);
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  dst[lane] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

template <typename K>
static cudaError_t ds_launch_pdl(K kernel, dim3 grid, int block, int smem, cudaStream_t s, const DsArgs& a) {
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
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int G, int P, bool FINE>
static cudaError_t ds_launch_split(const DsArgs& a, int warps, int nw, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};  // per device
  cudaError_t e = smem_limit_once(done, ds_split_kernel<G, P, FINE>, ds_max_warps(G) * DS_WARP_SMEM);
  if (e != cudaSuccess) return e;
  return ds_launch_pdl(ds_split_kernel<G, P, FINE>, dim3(warps / nw), 32 * nw, nw * DS_WARP_SMEM, s, a);
}

template <int G>
static cudaError_t ds_launch(const DsArgs& a, const void* q, int dtype, RotDev rot, int warps, cudaStream_t s) {
  const int H = a.g.n_kv_heads, units = a.n_seqs * H, sms = device_sm_count();
  // dense: several sequences a CTA once there are more units than two CTAs an SM, as R is loaded once a CTA (earlier it costs
  // more: 128 units one, two, four a CTA 61.9, 63.5, 68 us); without R to load one a CTA (640 units: three 32.8, one 30.8 us)
  const int seqs = rot.kind == KVQ_ROT_DENSE ? max(1, min(8, (units + 2 * sms - 1) / (2 * sms))) : 1;
  const dim3 grid(H, (a.n_seqs + seqs - 1) / seqs);
  if (rot.kind == KVQ_ROT_DENSE) ds_prepare_kernel<G, true><<<grid, DS_PREP_THREADS, 0, s>>>(a, q, dtype, rot, seqs);
  else ds_prepare_kernel<G, false><<<grid, DS_PREP_THREADS, 0, s>>>(a, q, dtype, rot, seqs);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a full wave is one block an SM, whose warps progress together; fewer warps run as blocks of four
  const int nw = warps == sms * ds_max_warps(G) ? ds_max_warps(G) : 4;
  // Values all at bit 9: 1,000 tokens 9.0e-7 -> 6.2e-7 off fp64, 16 x 16,384 1.1e-6 -> 9.1e-7, for three more shifts a word: 63.65
  // -> 65.7 us there, 64 ragged sequences 31.2 -> 33.1, 4 x 4,096 (seven warps an SM) 16.65 -> 17.9; nothing where a scheduler
  // has one warp at most and waits anyway (1,000 tokens 14.5 us either way).
  const bool fine = warps <= 4 * sms;
  if (a.g.page_tokens == 16) e = fine ? ds_launch_split<G, 16, true>(a, warps, nw, s) : ds_launch_split<G, 16, false>(a, warps, nw, s);
  else e = fine ? ds_launch_split<G, 8, true>(a, warps, nw, s) : ds_launch_split<G, 8, false>(a, warps, nw, s);
  if (e != cudaSuccess) return e;
  const int per_unit = (warps + units - 1) / units + 1;
  int join = 1;
  while (join < DS_MAX_JOIN && join * 8 < per_unit) join *= 2;  // about eight slots a warp
  return ds_launch_pdl(ds_combine_kernel<G>, dim3(units, G), 32 * join, 0, s, a);
}

cudaError_t launch_decode_score(const PageGeom& g, int n_q_heads, int n_seqs, const void* q, int q_dtype,
                                const int32_t* seq_lens, int max_seq_len, const int32_t* table, RotDev rot_k,
                                const uint8_t* pool, const ScoreDev& score, void* ws_base, size_t ws_bytes, float* o_rot,
                                unsigned* err, cudaStream_t s) {
  const int gqa = n_q_heads / g.n_kv_heads;
  const int warps = 4 * decode_auto_ctas(n_seqs, g.n_kv_heads, gqa, max_seq_len);
  DsArgs a{g, n_seqs, n_q_heads, max_seq_len, seq_lens, table, pool, score, {}, o_rot, err};
  if (ds_layout(ws_base, n_seqs * g.n_kv_heads, gqa, warps, &a.ws) > ws_bytes) return cudaErrorInvalidValue;
  switch (gqa) {
    case 1: return ds_launch<1>(a, q, q_dtype, rot_k, warps, s);
    case 2: return ds_launch<2>(a, q, q_dtype, rot_k, warps, s);
    case 4: return ds_launch<4>(a, q, q_dtype, rot_k, warps, s);
    case 8: return ds_launch<8>(a, q, q_dtype, rot_k, warps, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
