// From a layer's projections to what the cache write and the attention take: the
// heads of qkv normed one by one, turned by their position and split into q, k, v.
//
//   y = x w / sqrt(mean(x^2) + eps)                      (w NULL: y = x)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_a sin + y_b cos) for the pairs of the first
//   r channels; v is copied.  All in fp32, one rounding to the output's type.
//
// Angles.  A position times a frequency in fp32 is off by up to 2^-24 of itself: 0.06
// at position 10^6.  A frequency is therefore held as the fraction of a turn that one
// position adds, in 64-bit fixed point: an integer product modulo 2^64 drops whole
// turns without rounding, and what is left is off by 2^-64 turns a position at most.
//
// A half-warp owns a token's heads of a group, 8 channels a lane: one 16- or 32-byte
// load and store a head, the sum of squares over 16 lanes, and a pair's other channel
// from the lane that holds it (as it came, before the norm) or, side by side, from the
// same lane.  cos and sin are taken once a token (64 of each, shared by its heads),
// multiplied by the weights once a token and group.
// Bound: HBM, each element read and written once: 16,384 tokens of 32 / 8 heads in bf16 take
// 72.7 us, 5.5 TB/s (a plain copy of as many bytes 6.2), 7,777 of 16 / 4 in fp32 36.9, 5.2.
// Five blocks an SM of 256 threads with four heads' loads in flight: four 2 us more, six 12; two
// or eight heads in flight 22 and 20.
#include "async_copy.cuh"
#include "kvq_internal.cuh"

namespace kvq {

constexpr int NR_THREADS = 256;
constexpr int NR_TOKENS = NR_THREADS / 16;  // tokens a block, one a half-warp
constexpr float NR_LEAST = 0x1p-110f, NR_MOST = 0x1p126f;  // sums of squares that are as exact as their squares; below, an eps
                                                          // of as much hides what they lost

struct NrArgs {
  int n_tok, n_q, n_kv, heads_per_group;
  const void* qkv;
  long long stride;  // elements a row of qkv
  const int32_t* pos;
  const float* w_q;
  const float* w_k;
  float eps;
  bool wide;
  void* out[3];
  RopeDev rope;
};

template <bool F32>
struct NrRaw {
  uint32_t w[F32 ? 8 : 4];
};

// fp32: 32 bytes at once where everything lies on 32-byte boundaries (wide).  Two 16-byte accesses side by side take half of
// every 32-byte sector each.
template <bool F32>
__device__ __forceinline__ NrRaw<F32> nr_load(const void* base, size_t elem, bool wide) {
  NrRaw<F32> r;
  if constexpr (F32) {
    const float* p = static_cast<const float*>(base) + elem;
    if (wide) {
      asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                     "=r"(r.w[7])
                   : "l"(p));
      return r;
    }
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + elem));
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
  }
  return r;
}

template <bool F32>
__device__ __forceinline__ void nr_store(void* base, size_t elem, const NrRaw<F32>& r, bool wide) {
  if constexpr (F32) {
    float* p = static_cast<float*>(base) + elem;
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
                   "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
                   : "memory");
      return;
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + elem) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  }
}

template <bool F32>
__device__ __forceinline__ void nr_unpack(const NrRaw<F32>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = __uint_as_float(F32 ? r.w[i % (F32 ? 8 : 4)] : (i & 1) ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
}

template <bool F32>
__device__ __forceinline__ NrRaw<F32> nr_pack(const float (&x)[8]) {
  NrRaw<F32> r;
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return r;
}

// The heads of this thread's token whose squares leave fp32's range, once more, a power of two smaller or larger.  Out of line,
// out of the loops' registers (in them: 16,384 tokens 72 -> 80 us; looking for such heads is 0.9 of 73).
template <bool F32, bool SIDE>
__device__ __noinline__ void nr_again(const NrArgs& a, const float2 (*turn)[D / 2]) {
  const int tid = threadIdx.x, l = tid & 15, tok0 = blockIdx.x * NR_TOKENS, slot = tid >> 4, half = a.rope.dim / 2;
  const unsigned lanes16 = 0xffffu << (tid & 16);
  const int t = min(tok0 + slot, a.n_tok - 1), heads = a.n_q + a.n_kv, h0 = blockIdx.y * a.heads_per_group;
  const int lanes = half / 8, other = SIDE || l >= 2 * lanes ? 0 : l < lanes ? lanes : -lanes;
#pragma unroll 1
  for (int h = h0; h < min(heads, h0 + a.heads_per_group); ++h) {
    const int part = h >= a.n_q, n = part ? a.n_kv : a.n_q;
    const float* w = part ? a.w_k : a.w_q;
    if (!w) continue;
    float x[8], s = 0.f;
    nr_unpack<F32>(nr_load<F32>(a.qkv, (size_t)t * a.stride + 8 * l + (size_t)h * D, a.wide), x);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
    for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(lanes16, s, d);
    const bool small = s < NR_LEAST && a.eps < NR_LEAST;
    if (!small && s <= NR_MOST) continue;
    const float c = small ? 0x1p90f : 0x1p-70f;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] *= c;
      s = fmaf(x[i], x[i], s);
    }
    for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(lanes16, s, d);
    const float r = rsqrtf(fmaf(s, 1.f / D, a.eps * c * c));
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ch = 8 * l + i, o = SIDE ? ch ^ 1 : ch + 8 * other;
      const float p = SIDE ? x[i ^ 1] : __shfl_sync(lanes16, x[i], l + other, 16);
      y[i] = x[i] * __ldg(w + ch);
      if (l < 2 * lanes) {
        float2 cs = turn[t - tok0][SIDE ? ch / 2 : ch - (l < lanes ? 0 : half)];
        if (SIDE ? (i & 1) == 0 : l < lanes) cs.y = -cs.y;
        y[i] = fmaf(p, cs.y * __ldg(w + o), x[i] * (cs.x * __ldg(w + ch)));
      }
      y[i] *= r;
    }
    if (tok0 + slot < a.n_tok)
      nr_store<F32>(a.out[part], ((size_t)t * n + (h - (part ? a.n_q : 0))) * D + 8 * l, nr_pack<F32>(y), a.wide);
  }
}

// Grid (token blocks, head groups).  SIDE: pairs (2i, 2i + 1), else (i, i + r / 2).
template <bool F32, bool SIDE>
__global__ void __launch_bounds__(NR_THREADS, 5) norm_rope_kernel(const __grid_constant__ NrArgs a) {
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int AHEAD = F32 ? 2 : 4;  // heads whose loads are in flight
  __shared__ float2 turn[NR_TOKENS][D / 2];  // (cos, sin)
  const int tid = threadIdx.x, l = tid & 15;
  const int tok0 = blockIdx.x * NR_TOKENS, slot = tid >> 4;
  const int half = a.rope.dim / 2;

  {
    const int pair = tid & 63;
    if (pair < half) {
      const unsigned long long f = a.rope.turn[pair];
      const int32_t* pos = a.pos + (size_t)a.rope.axis[pair] * a.n_tok;
      for (int s = tid >> 6; s < NR_TOKENS && tok0 + s < a.n_tok; s += NR_THREADS / 64) {
        const unsigned long long t = (unsigned long long)(long long)__ldg(pos + tok0 + s) * f;
        float sn, cs;
        sincospif((float)(int)(t >> 32) * 0x1p-31f, &sn, &cs);
        turn[s][pair] = make_float2(cs, sn);
      }
    }
  }
  __syncthreads();
  // rows past the end follow the last token and store nothing: the shuffles keep all lanes
  const bool live = tok0 + slot < a.n_tok;
  const int t = min(tok0 + slot, a.n_tok - 1), ts = t - tok0;

  const int heads = a.n_q + 2 * a.n_kv;
  const int h0 = blockIdx.y * a.heads_per_group, h1 = min(heads, h0 + a.heads_per_group);
  const size_t row = (size_t)t * a.stride + 8 * l;
  // the lane's channels turn with those `other` lanes on, rest below r
  const int lanes = half / 8;
  const int other = SIDE || l >= 2 * lanes ? 0 : l < lanes ? lanes : -lanes;
  const bool turned = l < 2 * lanes;

  float odd = 0.f;  // not finite where some head's squares may have left fp32's range (the token's 16 lanes agree)
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int first = part ? a.n_q : 0, n = part ? a.n_kv : a.n_q;
    const int b0 = max(h0, first), b1 = min(h1, first + n);
    if (b0 >= b1) continue;
    const float* w = part ? a.w_k : a.w_q;
    // y'_i = r (x_i A_i + x_other(i) B_i)
    float A[8], B[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = 8 * l + i, o = SIDE ? c ^ 1 : c + 8 * other;
      float2 cs = make_float2(1.f, 0.f);
      if (turned) {
        cs = turn[ts][SIDE ? c / 2 : c - (l < lanes ? 0 : half)];
        if (SIDE ? (i & 1) == 0 : l < lanes) cs.y = -cs.y;
      }
      A[i] = cs.x * (w ? __ldg(w + c) : 1.f);
      B[i] = cs.y * (w ? __ldg(w + (turned ? o : c)) : 1.f);
    }
    void* out = a.out[part];
#pragma unroll 1
    for (int h = b0; h < b1; h += AHEAD) {
      NrRaw<F32> raw[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) raw[k] = nr_load<F32>(a.qkv, row + (size_t)min(h + k, b1 - 1) * D, a.wide);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (h + k >= b1) break;
        float x[8], y[8], p[8];
        nr_unpack<F32>(raw[k], x);
        float r = 1.f;
        if (w) {
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
          for (int d = 8; d > 0; d >>= 1) s += __shfl_xor_sync(FULL, s, d);
          r = rsqrtf(fmaf(s, 1.f / D, a.eps));
          odd = fmaf(r, 0x1p75f, odd + s);
        }
        if constexpr (SIDE) {
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = x[i ^ 1];
        } else {
          NrRaw<F32> q;
#pragma unroll
          for (int i = 0; i < (F32 ? 8 : 4); ++i) q.w[i] = __shfl_sync(FULL, raw[k].w[i], l + other, 16);
          nr_unpack<F32>(q, p);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (turned ? fmaf(p[i], B[i], x[i] * A[i]) : x[i] * A[i]) * r;
        if (live) nr_store<F32>(out, ((size_t)t * n + (h + k - first)) * D + 8 * l, nr_pack<F32>(y), a.wide);
      }
    }
  }
  if (__builtin_expect(!(odd < INFINITY), 0)) nr_again<F32, SIDE>(a, turn);
  const int first = a.n_q + a.n_kv;
  if (!live || !a.out[2]) return;
#pragma unroll 4
  for (int h = max(h0, first); h < h1; ++h)
    nr_store<F32>(a.out[2], ((size_t)t * a.n_kv + (h - first)) * D + 8 * l, nr_load<F32>(a.qkv, row + (size_t)h * D, a.wide),
                  a.wide);
}

cudaError_t launch_norm_rope(int n_tok, int n_q_heads, int n_kv_heads, const void* qkv, int dtype, long long stride,
                             const int32_t* pos, const RopeDev& rope, const float* w_q, const float* w_k, float eps,
                             void* q, void* k, void* v, cudaStream_t s) {
  const int heads = n_q_heads + 2 * n_kv_heads;
  const long long blocks = ((long long)n_tok + NR_TOKENS - 1) / NR_TOKENS;
  // 24 heads a group amortise a token's cos and sin; where that leaves SMs idle, four (one batch of loads).  16,384 tokens of 48
  // heads: 8, 16, 24, 48 heads a group 94, 73.5, 71.6, 77 us (other head counts not measured: a last group may be short)
  const int per = blocks * ((heads + 23) / 24) >= 4ll * device_sm_count() ? 24 : 4;
  const uintptr_t low = reinterpret_cast<uintptr_t>(qkv) | reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                        reinterpret_cast<uintptr_t>(v) | (uintptr_t)(stride * 4);
  NrArgs a{n_tok, n_q_heads, n_kv_heads, per, qkv, stride, pos, w_q, w_k, eps, (low & 31) == 0, {q, k, v}, rope};
  const dim3 grid((unsigned)blocks, (unsigned)((heads + per - 1) / per));
  if (dtype == KVQ_F32) {
    if (rope.side) norm_rope_kernel<true, true><<<grid, NR_THREADS, 0, s>>>(a);
    else norm_rope_kernel<true, false><<<grid, NR_THREADS, 0, s>>>(a);
  } else {
    if (rope.side) norm_rope_kernel<false, true><<<grid, NR_THREADS, 0, s>>>(a);
    else norm_rope_kernel<false, false><<<grid, NR_THREADS, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace kvq
