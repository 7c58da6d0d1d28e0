// ep_route_kernels.cu — the router: logits [T,E] to the top-k experts of each
// token and their weights, and the gradient of the weights back to the logits.
//
// Eight lanes share a token (16 beyond 256 experts; a whole warp, for few tokens
// or beyond 512 experts): its experts come in pieces of four, lane q of the token taking
// pieces q, q + L, ..., so that rows are read in whole sectors and a lane's own
// experts ascend.  Each lane keeps its keys in shared memory, a piece after
// another, and each piece's best in registers: taking the best expert costs
// those maxima, three exchanges between the lanes and one piece, for four
// tokens at once.  (One warp per token with its keys in registers, every one
// compared at each step: 16384 x 256 grouped 27.3 us, 65536 x 128 35.0 us.)
//
// Selection goes by fp32 keys: the scores with their bias, or, for a softmax or
// a sigmoid without bias, the logits themselves: both rise strictly with the
// logit, which keeps apart what the 32-bit scores would round together.  Groups
// are chosen by sums of scores, with or without a bias.
// -inf marks what cannot be taken: a masked expert (logit -inf or NaN), an
// expert of a group left out, one already taken.
//
// Bound by instructions, not by memory: scores that only decide the order, and
// the softmax's sum, take the hardware's exp2 and reciprocal (together within
// 2^-22 of the score's range).  The weights are expf or the sigmoid by IEEE
// division, times the IEEE reciprocal of the sum, times the scale; where a softmax
// is not renormalised that sum is the hardware's exp2 too (its terms' errors, 2^-22
// each, average out over a row).
#include <cuda_bf16.h>

#include "ep_internal.cuh"

namespace ep {
namespace {

constexpr int kRouteWarps = 4;

__device__ __forceinline__ float bf16_lo(unsigned v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(unsigned v) { return __uint_as_float(v & 0xffff0000u); }

// Experts e0 .. e0+3 of one row (fill beyond E); vec: the row's pieces are aligned.
template <typename In>
__device__ __forceinline__ void load4(const In* row, int e0, int E, bool vec, float fill, float v[4]);

template <>
__device__ __forceinline__ void load4<float>(const float* row, int e0, int E, bool vec, float fill, float v[4]) {
  if (vec && e0 + 4 <= E) {
    const float4 f = *reinterpret_cast<const float4*>(row + e0);
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = e0 + i < E ? row[e0 + i] : fill;
  }
}

template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* row, int e0, int E, bool vec, float fill,
                                                     float v[4]) {
  if (vec && e0 + 4 <= E) {
    const uint2 f = *reinterpret_cast<const uint2*>(row + e0);
    v[0] = bf16_lo(f.x);
    v[1] = bf16_hi(f.x);
    v[2] = bf16_lo(f.y);
    v[3] = bf16_hi(f.y);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = e0 + i < E ? __bfloat162float(row[e0 + i]) : fill;
  }
}

__device__ __forceinline__ void store4(float* row, int e0, int E, bool vec, const float v[4]) {
  if (vec && e0 + 4 <= E) {
    *reinterpret_cast<float4*>(row + e0) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e0 + i < E) row[e0 + i] = v[i];
  }
}

__device__ __forceinline__ void store4(__nv_bfloat16* row, int e0, int E, bool vec, const float v[4]) {
  if (vec && e0 + 4 <= E) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 f;
    f.x = *reinterpret_cast<const unsigned*>(&a);
    f.y = *reinterpret_cast<const unsigned*>(&b);
    *reinterpret_cast<uint2*>(row + e0) = f;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e0 + i < E) row[e0 + i] = __float2bfloat16_rn(v[i]);
  }
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Offset binary of a float, whose unsigned order is the floats' order, and back (-0 as +0).
__device__ __forceinline__ unsigned order_key(float f) {
  const unsigned u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_value(unsigned k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// Over the L lanes of a token.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  if (L == 32) return key_value(__reduce_max_sync(~0u, order_key(v)));
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ unsigned lanes_min(unsigned v) {
  if (L == 32) return __reduce_min_sync(~0u, v);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ unsigned lanes_or(unsigned v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v |= __shfl_xor_sync(~0u, v, o);
  return v;
}

__device__ __forceinline__ bool available(float z) { return z == z && z != -INFINITY; }
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// exp and sigmoid by the hardware's exp2 and reciprocal.
__device__ __forceinline__ float quick_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.442695041f));
  return y;
}
__device__ __forceinline__ float quick_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The lanes of one token, and where an expert's key lies.
template <int L, int NP>
struct Lanes {
  int lane, tok, q;  // lane of the warp, token of the warp, lane of the token
  __device__ Lanes() : lane(threadIdx.x & 31), tok(lane / L), q(lane % L) {}
  // expert j of this lane
  __device__ __forceinline__ int expert(int j) const { return 4 * (q + L * (j >> 2)) + (j & 3); }
  // word of expert e of this token in the warp's keys [NP][32][4]
  __device__ __forceinline__ int word(int e) const {
    const int p = e >> 2;
    return ((p / L) * 32 + tok * L + p % L) * 4 + (e & 3);
  }
};

// A token's experts that its lane holds; what is not available becomes -inf.
template <int L, int NP, typename In>
__device__ __forceinline__ void load_row(const In* row, const Lanes<L, NP>& at, int E, bool vec, float (&z)[4 * NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    float x[4];
    load4<In>(row, at.expert(4 * i), E, vec, -INFINITY, x);
#pragma unroll
    for (int c = 0; c < 4; ++c) z[4 * i + c] = fmaxf(x[c], -INFINITY);  // NaN too
  }
}

// The softmax's maximum over a token (0 if it has no expert).
template <int L, int NP>
__device__ __forceinline__ float row_max(const float (&z)[4 * NP]) {
  float m = z[0];
#pragma unroll
  for (int j = 1; j < 4 * NP; ++j) m = fmaxf(m, z[j]);
  m = lanes_max<L>(m);
  return m == -INFINITY ? 0.0f : m;
}

// What the selection goes by.
enum By {
  kLogits,       // no bias, no groups
  kScores,       // scores and a bias, with or without groups
  kGroupLogits,  // groups by scores, their experts by the logits (no bias).  A kernel of its own: as a
                 // branch it cost the biased one registers, 16384 x 256 grouped 14.4 -> 18.5 us
};

template <int L, int NP, By BY, typename In>
__global__ void __launch_bounds__(32 * kRouteWarps) ep_route_kernel(RouteDev d) {
  constexpr bool SCORED = BY != kLogits;  // every expert's score is needed
  constexpr int V = 4 * NP;               // keys of a lane
  constexpr int kTokens = 32 / L;         // of a warp
  __shared__ float4 s_key[kRouteWarps][NP * 32];
  __shared__ int s_expert[kRouteWarps][kTokens * 16];
  __shared__ float s_group[SCORED ? kRouteWarps : 1][SCORED ? kTokens * 32 : 1];
  pdl_wait();
  const Lanes<L, NP> at;
  const int warp = threadIdx.x >> 5, lane = at.lane, q = at.q;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp) * kTokens;
  if (t0 >= d.T) return;  // whole warps; only warp-wide synchronisation below
  const bool spare = t0 + at.tok >= d.T;  // repeats the last token and stores nothing
  const int64_t t = spare ? d.T - 1 : t0 + at.tok;
  const In* row = static_cast<const In*>(d.logits) + t * d.ld;
  float4* pieces = s_key[warp] + lane;

  float z[V];
  load_row<L, NP, In>(row, at, d.E, d.vec, z);
  float top = 0.0f, total = 0.0f;
  if (!d.sigmoid && (SCORED || !d.renorm)) {
    top = row_max<L, NP>(z);
#pragma unroll
    for (int j = 0; j < V; ++j) total += quick_exp(z[j] - top);
    total = lanes_sum<L>(total);
  }

  float key[V];
  const float per_total = SCORED && !d.sigmoid ? quick_rcp(total) : 0.0f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (BY == kScores) load4<float>(d.bias, at.expert(4 * i), d.E, d.vec_bias, 0.0f, b);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float x = z[4 * i + c];
      key[4 * i + c] = x;
      if (SCORED) {
        const float s = (d.sigmoid ? quick_rcp(1.0f + quick_exp(-x)) : quick_exp(x - top) * per_total) + b[c];
        key[4 * i + c] = x == -INFINITY ? x : fmaxf(s, -INFINITY);
      }
    }
  }

  if (SCORED && d.G > 1) {
    // A group's score is the sum of its two best experts' (of what it has).
#pragma unroll
    for (int i = 0; i < NP; ++i) pieces[i * 32] = make_float4(key[4 * i], key[4 * i + 1], key[4 * i + 2], key[4 * i + 3]);
    __syncwarp();
    const float* keys = reinterpret_cast<const float*>(s_key[warp]);
    const int per = d.E / d.G;
    float* group = &s_group[warp][at.tok * 32];
    for (int g = q; g < d.G; g += L) {
      float a = -INFINITY, b = -INFINITY;  // the two largest keys
      auto take = [&](float k) {
        b = fmaxf(b, fminf(a, k));
        a = fmaxf(a, k);
      };
      if (per % 4 == 0) {
        // by pieces, each lane from another one on: no two in the same banks
        const int n = per / 4;
        int i = q % n;
        for (int left = n; left > 0; --left) {
          const int p = g * n + i;
          const float4 k = s_key[warp][p / L * 32 + at.tok * L + p % L];
          take(k.x);
          take(k.y);
          take(k.z);
          take(k.w);
          if (++i == n) i = 0;
        }
      } else {
        for (int i = 0; i < per; ++i) take(keys[at.word(g * per + i)]);
      }
      group[g] = b > -INFINITY ? a + b : a;
    }
    __syncwarp();
    unsigned in = 0;  // the groups that come before all but TG - 1 others
    for (int g = q; g < d.G; g += L) {
      const float mine = group[g];
      int before = 0;
      for (int h = 0; h < d.G; ++h) {
        const float other = group[h];
        before += other > mine || (other == mine && h < g) ? 1 : 0;
      }
      if (before < d.TG) in |= 1u << g;
    }
    in = lanes_or<L>(in);
    __syncwarp();
    if (per % 4 == 0) {  // a piece lies in one group
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const unsigned g = __umulhi(static_cast<unsigned>(at.expert(4 * i)), d.per_magic);
        if (!(in >> (g & 31) & 1)) key[4 * i] = key[4 * i + 1] = key[4 * i + 2] = key[4 * i + 3] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const unsigned e = at.expert(j);
        const unsigned g = per == 1 ? e : __umulhi(e, d.per_magic);
        if (!(in >> (g & 31) & 1)) key[j] = -INFINITY;
      }
    }
    if (BY == kGroupLogits) {  // the groups stand: the logits are read again
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float x[4];
        load4<In>(row, at.expert(4 * i), d.E, d.vec, -INFINITY, x);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (key[4 * i + c] > -INFINITY) key[4 * i + c] = x[c];
      }
    }
  }

  float best_of[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    pieces[i * 32] = make_float4(key[4 * i], key[4 * i + 1], key[4 * i + 2], key[4 * i + 3]);
    best_of[i] = fmaxf(fmaxf(key[4 * i], key[4 * i + 1]), fmaxf(key[4 * i + 2], key[4 * i + 3]));
  }

  // the K best, one by one
  if (q < 16)
    for (int k = q; k < d.K; k += L) s_expert[warp][at.tok * 16 + k] = -1;
  __syncwarp();
  const unsigned others = (L == 32 ? ~0u : ((1u << (L & 31)) - 1) << (at.tok * L)) & ~(1u << lane);
  for (int k = 0; k < d.K; ++k) {
    float best = best_of[0];
#pragma unroll
    for (int i = 1; i < NP; ++i) best = fmaxf(best, best_of[i]);
    const float most = lanes_max<L>(best);
    bool mine = best == most && most > -INFINITY;
    const unsigned holders = __ballot_sync(~0u, mine);
    if (holders == 0) break;  // no token has any left
    // the piece, and in it the first key that is the best
    int g = 0;
#pragma unroll
    for (int i = NP - 1; i >= 0; --i)
      if (best_of[i] == best) g = i;
    float4 p = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (mine) p = pieces[g * 32];
    const int o = p.x == best ? 0 : p.y == best ? 1 : p.z == best ? 2 : 3;
    const int e = at.expert(4 * g) + o;
    if (__any_sync(~0u, mine && (holders & others))) {  // equal keys in two lanes: the lower expert
      const unsigned low = lanes_min<L>(mine ? static_cast<unsigned>(e) : ~0u);
      mine = mine && static_cast<unsigned>(e) == low;
    }
    if (mine) {
      s_expert[warp][at.tok * 16 + k] = e;
      if (o == 0) p.x = -INFINITY;
      if (o == 1) p.y = -INFINITY;
      if (o == 2) p.z = -INFINITY;
      if (o == 3) p.w = -INFINITY;
      pieces[g * 32] = p;
      const float next = fmaxf(fmaxf(p.x, p.y), fmaxf(p.z, p.w));
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (i == g) best_of[i] = next;
    }
  }
  __syncwarp();

  // weights: lane q has the slots q, q + L, ...
  constexpr int kSlots = L < 16 ? 16 / L : 1;
  int chosen[kSlots];
  float w[kSlots], zk[kSlots];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int k = q + i * L;
    chosen[i] = k < d.K ? s_expert[warp][at.tok * 16 + k] : -1;
    zk[i] = chosen[i] >= 0 ? to_f32(row[chosen[i]]) : -INFINITY;
    m = fmaxf(m, zk[i]);
  }
  // the softmax over the chosen ones is the softmax over all, renormalised
  if (!d.sigmoid && d.renorm) top = lanes_max<L>(m);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    w[i] = 0.0f;
    if (chosen[i] >= 0) w[i] = d.sigmoid ? sigmoid(zk[i]) : expf(zk[i] - top);
    sum += w[i];
  }
  float per_sum = 1.0f;
  if (d.renorm) {
    sum = lanes_sum<L>(sum);
    per_sum = sum == 0.0f ? 0.0f : 1.0f / sum;
  } else if (!d.sigmoid) {
    per_sum = 1.0f / total;
  }
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int k = q + i * L;
    if (k < d.K && !spare) {
      d.topk_idx[t * d.K + k] = chosen[i];
      d.topk_weights[t * d.K + k] = chosen[i] >= 0 ? w[i] * per_sum * d.scale : 0.0f;
    }
  }
}

// ---- bf16 logits that compete by themselves, up to eight experts a token ----
//
// A bf16 logit leaves room for its expert's number in one 32-bit key: the order
// of the logit above, 0xffff - e below.  Keys differ, so that ties need no care,
// and a key is all that moves.  A lane keeps its eight best in registers in
// descending order, takes eight experts at a time through a sorting network and
// joins lists as bitonic sequences; then lists are joined between the lanes.  No
// selection waits for another: 65536 x 128 top-8 16.8 -> 12.0 us, 2048 x 64 top-6
// 2.8 -> 1.6, bound by the minima and maxima (14 an expert at 128 of them).

constexpr int kListed = 8;

__device__ __forceinline__ void order2(unsigned& a, unsigned& b) {
  const unsigned lo = min(a, b);
  a = max(a, b);
  b = lo;
}

// Batcher's odd-even merge sort of eight, descending.
__device__ __forceinline__ void sort8(unsigned (&k)[8]) {
  order2(k[0], k[1]), order2(k[2], k[3]), order2(k[4], k[5]), order2(k[6], k[7]);
  order2(k[0], k[2]), order2(k[1], k[3]), order2(k[4], k[6]), order2(k[5], k[7]);
  order2(k[1], k[2]), order2(k[5], k[6]);
  order2(k[0], k[4]), order2(k[1], k[5]), order2(k[2], k[6]), order2(k[3], k[7]);
  order2(k[2], k[4]), order2(k[3], k[5]);
  order2(k[1], k[2]), order2(k[3], k[4]), order2(k[5], k[6]);
}

// The eight best of two descending lists: the larger of opposite elements, a
// bitonic sequence, put in order.
__device__ __forceinline__ void join8(unsigned (&k)[8], const unsigned (&other)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) k[i] = max(k[i], other[7 - i]);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) order2(k[i], k[i + d]);
}

// Keys of logits that are not available end up at or below this.
constexpr unsigned kNoKey = 0x007fffffu;

__device__ __forceinline__ unsigned packed_key(float z, int e) {
  // NaN as -inf, -0 as +0; the low half of a bf16's word is zero
  const unsigned u = __float_as_uint(fmaxf(z + 0.0f, -INFINITY));
  const unsigned up = u ^ (static_cast<unsigned>(static_cast<int>(u) >> 31) | 0x80000000u);
  return __byte_perm(up, 0xffffu - e, 0x3254);
}

__device__ __forceinline__ float packed_logit(unsigned key) {
  return key_value((key & 0x80000000u) ? key & 0xffff0000u : key | 0xffffu);
}

template <int L>
__global__ void __launch_bounds__(32 * kRouteWarps) ep_route_packed_kernel(RouteDev d) {
  constexpr int kTokens = 32 / L, kSlots = L < kListed ? kListed / L : 1;
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tok = lane / L, q = lane % L;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp) * kTokens;
  if (t0 >= d.T) return;
  const bool spare = t0 + tok >= d.T;  // repeats the last token and stores nothing
  const int64_t t = spare ? d.T - 1 : t0 + tok;
  const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(d.logits) + t * d.ld;

  unsigned best[8];
  auto keys = [&](int base, unsigned (&k)[8]) {
    const int e = base + 8 * q;
    float z[8];
    load4(row, e, d.E, d.vec, -INFINITY, *reinterpret_cast<float(*)[4]>(z));
    load4(row, e + 4, d.E, d.vec, -INFINITY, *reinterpret_cast<float(*)[4]>(z + 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = packed_key(z[i], e + i);
    sort8(k);
  };
  keys(0, best);
  for (int base = 8 * L; base < d.E; base += 8 * L) {
    unsigned more[8];
    keys(base, more);
    join8(best, more);
  }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) {
    unsigned other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(~0u, best[i], o);
    join8(best, other);
  }

  const float first = packed_logit(best[0]), top = first == -INFINITY ? 0.0f : first;
  float total = 0.0f;
  if (!d.sigmoid && !d.renorm) {
    for (int e = 4 * q; e < d.E; e += 4 * L) {
      float z[4];
      load4(row, e, d.E, d.vec, -INFINITY, z);
#pragma unroll
      for (int i = 0; i < 4; ++i) total += quick_exp(fmaxf(z[i], -INFINITY) - top);
    }
    total = lanes_sum<L>(total);
  }

  // lane q has the slots q, q + L, ...
  int chosen[kSlots];
  float w[kSlots], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int k = q + i * L;
    unsigned key = 0;
#pragma unroll
    for (int j = 0; j < kListed; ++j)
      if (j == k && j < d.K) key = best[j];
    chosen[i] = key > kNoKey ? static_cast<int>(0xffffu - (key & 0xffffu)) : -1;
    const float z = packed_logit(key);
    w[i] = 0.0f;
    if (chosen[i] >= 0) w[i] = d.sigmoid ? sigmoid(z) : expf(z - top);
    sum += w[i];
  }
  float per_sum = 1.0f;
  if (d.renorm) {
    sum = lanes_sum<L>(sum);
    per_sum = sum == 0.0f ? 0.0f : 1.0f / sum;
  } else if (!d.sigmoid) {
    per_sum = 1.0f / total;
  }
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int k = q + i * L;
    if (k < d.K && !spare) {
      d.topk_idx[t * d.K + k] = chosen[i];
      d.topk_weights[t * d.K + k] = chosen[i] >= 0 ? w[i] * per_sum * d.scale : 0.0f;
    }
  }
}

// dL/dlogits from dL/dweights.  With s the scores of the token, c the scale,
// g the gradient of its weights and w the weights without c:
//   renormalised softmax:  dz_k = c w_k (g_k - sum_j g_j w_j) on the chosen experts, 0 elsewhere
//   renormalised sigmoid:  the same times (1 - s_k)
//   plain sigmoid:         dz_k = c g_k s_k (1 - s_k)
//   plain softmax:         dz_e = c s_e ([e chosen] g_e - sum_j g_j s_j) on every expert
// The selection itself, and with it the bias, has no gradient.  The row is
// written first as if none were chosen (zeros, or the plain softmax's second
// term), then the chosen experts over it by the same warp.
template <int L, int NP, bool DENSE, typename In>
__global__ void __launch_bounds__(32 * kRouteWarps) ep_route_backward_kernel(RouteBwdDev d) {
  constexpr int V = 4 * NP, kTokens = 32 / L, kSlots = L < 16 ? 16 / L : 1;
  pdl_wait();
  const Lanes<L, NP> at;
  const int q = at.q;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5)) * kTokens;
  if (t0 >= d.T) return;
  const bool spare = t0 + at.tok >= d.T;  // repeats the last token and stores nothing
  const int64_t t = spare ? d.T - 1 : t0 + at.tok;
  const In* row = static_cast<const In*>(d.logits) + t * d.ld;
  In* to = static_cast<In*>(d.grad_logits) + t * d.E;

  int e[kSlots];
  float g[kSlots], zk[kSlots], dz[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int k = q + i * L;
    e[i] = -1;
    g[i] = 0.0f;
    zk[i] = -INFINITY;
    if (k < d.K) {
      const int64_t x = d.topk_idx[t * d.K + k];
      if (x >= 0 && x < d.E) {
        const float v = to_f32(row[x]);
        e[i] = static_cast<int>(x);
        if (available(v)) {
          g[i] = d.grad_weights[t * d.K + k] * d.scale;
          zk[i] = v;
        }
      }
    }
  }
  if constexpr (DENSE) {
    float z[V];
    load_row<L, NP, In>(row, at, d.E, d.vec, z);
    const float top = row_max<L, NP>(z);
    float total = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      z[j] = quick_exp(z[j] - top);
      total += z[j];
    }
    total = lanes_sum<L>(total);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      dz[i] = zk[i] == -INFINITY ? 0.0f : expf(zk[i] - top) / total;  // s_k
      dot += g[i] * dz[i];
    }
    dot = lanes_sum<L>(dot);
#pragma unroll
    for (int i = 0; i < kSlots; ++i) dz[i] *= g[i] - dot;
    const float f = total > 0.0f ? -dot / total : 0.0f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = z[4 * i + c] * f;
      if (!spare) store4(to, at.expert(4 * i), d.E, d.vec_out, x);
    }
  } else {
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (!spare) store4(to, at.expert(4 * i), d.E, d.vec_out, zero);
    float m = -INFINITY;
    if (!d.sigmoid) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i) m = fmaxf(m, zk[i]);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    }
    float s[kSlots], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      s[i] = zk[i] == -INFINITY ? 0.0f : d.sigmoid ? sigmoid(zk[i]) : expf(zk[i] - m);
      sum += s[i];
    }
    float dot = 0.0f;
    if (d.renorm) {
      sum = lanes_sum<L>(sum);
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        s[i] = sum == 0.0f ? 0.0f : s[i] / sum;
        dot += g[i] * s[i];
      }
      dot = lanes_sum<L>(dot);
    }
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      dz[i] = s[i] * (g[i] - dot);
      // 1 - sigmoid without the cancellation
      if (d.sigmoid) dz[i] *= zk[i] == -INFINITY ? 0.0f : 1.0f / (1.0f + expf(zk[i]));
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (e[i] >= 0 && !spare) to[e[i]] = static_cast<In>(dz[i]);
}

template <int L, int NP, typename In>
cudaError_t route_lanes(const RouteDev& d, cudaStream_t stream) {
  const int tokens = kRouteWarps * (32 / L);
  const unsigned grid = static_cast<unsigned>((d.T + tokens - 1) / tokens);
  if (d.bias != nullptr) return launch_pdl(ep_route_kernel<L, NP, kScores, In>, grid, 32 * kRouteWarps, stream, d);
  if (d.G > 1) return launch_pdl(ep_route_kernel<L, NP, kGroupLogits, In>, grid, 32 * kRouteWarps, stream, d);
  return launch_pdl(ep_route_kernel<L, NP, kLogits, In>, grid, 32 * kRouteWarps, stream, d);
}

// Few tokens do not fill the SMs eight lanes each, and end sooner a warp each:
// 2048 x 256 6.3 us against 8.3, 4096 x 128 6.4 against 8.4; 16384 x 256 18.5
// against 12.5.
constexpr int64_t kFewTokens = 4096;

template <int L>
cudaError_t route_packed(const RouteDev& d, cudaStream_t stream) {
  const int tokens = kRouteWarps * (32 / L);
  const unsigned grid = static_cast<unsigned>((d.T + tokens - 1) / tokens);
  return launch_pdl(ep_route_packed_kernel<L>, grid, 32 * kRouteWarps, stream, d);
}

template <typename In>
cudaError_t route_type(const RouteDev& d, cudaStream_t stream) {
  if (d.T > kFewTokens) {
    if (d.E <= 64) return route_lanes<8, 2, In>(d, stream);
    if (d.E <= 128) return route_lanes<8, 4, In>(d, stream);
    if (d.E <= 256) return route_lanes<8, 8, In>(d, stream);
    if (d.E <= 512) return route_lanes<16, 8, In>(d, stream);  // 65536 x 512 56.1 us, with eight lanes 74.7
  }
  if (d.E <= 128) return route_lanes<32, 1, In>(d, stream);
  if (d.E <= 256) return route_lanes<32, 2, In>(d, stream);
  if (d.E <= 512) return route_lanes<32, 4, In>(d, stream);
  return route_lanes<32, 16, In>(d, stream);
}

template <int L, int NP, typename In>
cudaError_t route_backward_lanes(const RouteBwdDev& d, cudaStream_t stream) {
  const int tokens = kRouteWarps * (32 / L);
  const unsigned grid = static_cast<unsigned>((d.T + tokens - 1) / tokens);
  if (!d.sigmoid && !d.renorm)
    return launch_pdl(ep_route_backward_kernel<L, NP, true, In>, grid, 32 * kRouteWarps, stream, d);
  return launch_pdl(ep_route_backward_kernel<L, NP, false, In>, grid, 32 * kRouteWarps, stream, d);
}

template <typename In>
cudaError_t route_backward_type(const RouteBwdDev& d, cudaStream_t stream) {
  if (d.E <= 128) return route_backward_lanes<8, 4, In>(d, stream);
  if (d.E <= 256) return route_backward_lanes<8, 8, In>(d, stream);
  if (d.E <= 512) return route_backward_lanes<8, 16, In>(d, stream);
  return route_backward_lanes<32, 16, In>(d, stream);
}

}  // namespace

cudaError_t launch_route(const RouteDev& d, bool bf16, cudaStream_t stream) {
  if (bf16 && d.bias == nullptr && d.G == 1 && d.K <= kListed) {
    // Lanes a token: 4096 x 256 3.0 us with eight, 3.1 with 16; 2048 x 512 4.1 with
    // eight, 3.1 with 16 (65536 x 512 33 and 38); 2048 x 2048 7.6 with 16, 7.0 with 32.
    if (d.E <= 256) return route_packed<8>(d, stream);
    if (d.E <= 512) return route_packed<16>(d, stream);
    return route_packed<32>(d, stream);
  }
  return bf16 ? route_type<__nv_bfloat16>(d, stream) : route_type<float>(d, stream);
}

cudaError_t launch_route_backward(const RouteBwdDev& d, bool bf16, cudaStream_t stream) {
  return bf16 ? route_backward_type<__nv_bfloat16>(d, stream) : route_backward_type<float>(d, stream);
}

}  // namespace ep
