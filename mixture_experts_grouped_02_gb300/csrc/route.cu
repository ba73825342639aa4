// route.cu -- experts of each token from its router logits, and the gradient
// of the logits.
//
//   p = softmax(l) over the E experts, or sigmoid(l);  choice = p + bias
//   groups of E / G experts: a group's score is the sum of its two largest
//   choices, or the largest; the topk_groups best groups stay
//   ids: the K largest choices that are left, in descending order, ties to the
//   lower id;  weights = scale * p[ids], over their sum when renormalised
//
// A warp per token, the row in registers: a lane holds up to V consecutive experts, a
// lower lane lower ids, and a group is a power of two of lanes (the last of which may
// hold fewer or none), so that a group's best two are found by shuffles among its
// lanes alone.  V is the smallest power of two for which this fits a warp.
//
// What is chosen hangs on the last bits of two choices, and fp32 scores are off
// by more than the gaps that some tokens of a large batch have (8192 tokens of
// 256 experts: about one token's choice in a batch).  Where the choice is simply
// that of the logits (no bias, no sums of two scores) it is made on them.  Otherwise
// a token is first routed by fp32 scores, which settles it unless two neighbours of
// the order come nearer than 2^-18 of the scores, several times their error (one
// token in some hundred); then the candidates, or, where the groups that stay are
// open too or a value is not finite, all experts are put in order by scores that are
// sums of two floats, exact to 2^-44 (for scores above e^-86; lower ones count as
// zero): exp by a table of 2^(j/32) and a short polynomial (P. T. P. Tang, Table-driven
// implementation of the exponential function, 1989) in the exact two-float sums and
// products of T. J. Dekker (1971) and D. E. Knuth.  A choice becomes a 64-bit key
// whose unsigned order is the choices'; key 0 is below all of them and marks what
// cannot be chosen.
//
// Bound by instructions and by what they wait for, not by HBM.  16384 tokens, top 8 of 256
// experts, sigmoid, bias and 8 groups: 823 instructions a token where HBM would allow 100, which
// fill two thirds of an SM's issue slots while it has warps and half of the kernel's time; the
// rest are the rounds of the choice, each of which needs the one before it, and the first and
// last warps.  GB300, operands from HBM, us (at the copy rate): 18.9 to 19.4 (2.6), every token
// by two-float scores 46; softmax 12.6 to 12.9 (2.6; 647 instructions), of 1024 experts and 8192
// tokens 23.4 (5.0); one token 3.0.
//
// Weights are fp32, from the logits by expf; renormalised ones relative to the
// largest chosen, so that they do not underflow together.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float logit_at(const void* logits, int bf16, long long i) {
  if (bf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(logits)[i]);
  return static_cast<const float*>(logits)[i];
}

// Which experts a lane holds: e, e + 1, ... up to n of them.
struct Held {
  int e, n;
};
__device__ __forceinline__ Held held(const RouteTokensArgs& a, int lane, int V) {
  const int g = lane >> a.lanes_log2, at = (lane & (a.lanes - 1)) * V;
  const int e = g * a.run + at;
  return {e, e < a.E ? max(0, min(V, a.run - at)) : 0};
}

// A lane's elements of a row, `fill` past them; wide: rows on 16 bytes (8 for bf16),
// e and n multiples of 4.
template <int V>
__device__ __forceinline__ void load_row(const void* p, int bf16, bool wide, long long row, Held h,
                                         float fill, float (&v)[V]) {
  if constexpr (V >= 4) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        float4 q = make_float4(fill, fill, fill, fill);
        if (i < h.n) {
          if (bf16) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(
                static_cast<const __nv_bfloat16*>(p) + row + h.e + i));
            q = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                            __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
          } else {
            q = __ldg(
                reinterpret_cast<const float4*>(static_cast<const float*>(p) + row + h.e + i));
          }
        }
        v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = i < h.n ? logit_at(p, bf16, row + h.e + i) : fill;
}

// ---------------------------------------------------------- sums of two floats

struct F2 {  // hi + lo, |lo| at most half an ulp of hi
  float hi, lo;
};

__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
// |a| >= |b|
__device__ __forceinline__ F2 quick_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  const F2 s = two_sum(a.hi, b.hi);
  return quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ F2 divide(F2 a, F2 b) {
  const float y = __frcp_rn(b.hi);
  const float q = __fmul_rn(a.hi, y);
  const float r = __fadd_rn(__fmaf_rn(-q, b.hi, a.hi), __fmaf_rn(-q, b.lo, a.lo));
  return quick_sum(q, __fmul_rn(r, y));
}

// 2^(j / 32) as sums of two floats.
__device__ const float2 kExp2Table[32] = {
    {1.000000000e+00f, 0.000000000e+00f}, {1.021897197e+00f, -4.811559862e-08f},
    {1.044273734e+00f, 4.833470157e-08f}, {1.067140460e+00f, -5.933751979e-08f},
    {1.090507746e+00f, -1.307753994e-08f}, {1.114386797e+00f, -5.435540018e-08f},
    {1.138788581e+00f, 5.386222313e-08f}, {1.163724899e+00f, -4.051441493e-08f},
    {1.189207077e+00f, 3.797635273e-08f}, {1.215247393e+00f, -3.267394888e-08f},
    {1.241857767e+00f, 4.496838102e-08f}, {1.269050956e+00f, 1.419333318e-09f},
    {1.296839595e+00f, -4.018999533e-08f}, {1.325236678e+00f, -3.496373324e-08f},
    {1.354255557e+00f, -1.012334927e-08f}, {1.383909941e+00f, -5.875577358e-08f},
    {1.414213538e+00f, 2.420323497e-08f}, {1.445180774e+00f, 3.324199938e-08f},
    {1.476826191e+00f, -4.500898854e-08f}, {1.509164453e+00f, -2.495937323e-08f},
    {1.542210817e+00f, 8.070904833e-09f}, {1.575980902e+00f, -5.661025426e-08f},
    {1.610490322e+00f, 9.836217174e-09f}, {1.645755529e+00f, -5.124972091e-08f},
    {1.681792855e+00f, -2.475532668e-08f}, {1.718619347e+00f, -4.849617596e-08f},
    {1.756252170e+00f, -9.235770371e-09f}, {1.794709086e+00f, -1.141504491e-08f},
    {1.834008098e+00f, -1.123927795e-08f}, {1.874167681e+00f, -4.663005626e-08f},
    {1.915206552e+00f, 9.845328108e-09f}, {1.957144141e+00f, -1.702180441e-08f},
};

// exp(d) for d <= 0: d = (32 m + j) ln 2 / 32 + r with |r| <= ln 2 / 64, exp(d) =
// 2^m 2^(j/32) (1 + r + r^2/2 + r^3/6 + r^4/24 + r^5/120).  The next term is
// below 2^-48, the polynomial's part in one float below 2^-22.
__device__ __forceinline__ F2 exp2f(F2 d) {
  // ln 2 / 32 as a sum of three: 11 bits, so that k times it is exact, 24 and 24
  constexpr float kC1 = 2.165222168e-02f, kC2 = 8.627713214e-06f, kC3 = -4.032912513e-13f;
  if (!(d.hi > -86.0f)) return {0.0f, 0.0f};
  const float k = rintf(d.hi * 46.16624131f);
  const float p = __fmul_rn(k, kC2);
  const F2 r0 = two_sum(__fmaf_rn(-k, kC1, d.hi), -p);
  const F2 r = quick_sum(r0.hi, r0.lo + (d.lo - __fmaf_rn(k, kC2, -p)) - k * kC3);
  const float rr = __fmul_rn(r.hi, r.hi);
  const float rr_lo = __fmaf_rn(r.hi, r.hi, -rr) + 2.0f * r.hi * r.lo;
  const float tail =
      rr * r.hi * (1.6666667e-1f + r.hi * (4.1666668e-2f + r.hi * 8.3333338e-3f));
  const F2 q0 = quick_sum(r.hi, 0.5f * rr);
  const float q_lo = q0.lo + (r.lo + (0.5f * rr_lo + tail));
  const int ki = static_cast<int>(k);
  const float2 t = __ldg(&kExp2Table[ki & 31]);
  const float tq = __fmul_rn(t.x, q0.hi);
  const float tq_lo = __fmaf_rn(t.x, q0.hi, -tq) + (t.x * q_lo + t.y * q0.hi);
  const F2 s = quick_sum(t.x, tq);
  const F2 e = quick_sum(s.hi, s.lo + (tq_lo + t.y));
  const float scale = __int_as_float((127 + (ki >> 5)) << 23);
  return {e.hi * scale, e.lo * scale};
}

// 1 / (1 + e^-l)
__device__ __forceinline__ F2 sigmoid2f(float l) {
  const F2 e = exp2f({-fabsf(l), 0.0f});
  const F2 d = add({1.0f, 0.0f}, e);
  return divide(l >= 0.0f ? F2{1.0f, 0.0f} : e, d);
}

// ------------------------------------------------------------------------ keys

__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);  // -0 as 0
  return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
// 0 for a NaN.  An infinite hi has no lo.
__device__ __forceinline__ uint64_t key_of(F2 v) {
  if (v.hi != v.hi) return 0;
  const float lo = fabsf(v.hi) == INFINITY ? 0.0f : v.lo;
  return static_cast<uint64_t>(ordered(v.hi)) << 32 | ordered(lo);
}
__device__ __forceinline__ F2 value_of(uint64_t key) {
  return {from_ordered(static_cast<uint32_t>(key >> 32)),
          from_ordered(static_cast<uint32_t>(key))};
}

// The two largest keys of a group, in order.
struct Best2 {
  uint64_t a, b;
};
__device__ __forceinline__ void insert(Best2& s, uint64_t k) {
  if (k > s.a) {
    s.b = s.a;
    s.a = k;
  } else if (k > s.b) {
    s.b = k;
  }
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int d) {
  return static_cast<uint64_t>(__shfl_xor_sync(kFull, static_cast<unsigned>(v >> 32), d)) << 32 |
         __shfl_xor_sync(kFull, static_cast<unsigned>(v), d);
}
__device__ __forceinline__ Best2 merged(Best2 s, int d) {
  const uint64_t a = shfl_xor64(s.a, d), b = shfl_xor64(s.b, d);
  insert(s, a);
  insert(s, b);
  return s;
}

// The lowest lane that holds the warp's largest key.
__device__ __forceinline__ int argmax_lane(uint64_t key, uint64_t& top) {
  const unsigned hi = static_cast<unsigned>(key >> 32), lo = static_cast<unsigned>(key);
  const unsigned m = __reduce_max_sync(kFull, hi);
  const unsigned n = __reduce_max_sync(kFull, hi == m ? lo : 0u);
  top = static_cast<uint64_t>(m) << 32 | n;
  return __ffs(__ballot_sync(kFull, key == top)) - 1;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
  return v;
}

// exp(l - m) with l <= m: 1 for the largest, also an infinite one, 0 for -inf (in
// a row of nothing else too) and for a NaN.
__device__ __forceinline__ float exp_below(float l, float m) {
  return !(l > -INFINITY) ? 0.0f : l == m ? 1.0f : expf(l - m);
}

// ---------------------------------------------------------------------- forward

// Keys of the groups that do not stay become 0.
template <int V>
__device__ __forceinline__ void keep_groups(const RouteTokensArgs& a, uint64_t (&key)[V], Held h,
                                            int lane) {
  auto score = [&](Best2 s) {
    // one expert to a group, or a second one that cannot be chosen
    if (!a.top2 || s.b == 0) return s.a;
    const F2 u = value_of(s.a), v = value_of(s.b);
    const float sum = u.hi + v.hi;  // infinite or not a number where a choice is infinite
    return key_of(fabsf(sum) < INFINITY ? add(u, v) : F2{sum, 0.0f});
  };
  if (a.by_lanes) {
    Best2 s = {0, 0};
#pragma unroll
    for (int i = 0; i < V; ++i) insert(s, key[i]);
    for (int d = 1; d < a.lanes; d <<= 1) s = merged(s, d);
    // the group's first lane stands for it: lower lanes are lower groups
    const int first = lane & ~(a.lanes - 1);
    uint64_t mine = lane == first ? score(s) : 0;
    bool stays = false;
    for (int k = 0; k < a.topk_groups; ++k) {
      uint64_t top;
      const int winner = argmax_lane(mine, top);
      if (top == 0) break;
      if (lane == winner) mine = 0;
      stays |= first == winner;
    }
    if (!stays) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = 0;
    }
  } else {
    // lane g gets group g's score, one group at a time
    const int size = a.E / a.groups;
    uint64_t mine = 0;
    for (int g = 0; g < a.groups; ++g) {
      Best2 s = {0, 0};
#pragma unroll
      for (int i = 0; i < V; ++i) insert(s, (h.e + i) / size == g ? key[i] : 0);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) s = merged(s, d);
      if (lane == g) mine = score(s);
    }
    unsigned stays = 0;
    for (int k = 0; k < a.topk_groups; ++k) {
      uint64_t top;
      const int winner = argmax_lane(mine, top);
      if (top == 0) break;
      if (lane == winner) mine = 0;
      stays |= 1u << winner;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < h.n && !((stays >> ((h.e + i) / size)) & 1u)) key[i] = 0;
  }
}

// e^(l - m) of the exact scores, with the conventions of exp_below.
__device__ __forceinline__ F2 softmax_part(float l, float m) {
  return !(l > -INFINITY) ? F2{0.0f, 0.0f}
         : l == m         ? F2{1.0f, 0.0f}
         : m == INFINITY  ? F2{0.0f, 0.0f}
                          : exp2f(two_sum(l, -m));
}
__device__ __forceinline__ F2 warp_total(F2 v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    v = add(v, {__shfl_xor_sync(kFull, v.hi, d), __shfl_xor_sync(kFull, v.lo, d)});
  return v;
}

// A token's choice in full: the id of choice `lane`, -1 where nothing was left.  m: the
// row's largest logit (softmax).
template <int V, bool BY_SCORE>
__device__ __forceinline__ int choose_exact(const RouteTokensArgs& a, const float (&l)[V], Held h,
                                            float m, int lane) {
  uint64_t key[V];
  if constexpr (BY_SCORE) {
    F2 p[V];
    if (a.softmax) {
      F2 total = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        p[i] = softmax_part(l[i], m);
        total = add(total, p[i]);
      }
      total = warp_total(total);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (total.hi > 0.0f) p[i] = divide(p[i], total);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] = sigmoid2f(l[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (a.bias != nullptr && i < h.n) {
        const float b = a.bias[h.e + i];
        p[i] = fabsf(b) == INFINITY ? F2{b, 0.0f} : add(p[i], {b, 0.0f});
      }
      key[i] = i < h.n && l[i] == l[i] ? key_of(p[i]) : 0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = i < h.n ? key_of({l[i], 0.0f}) : 0;
  }
  if (a.groups > 1) keep_groups<V>(a, key, h, lane);

  // K rounds: every lane's largest key (the lowest id of equal ones), then the
  // warp's
  int my_id = -1;
  for (int k = 0; k < a.K; ++k) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    uint64_t top;
    const int winner = argmax_lane(best, top);
    if (top == 0) break;  // nothing left that compares
    const int id = __shfl_sync(kFull, h.e + at, winner);
    if (lane == winner) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at) key[i] = 0;
    }
    if (lane == k) my_id = id;
  }
  return my_id;
}

// The largest of the lanes' values; the lowest lane that has it.
__device__ __forceinline__ float warp_top(float v, int& lane) {
  const float top = from_ordered(__reduce_max_sync(kFull, ordered(v)));
  lane = __ffs(__ballot_sync(kFull, v == top)) - 1;
  return top;
}

// A lane's keys in descending order: exchanges of a bitonic network.
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[V]) {
#pragma unroll
  for (int n = 2; n <= V; n *= 2) {
#pragma unroll
    for (int d = n / 2; d > 0; d /= 2) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = i ^ d;
        if (j <= i) continue;
        const uint32_t hi = max(k[i], k[j]), lo = min(k[i], k[j]);
        k[i] = (i & n) != 0 && n < V ? lo : hi;
        k[j] = (i & n) != 0 && n < V ? hi : lo;
      }
    }
  }
}

// The same by fp32 scores, or by the logits where these are the choices; false
// where it is not settled by them.  A key is a choice's
// ordered bits, the last log2 V of them replaced by the expert's place in its lane
// (lower ones larger), so that a lane can sort its experts once and give one up a
// round; choices whose keys differ in the place alone are not settled (bf16 logits
// have none of these bits, their ties go to the lower id as they are).
// Where only the order of neighbours is open, those after the K-th too until one is
// clearly above the next, the lanes' candidates are put in order by exact scores, one to a
// lane, instead of the whole row's (16384 tokens of 256 experts in 8 groups: 19.8 us against
// 23.4, where one token in a hundred has such neighbours and the grid's end waits for them).
template <int V, bool BY_SCORE>
__device__ __forceinline__ bool choose_fast(const RouteTokensArgs& a, const float (&l)[V], Held h,
                                            float m, float sum, long long row, int lane,
                                            int& my_id) {
  constexpr float kNear = V <= 8 ? 3.8146973e-6f : 1.5258789e-5f;  // 2^-18, 2^-16
  // where a lane holds no expert c is -inf, and so is the least that is not chosen
  float c[V], most = 1.0f;  // most: the largest score there can be
  float sound = 0.0f;       // not finite where a choice is not
  if constexpr (BY_SCORE) {
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = 0.0f;
    if (a.bias != nullptr) load_row<V>(a.bias, 0, a.wide_bias, 0, h, 0.0f, bias);
    if (a.softmax) {
      most = __frcp_rn(sum);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        c[i] = fmaf(exp_below(l[i], m), most, bias[i]);
        sound += l[i] == l[i] ? c[i] : l[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const int j = V > 1 ? i + 1 : i;
        const float2 e = exp2_fast(__fmul2_rn(make_float2(l[i], l[j]), both(-1.44269504f)));
        const float2 p = __fadd2_rn(inverse_fast(__fadd2_rn(e, both(1.0f))),
                                    make_float2(bias[i], bias[j]));
        c[i] = p.x, c[j] = p.y;
        sound += p.x + p.y;  // a NaN logit's is NaN
      }
    }
    if (h.n < V) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i >= h.n) c[i] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = l[i];
      if (a.groups > 1 && i < h.n) sound += l[i];
    }
  }
  if (!__all_sync(kFull, fabsf(sound) < INFINITY)) return false;
  bool stays = true;
  if (a.groups > 1) {
    if (!a.by_lanes) return false;
    float s = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      second = fmaxf(second, fminf(s, c[i]));
      s = fmaxf(s, c[i]);
    }
    for (int d = 1; d < a.lanes; d <<= 1) {
      const float s1 = __shfl_xor_sync(kFull, s, d);
      const float s2 = __shfl_xor_sync(kFull, second, d);
      second = fmaxf(fmaxf(second, s2), fminf(s, s1));
      s = fmaxf(s, s1);
    }
    // how far from the exact one a group's score may be: a sum's terms count, which may
    // be far larger than the sum
    float off = most + fabsf(s);
    if (a.top2 && a.run > 1) {
      off += fabsf(second);
      s += second;
    }
    off *= kNear;
    // the group's first lane stands for it
    const int first = lane & ~(a.lanes - 1);
    const bool group = lane == first && h.n > 0;
    float left = group ? s : -INFINITY;
    stays = false;
    for (int k = 0; k < a.topk_groups; ++k) {
      int winner;
      warp_top(left, winner);
      if (lane == winner) left = -INFINITY;
      stays |= first == winner;
    }
    if (BY_SCORE && a.topk_groups < a.groups) {
      // every group that stays has to be clearly above every one that goes; a NaN of two
      // infinities is not
      const float low = group && stays ? fmaxf(s - off, -INFINITY) : INFINITY;
      const float high = group && !stays ? fminf(s + off, INFINITY) : -INFINITY;
      if (__reduce_min_sync(kFull, ordered(low)) <= __reduce_max_sync(kFull, ordered(high)))
        return false;
    }
  }
  constexpr uint32_t kPlace = V - 1;
  const uint32_t none = ordered(-INFINITY) | kPlace;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = (ordered(c[i]) & ~kPlace) | (V - 1u - i);
    if (!BY_SCORE && c[i] != c[i]) key[i] = 0;
  }
  sort_keys<V>(key);
  if (!stays) key[0] = 0;  // the others come after it
  uint32_t my_key = 0, next = 0;
  int my_lane = 0;
  // choice k, whose key is `next`, to lane k
  auto take = [&](int k) {
    const unsigned who = __ballot_sync(kFull, ((key[0] ^ next) & ~kPlace) == 0);
    const int winner = __ffs(who) - 1;
    const uint32_t taken = __shfl_sync(kFull, key[0], winner);
    if (lane == winner) {
#pragma unroll
      for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
      key[V - 1] = 0;
    }
    if (lane == k) {
      my_key = taken;
      my_lane = winner;
    }
    next = __reduce_max_sync(kFull, key[0]);
  };
  next = __reduce_max_sync(kFull, key[0]);
  for (int k = 0; k < a.K; ++k) take(k);
  if (!__all_sync(kFull, lane >= a.K || my_key > none)) return false;
  auto apart = [&](uint32_t above, uint32_t below) {
    const float u = from_ordered(above & ~kPlace), v = from_ordered(below & ~kPlace);
    return BY_SCORE ? u - v > kNear * (most + fabsf(u)) : a.bf16 || u != v;
  };
  auto mine = [&] {
    return held(a, my_lane, V).e + static_cast<int>(V - 1u - (my_key & kPlace));
  };
  // every choice against the one after it, the last against the first left out
  uint32_t after = __shfl_down_sync(kFull, my_key, 1);
  if (lane == a.K - 1) after = next;
  if (__all_sync(kFull, lane >= a.K || after <= none || apart(my_key, after))) {
    if (lane < a.K) my_id = mine();
    return true;
  }
  if constexpr (!BY_SCORE) return false;
  int n = a.K;
  while (next > none && !apart(__shfl_sync(kFull, my_key, n - 1), next)) {
    if (n == 32) return false;
    take(n++);
  }
  F2 p = {0.0f, 0.0f};
  if (a.softmax) {
#pragma unroll
    for (int i = 0; i < V; ++i) p = add(p, softmax_part(l[i], m));
    p = warp_total(p);
  }
  const int id = lane < n ? mine() : a.E;
  uint64_t exact = 0;
  if (lane < n) {
    const float x = logit_at(a.logits, a.bf16, row + id);
    p = a.softmax ? divide(softmax_part(x, m), p) : sigmoid2f(x);
    if (a.bias != nullptr) p = add(p, {a.bias[id], 0.0f});
    exact = key_of(p);
  }
  // the candidates ahead of a lane's own, ties to the lower id
  int ahead = 0;
  for (int i = 0; i < n; ++i) {
    const unsigned hi = __shfl_sync(kFull, static_cast<unsigned>(exact >> 32), i);
    const unsigned lo = __shfl_sync(kFull, static_cast<unsigned>(exact), i);
    const uint64_t k = static_cast<uint64_t>(hi) << 32 | lo;
    const int other = __shfl_sync(kFull, id, i);
    ahead += k > exact || (k == exact && other < id);
  }
  for (int i = 0; i < n; ++i) {
    const int to = __shfl_sync(kFull, ahead, i), other = __shfl_sync(kFull, id, i);
    if (lane == to && lane < a.K) my_id = other;
  }
  return true;
}

// BY_SCORE: a bias or sums of two scores decide; otherwise the order of the logits does.
template <int V, bool BY_SCORE>
__global__ void __launch_bounds__(32 * kWarps)
    route_tokens_kernel(const __grid_constant__ RouteTokensArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const long long row = t * a.E;
  float l[V];
  const Held h = held(a, lane, V);
  load_row<V>(a.logits, a.bf16, a.wide, row, h, -INFINITY, l);

  // the row's largest logit and the sum of the exponentials below it
  float m = -INFINITY, sum = 0.0f;
  if (a.softmax) {
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    if (!a.renormalize || BY_SCORE) {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += exp_below(l[i], m);
      sum = warp_sum(sum);
    }
  }

  int my_id = -1;
  if (!choose_fast<V, BY_SCORE>(a, l, h, m, sum, row, lane, my_id))
    my_id = choose_exact<V, BY_SCORE>(a, l, h, m, lane);

  const bool mine = lane < a.K && my_id >= 0;
  if (__any_sync(kFull, lane < a.K && my_id < 0) && lane == 0)
    report_error(a.status, MOE_ERR_DEVICE_BAD_ID);
  const float lk = mine ? logit_at(a.logits, a.bf16, row + my_id) : -INFINITY;
  float w;
  if (a.softmax) {
    w = exp_below(lk, a.renormalize ? warp_max(lk) : m);
  } else {
    // relative to the largest when all are small: e^(l - c) / (1 + e^l)
    const float c = a.renormalize ? fminf(warp_max(lk), 0.0f) : 0.0f;
    const float e = expf(-fabsf(lk));
    w = lk == -INFINITY ? 0.0f
        : lk >= 0.0f    ? __fdividef(1.0f, 1.0f + e)
                        : __fdividef(c < 0.0f ? expf(lk - c) : e, 1.0f + e);
  }
  if (a.renormalize) sum = warp_sum(mine ? w : 0.0f);
  if (a.renormalize || a.softmax) w = sum > 0.0f ? w / sum : 0.0f;
  if (lane < a.K) {
    a.ids[t * a.K + lane] = mine ? my_id : 0;
    a.weights[t * a.K + lane] = mine ? w * a.scale : 0.0f;
  }
}

template <int V>
cudaError_t launch_v(const RouteTokensArgs& a, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3((a.T - 1) / kWarps + 1), dim3(32 * kWarps), 0, s, attr);
  return cudaLaunchKernelEx(&cfg,
                            a.bias != nullptr || (a.groups > 1 && a.top2)
                                ? route_tokens_kernel<V, true>
                                : route_tokens_kernel<V, false>,
                            a);
}

// ---------------------------------------------------------------------- gradient
// With q the weights before the scale and g the weights' gradient times the scale:
//   sigmoid               dl_k = g_k p_k (1 - p_k)
//   sigmoid, renormalised dl_k = q_k (g_k - sum g q) (1 - p_k)
//   softmax, renormalised dl_k = q_k (g_k - sum g q)
//   softmax               dl_e = p_e (g_e - sum g p), g_e = 0 where not chosen
// and 0 elsewhere.  A warp per token; the row is put together in shared memory
// (an id that comes twice adds up, in order) and written whole.  A chain of loads,
// shuffles and one write: 8191 tokens of 128 experts 6.0 us (0.7 at the copy rate),
// one token 2.2.
__global__ void __launch_bounds__(32 * kWarps)
    route_tokens_grad_kernel(const __grid_constant__ RouteTokensGradArgs a) {
  extern __shared__ float rows[];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (t >= a.T) return;
  float* d = rows + warp * a.E;
  const long long row = t * a.E;
  int id = lane < a.K ? a.ids[t * a.K + lane] : -1;
  const bool bad = lane < a.K && (id < 0 || id >= a.E);
  if (__any_sync(kFull, bad) && lane == 0) report_error(a.status, MOE_ERR_DEVICE_BAD_ID);
  const bool mine = lane < a.K && !bad;
  const float l = mine ? logit_at(a.logits, a.bf16, row + id) : -INFINITY;
  const float g = mine ? a.grad[t * a.K + lane] * a.scale : 0.0f;
  float v = 0.0f;  // this choice's part of its logit's gradient
  if (a.softmax && !a.renormalize) {
    float m = -INFINITY, sum = 0.0f;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, logit_at(a.logits, a.bf16, row + e));
    m = warp_max(m);
    for (int e = lane; e < a.E; e += 32) {
      const float x = exp_below(logit_at(a.logits, a.bf16, row + e), m);
      d[e] = x;
      sum += x;
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const float p = exp_below(l, m) * inv;
    const float dot = warp_sum(mine ? g * p : 0.0f);
    for (int e = lane; e < a.E; e += 32) d[e] = -(d[e] * inv) * dot;
    v = g * p;
  } else {
    for (int e = lane; e < a.E; e += 32) d[e] = 0.0f;
    if (a.softmax) {
      const float x = exp_below(l, warp_max(l));
      const float sum = warp_sum(mine ? x : 0.0f);
      const float q = sum > 0.0f ? x / sum : 0.0f;
      v = q * (g - warp_sum(mine ? g * q : 0.0f));
    } else {
      const float not_p = l >= 0.0f ? expf(-l) / (1.0f + expf(-l)) : 1.0f / (1.0f + expf(l));
      const float c = a.renormalize ? fminf(warp_max(l), 0.0f) : 0.0f;
      const float p = l == -INFINITY ? 0.0f
                      : l >= 0.0f    ? 1.0f / (1.0f + expf(-l))
                                     : expf(l - c) / (1.0f + expf(l));
      if (a.renormalize) {
        const float sum = warp_sum(mine ? p : 0.0f);
        const float q = sum > 0.0f ? p / sum : 0.0f;
        v = q * (g - warp_sum(mine ? g * q : 0.0f)) * not_p;
      } else {
        v = g * p * not_p;
      }
    }
  }
  __syncwarp();
  for (int k = 0; k < a.K; ++k) {
    if (lane == k && mine) d[id] += v;
    __syncwarp();
  }
  for (int e = lane; e < a.E; e += 32) {
    if (a.bf16)
      static_cast<__nv_bfloat16*>(a.dlogits)[row + e] = __float2bfloat16_rn(d[e]);
    else
      static_cast<float*>(a.dlogits)[row + e] = d[e];
  }
}

}  // namespace

cudaError_t launch_route_tokens(RouteTokensArgs a, cudaStream_t s) {
  // the smallest V for which every group has its lanes; where there is none (with G the
  // next power of two from the groups' number on, more than 1024 / G experts to a group:
  // 3 groups of more than 256, 5 of more than 128) the experts lie through, groups are
  // looked up one by one, and every token is chosen by two-float scores (8192 tokens,
  // 2 of 3 groups: of 256 experts 45 us, of 341 181)
  const int size = a.E / a.groups;
  int V = 1;
  a.by_lanes = 0;
  for (; a.groups > 1 && V <= 32; V *= 2) {
    a.lanes = 1;
    while (a.lanes * V < size) a.lanes *= 2;
    if (a.lanes * a.groups <= 32) {
      a.by_lanes = 1;
      break;
    }
  }
  a.run = size;
  a.lanes_log2 = 0;
  if (!a.by_lanes) {
    a.lanes = 32;
    a.run = a.E;
    for (V = 1; 32 * V < a.E;) V *= 2;
  }
  while (1 << a.lanes_log2 < a.lanes) ++a.lanes_log2;
  a.wide = a.run % 4 == 0 && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
  a.wide_bias = a.run % 4 == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  switch (V) {
    case 1:
      return launch_v<1>(a, s);
    case 2:
      return launch_v<2>(a, s);
    case 4:
      return launch_v<4>(a, s);
    case 8:
      return launch_v<8>(a, s);
    case 16:
      return launch_v<16>(a, s);
    default:
      return launch_v<32>(a, s);
  }
}

cudaError_t launch_route_tokens_grad(const RouteTokensGradArgs& a, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((a.T - 1) / kWarps + 1), dim3(32 * kWarps),
                                            static_cast<size_t>(kWarps) * a.E * 4, s, attr);
  return cudaLaunchKernelEx(&cfg, route_tokens_grad_kernel, a);
}

}  // namespace moe
