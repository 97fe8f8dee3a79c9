// Scored router: scores of all E logits (sigmoid, or softmax over the E), a bias per expert that
// moves the choice but not the weight, the best groups of experts, the best k experts in them,
// and the weights formed from the unbiased scores; then the same stable placement as the plain
// router's (route.cu).
//
// For token t with logits l:
//   s_e = 1 / (1 + exp(-l_e))   or   exp(l_e - max l) / sum exp(l - max l)
//   c_e = s_e + bias_e
//   group g (E / G consecutive experts): the sum of its `group_top` largest c (1 or 2); the
//   `top_groups` groups with the largest sums stay (ties: the lower group);
//   ids = the k largest c in the groups that stay, ties to the lower index, NaN below -inf;
//   w_j = s[ids_j] (divided by their sum if renormalize) * scale.
//
// Choices are those of 64-bit scores: with 8192 tokens of 256 experts some two scores that decide
// a choice lie within one step of 32 bits of each other in almost every call, and the rounding of
// the exponential would then decide.  A token is chosen for in 32 bits first; where two of the
// values that decide lie nearer to each other than those 32 bits can be off, or anything is not
// finite, 64 bits decide.  Weights are formed in 32 bits, and in 64 where they come near the end of those.
//
// The kernels keep nothing between calls and use no scratch: the rows per expert of each chunk of
// tokens wait in the chunk's own part of inv (at least E ints long by the choice of the chunk)
// until the placement kernel, which reads them before it writes that part.  Calls on different
// streams, or captured into graphs, therefore share nothing.
//
// What bounds it: one call's bytes (8192 tokens of 256 experts: 9.4 MB, 1.4 us) are nothing beside the chain
// load - choice - counts - placement of a token.  With many tokens it is that chain still: a warp walks one token's
// rounds of the choice one after another, about 890 instructions a token, and 64 registers leave 32 warps an SM to
// fill its waits (4096 tokens: issue slots busy 47 %, 36 % of the warps resident; 8192: the choice takes about half
// of the time).  So: one launch and one CTA up to 8 tokens; a choice
// over CTAs of a few tokens and a placement that counts the call's ids itself up to 8192 rows; above, the choice,
// counts per chunk, a scan over the chunks and the placement, each set up while the one before runs.  (Counting in
// the choice saves a launch, but chunks that hold their counts are long where experts are many: 32768 tokens of
// 1024 experts, k = 1, 1108 us, now 256; 8192, k = 4, 295, now 82; 1025 of 256, k = 8, 16.1, now 11.2.)
// Measured in a graph, 256 experts in 8 groups, k = 8 (us; in brackets the neighbouring way): 1 token 4.1,
// 8 5.0 (5.5), 16 5.6 (6.5), 67 6.8, 512 8.0 (13.8), 1024 9.6, 8192 20 (44).
#define MOE_OWN_STATUS
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "route_place.cuh"
#include "route_warp.cuh"

namespace moe {

namespace {

constexpr int kOneTokens = 8;        // tokens one CTA routes and places alone (one launch), a warp each
constexpr int kChoiceWarps = 8;      // tokens of a choice's CTA at most
constexpr int kFewRows = 8192;       // rows up to which the placement counts,
constexpr int kFewPlace = 512;       // and rows of such a placement's CTA
constexpr int kChunkMin = 32;        // fewest tokens of a chunk
constexpr int kMaxChunks = 512;
constexpr int kScanSegs = 32;        // threads that share an expert's chunks in the scan
constexpr int kPlaceWarps = 8;        // (256 threads scan up to 1024 counts, four each)

// Programmatic launches: the kernels after this one may be set up now; and the wait for the one before.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_dependency() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Order-preserving 64-bit key; -0.0 equal to +0.0, NaN lowest (0).
__device__ __forceinline__ uint64_t okey(double v) {
  if (v != v) return 0ull;
  const uint64_t b = (uint64_t)__double_as_longlong(v == 0.0 ? 0.0 : v);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ double okey_value(uint64_t k) {
  if (k == 0ull) return __longlong_as_double(0x7FF8000000000000ll);
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}
__device__ __forceinline__ uint64_t umax64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t umin64(uint64_t a, uint64_t b) { return a < b ? a : b; }

__device__ __forceinline__ double shfl_xor_f64(double v, int o) { return __shfl_xor_sync(kFull, v, o); }

// One token by one warp, in 64 bits.  Group g's experts sit in lanes g * lpg .. g * lpg + lpg - 1 (lpg the
// largest power of two with G * lpg <= 32), lane q of the group holding its experts q * PER ..
// q * PER + PER - 1: lanes then ascend in the expert index, so the lowest lane, and in it the
// lowest slot, is the lowest index among equals, and a group's statistics are a butterfly over its
// own lanes.  Lane j < k gets the expert of rank j and its weight.
template <int PER>
__device__ __noinline__ void select_exact(const float* __restrict__ row, const ScoreRule& r, int E, int k, int lane,
                                          int& id, float& weight) {
  using Mask = uint64_t;
  const int gsize = E / r.groups, g = lane / r.lpg, q = lane % r.lpg;
  const int m0 = q * PER;                                // first member of the group in this lane
  const int n = g < r.groups ? min(PER, max(0, gsize - m0)) : 0;
  const int e0 = g * gsize + m0;
  double v[PER];
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = i < n ? (double)__ldg(row + e0 + i) : -INFINITY;
    top = fmax(top, v[i]);                               // (a NaN is passed over)
  }
  double norm = 1.0;                                     // softmax: max and sum over the E logits
  if (r.softmax) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, shfl_xor_f64(top, o));
    norm = 0.0;
  }
  auto score = [&](double l) -> double {
    if (!r.softmax) return 1.0 / (1.0 + exp(-l));
    if (l == top && top > -INFINITY) return 1.0;         // also +inf, whose difference is NaN
    return top > -INFINITY || l != l ? exp(l - top) : 0.0;   // a row of -inf scores 0
  };
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i < n) {
      v[i] = score(v[i]);
      if (r.softmax && v[i] == v[i]) norm += v[i];       // a NaN logit takes no part in the sum
    }
  if (r.softmax) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) norm += shfl_xor_f64(norm, o);
    if (norm == 0.0) norm = 1.0;
  }
  uint64_t key[PER];
  Mask avail = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    key[i] = 0ull;
    if (i < n) {
      const double s = r.softmax ? v[i] / norm : v[i];
      key[i] = okey(r.bias ? s + (double)__ldg(r.bias + e0 + i) : s);
      avail |= (Mask)1 << i;
    }
  }
  if (r.top_groups < r.groups) {
    uint64_t a = 0ull, b = 0ull;                         // the lane's two largest, then the group's
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      b = umax64(b, umin64(a, key[i]));
      a = umax64(a, key[i]);
    }
    for (int o = 1; o < r.lpg; o <<= 1) {
      const uint64_t a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
      b = umax64(umin64(a, a2), umax64(b, b2));
      a = umax64(a, a2);
    }
    const uint64_t mine = okey(r.group_top == 2 ? okey_value(a) + okey_value(b) : okey_value(a));
    int ahead = 0;
    for (int h = 0; h < r.groups; ++h) {
      const uint64_t other = __shfl_sync(kFull, mine, h * r.lpg);
      ahead += other > mine || (other == mine && h < g);
    }
    if (ahead >= r.top_groups) avail = 0;
  }
  uint64_t bk;
  int bi;
  auto rescan = [&]() {
    bk = 0ull;
    bi = -1;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (((avail >> i) & 1) && (bi < 0 || key[i] > bk)) {
        bk = key[i];
        bi = i;
      }
  };
  rescan();
  id = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t hi = bi >= 0 ? (uint32_t)(bk >> 32) : 0u;
    const uint32_t mh = __reduce_max_sync(kFull, hi);
    const bool in = bi >= 0 && hi == mh;
    const uint32_t ml = __reduce_max_sync(kFull, in ? (uint32_t)bk : 0u);
    const int who = __ffs(__ballot_sync(kFull, in && (uint32_t)bk == ml)) - 1;
    const int e = __shfl_sync(kFull, e0 + bi, who);
    if (lane == j) id = e;
    if (lane == who) avail &= ~((Mask)1 << bi);
    rescan();
  }
  double s = 0.0;
  if (lane < k) {
    s = score((double)__ldg(row + id));
    if (r.softmax) s /= norm;
  }
  if (r.renormalize) {
    double sum = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += shfl_xor_f64(sum, o);
    s = sum == 0.0 ? 0.0 : s / sum;
  }
  weight = (float)(s * (double)r.scale);
}

// The same in 32 bits; false (in all lanes) where select_exact has to decide.
//
// An expert's key is the order-preserving image of its biased score with the lowest bits replaced by its
// slot (PER - 1 - i: the lower slot is the larger), so a lane sorts its experts once, by min and max of
// plain integers, and a round of the choice is one maximum over the lanes' heads.
//
// How far off the keys are, with u = 2^-24: a sigmoid (its exponential by 4 u and the rounding of its
// argument, both times s (1 - s) <= 1/4; the reciprocal by 2 u) by less than 4 u; a softmax score by less
// than (PER + 21) u of the row's largest (4 u of its exponential and 0.4 u of the rounding of its argument; the
// sum 4 u of its exponentials, 6 u of the roundings of their arguments, PER + 4 additions; the reciprocal and the
// product); the bias adds u of the sum, the slot 2^-(23 - bits) of it.  near() takes twice that and more: values
// further apart are in the order of their 64-bit values.  Where two that decide
// the order are nearer, the candidates (one a lane) are ordered by their scores in 64 bits.
__device__ __forceinline__ uint32_t fkey(float v) {      // finite, not -0
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float fkey_value(uint32_t k) {
  return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ float rcp_approx(float v) {   // 1 step off at most
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The score of a logit in 64 bits (a softmax's divided by norm).  Not inlined: rarely called.
__device__ __noinline__ double score64(float l, float top, double norm, int softmax) {
  return softmax ? exp((double)l - (double)top) / norm : 1.0 / (1.0 + exp(-(double)l));
}

// A lane's part of a softmax's sum in 64 bits.
__device__ __noinline__ double sum64(const float* l, int n, float top) {
  double sum = 0.0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) sum += exp((double)__ldg(l + i) - (double)top);
  return sum;
}

// FULL: every lane has PER experts (E = 32 PER).
template <int PER, bool FULL>
__device__ __forceinline__ bool select_fast(const float* __restrict__ row, const ScoreRule& r, int E, int k, int lane,
                                            int2* won, int& id, float& weight) {
  constexpr uint32_t kSlot = PER - 1;                    // PER is a power of two
  constexpr float kRel = (PER + 2) / 8388608.0f;         // the slot (one-sided), and u of either value
  const int gsize = E / r.groups, g = lane / r.lpg, q = lane % r.lpg;
  const int m0 = q * PER;
  const int n = FULL ? PER : g < r.groups ? min(PER, max(0, gsize - m0)) : 0;
  const int e0 = FULL ? lane * PER : g * gsize + m0;
  const auto near = [&](uint32_t x, uint32_t y, float tol) {
    const float a = fkey_value(x & ~kSlot), b = fkey_value(y & ~kSlot);
    return fabsf(a - b) <= tol + kRel * fmaxf(fabsf(a), fabsf(b));
  };
  double norm = 1.0;                                     // a softmax's sum in 64 bits, where it is needed
  float top = 0.0f, inv_norm = 1.0f, abs_tol = 0x1p-21f;
  const auto find_norm = [&]() {                         // (called by whole warps)
    norm = sum64(row + e0, n, top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) norm += shfl_xor_f64(norm, o);
  };
  const auto score = [&](float l) -> double { return score64(l, top, norm, r.softmax); };
  float v[PER], add[PER];
  bool odd = false;                                      // a NaN, or something far out
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    v[i] = i < n ? __ldg(row + e0 + i) : -INFINITY;
    add[i] = r.bias != nullptr && i < n ? __ldg(r.bias + e0 + i) : 0.0f;
  }
  if (r.softmax) {
    top = -1e30f;
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, v[i]);
    top = fkey_value(__reduce_max_sync(kFull, fkey(top == 0.0f ? 0.0f : top)));
    if (!(fabsf(top) < 1e30f)) return false;             // (the same in all lanes)
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < n) {
        odd |= v[i] != v[i];
        v[i] = expf(v[i] - top);                         // 0 for a masked logit
        sum += v[i];
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    inv_norm = 1.0f / sum;
    abs_tol = (PER + 24) / 8388608.0f * inv_norm;
  }
  uint32_t key[PER];                                     // 0: none (a finite value's key is not)
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    key[i] = 0;
    if (i < n) {
      float c;
      if (r.softmax) {
        c = v[i] * inv_norm + add[i];
      } else {
        c = rcp_approx(1.0f + __expf(-v[i])) + add[i];   // 0 for a masked logit
      }
      odd |= !(c <= 1e30f);
      c = fmaxf(c, -3e38f);                              // an expert that its bias excludes
      key[i] = (fkey(c) & ~kSlot) | (uint32_t)(PER - 1 - i);
    }
  }
  if (__any_sync(kFull, odd)) return false;
#pragma unroll
  for (int kk = 2; kk <= PER; kk <<= 1)                  // bitonic, descending
#pragma unroll
    for (int jj = kk >> 1; jj > 0; jj >>= 1)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int l = i ^ jj;
        if (l > i) {
          const uint32_t hi = max(key[i], key[l]), lo = min(key[i], key[l]);
          key[i] = (i & kk) == 0 ? hi : lo;
          key[l] = (i & kk) == 0 ? lo : hi;
        }
      }
  if (r.top_groups < r.groups) {
    uint32_t a = key[0], b = key[1];                     // the lane's two largest, then the group's
    for (int o = 1; o < r.lpg; o <<= 1) {
      const uint32_t a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
      b = max(min(a, a2), max(b, b2));
      a = max(a, a2);
    }
    const bool in = FULL || g < r.groups;
    float value = fkey_value(a & ~kSlot), size = fabsf(value);
    if (r.group_top == 2) {
      const float second = fkey_value(b & ~kSlot);
      value = fmaxf(value + second, -3e38f);
      size += fabsf(second);
    }
    const uint32_t mine = in ? fkey(value == 0.0f ? 0.0f : value) : 0u;
    int ahead = 0;
    for (int h = 0; h < r.groups; ++h) {
      const uint32_t other = __shfl_sync(kFull, mine, h * r.lpg);
      ahead += other > mine || (other == mine && h < g);
    }
    bool stays = in && ahead < r.top_groups;
    const float x = fkey_value(__reduce_min_sync(kFull, stays ? mine : 0xFFFFFFFFu));
    const float y = fkey_value(__reduce_max_sync(kFull, stays ? 0u : mine));
    const float most = fkey_value(__reduce_max_sync(kFull, fkey(in ? size : 0.0f)));
    if (x - y <= 2.0f * abs_tol + kRel * most) {         // the groups again, in 64 bits
      // A lane's three largest hold its two largest in 64 bits, unless the fourth is near the second.
      if (__any_sync(kFull, n > 3 && key[3] != 0 && near(key[3], key[1], abs_tol))) return false;
      if (r.softmax) find_norm();
      double c0 = -INFINITY, c1 = -INFINITY;
#pragma unroll 1
      for (int i = 0; i < 3; ++i) {
        const uint32_t kk = i == 0 ? key[0] : i == 1 ? key[1] : key[2];
        const int e = e0 + PER - 1 - (int)(kk & kSlot);
        double c = score(kk != 0 ? __ldg(row + e) : 0.0f);
        if (r.bias && kk != 0) c += (double)__ldg(r.bias + e);
        if (kk == 0) c = -INFINITY;
        c1 = fmax(c1, fmin(c0, c));
        c0 = fmax(c0, c);
      }
      for (int o = 1; o < r.lpg; o <<= 1) {
        const double a2 = shfl_xor_f64(c0, o), b2 = shfl_xor_f64(c1, o);
        c1 = fmax(fmin(c0, a2), fmax(c1, b2));
        c0 = fmax(c0, a2);
      }
      const double exact = r.group_top == 2 ? c0 + c1 : c0;
      ahead = 0;
      for (int h = 0; h < r.groups; ++h) {
        const double other = __shfl_sync(kFull, exact, h * r.lpg);
        ahead += other > exact || (other == exact && h < g);
      }
      stays = in && ahead < r.top_groups;
    }
    if (!stays)
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = 0;
  }
  // Round j: the largest head over the lanes; lane j notes it and whose it was.  One round more than there
  // are places tells how near the first one left out is.
  uint32_t mine = 0, from = 0;
  const auto pop = [&](int j) -> uint32_t {
    const uint32_t m = __reduce_max_sync(kFull, key[0]);
    const uint32_t who = __ffs(__ballot_sync(kFull, key[0] == m)) - 1;
    mine = lane == j ? m : mine;
    from = lane == j ? who : from;
    const bool drop = lane == (int)who;
#pragma unroll
    for (int i = 0; i + 1 < PER; ++i) key[i] = drop ? key[i + 1] : key[i];
    key[PER - 1] = drop ? 0u : key[PER - 1];
    return m;
  };
#pragma unroll 1
  for (int j = 0; j < k; ++j) pop(j);
  const uint32_t next = __reduce_max_sync(kFull, key[0]);   // the best one left out; 0: none is
  const uint32_t before = __shfl_up_sync(kFull, mine, 1);
  const uint32_t last = __shfl_sync(kFull, mine, k - 1);
  const bool open = next != 0 && near(next, last, abs_tol);
  const auto expert = [&]() -> int {
    return (int)(from / r.lpg) * gsize + (int)(from % r.lpg) * PER + (PER - 1 - (int)(mine & kSlot));
  };
  float l;
  if (__any_sync(kFull, open || (lane >= 1 && lane < k && near(mine, before, abs_tol)))) {
    int c = k;                                           // candidates: those chosen and all near the last of them
    uint32_t prev = last;
    for (bool more = open; more;) {
      if (c == 32) return false;
      prev = pop(c++);
      const uint32_t head = __reduce_max_sync(kFull, key[0]);
      more = head != 0 && near(head, prev, abs_tol);
    }
    const int e = lane < c ? expert() : 0;
    l = lane < c ? __ldg(row + e) : top;
    // Without a bias a softmax's order is that of the exponentials, but where unlike ones divided by the sum are one
    // double.  That takes two logits within 2^-50 of each other, so one of them, in 32 bits, under 2^-25; or quotients
    // at the end of 64 bits.
    const bool by_quotient = r.bias != nullptr || (l != 0.0f && fabsf(l) < 0x1p-25f) || (l - top < -600.0f && l > -INFINITY);
    if (r.softmax && __any_sync(kFull, by_quotient)) find_norm();
    double value = score(l);
    if (r.bias) value += (double)__ldg(r.bias + e);
    int rank = 0;
    for (int i = 0; i < c; ++i) {
      const double other = __shfl_sync(kFull, value, i);
      const int oe = __shfl_sync(kFull, e, i);
      rank += other > value || (other == value && oe < e);
    }
    if (lane < c) won[rank] = make_int2(e, __float_as_int(l));
    __syncwarp();
    const int2 w2 = won[lane];
    __syncwarp();                                        // before the next token's
    id = w2.x;
    l = lane < k ? __int_as_float(w2.y) : 0.0f;
  } else {
    id = lane < k ? expert() : 0;
    l = lane < k ? __ldg(row + id) : 0.0f;
  }
  // Weights at the end of 32 bits (and within that of 64): a sigmoid's under 2^-115, a softmax's of an exponent below
  // -48, whose rounding (2^-24 of it) would also be the larger part of the weight's error.
  const float least = r.softmax ? top - 48.0f : -80.0f;
  if (__any_sync(kFull, lane < k && l < least && l > least - 720.0f)) return false;
  float s = 0.0f;
  if (lane < k) s = r.softmax ? expf(l - top) * inv_norm : 1.0f / (1.0f + expf(-l));
  if (r.renormalize) {
    float sum = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (sum < 1e-30f) return false;                      // (the same in all lanes)
    s = s / sum;
  }
  weight = s * r.scale;
  return true;
}

template <int PER>
__device__ __forceinline__ void select_token(const float* __restrict__ row, const ScoreRule& r, int E, int k, int lane,
                                             int2* won, int& id, float& weight) {
  const bool done = E == 32 * PER && r.lpg * r.groups == 32 ? select_fast<PER, true>(row, r, E, k, lane, won, id, weight)
                                                            : select_fast<PER, false>(row, r, E, k, lane, won, id, weight);
  if (!done) select_exact<PER>(row, r, E, k, lane, id, weight);
}

// Exclusive prefix over E counts in shared memory, four experts a thread of the first 256: own counts in c, the
// prefix of the first returned.  A barrier inside; warp_tmp holds 8 ints.
__device__ __forceinline__ int scan_counts(const int* cnt, int* warp_tmp, int E, int (&c)[4]) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, e4 = 4 * threadIdx.x;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = e4 + i < E ? cnt[e4 + i] : 0;
    sum += c[i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31 && wid < 8) warp_tmp[wid] = inc;
  __syncthreads();
  int at = inc - sum;
#pragma unroll
  for (int w = 0; w < 7; ++w) at += w < wid ? warp_tmp[w] : 0;
  return at;
}
// From the counts of all rows (256 threads or more): run -> where the rows after the prefixes `pre` (of experts
// 4 threadIdx.x ..) go.  The last CTA writes the offsets and, if wanted, the counts and group lists.
__device__ __forceinline__ void start_places(int* run, const int (&pre)[4], bool last, int* tmp, int* tmp1, int* tmp2,
                                             int* warp_tmp, int E, const RouteBufs& b) {
  if (last && b.groups) {
    finish_counts(run, tmp, tmp1, tmp2, warp_tmp, E, b.group_rows, b);   // run = offsets
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * (int)threadIdx.x + i < E) run[4 * threadIdx.x + i] += pre[i];
  } else {
    int c[4], at = scan_counts(run, warp_tmp, E, c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * threadIdx.x + i;
      if (e < E) {
        run[e] = at + pre[i];
        if (last) b.offsets[e] = at;
      }
      at += c[i];
    }
    if (last && threadIdx.x == 255) b.offsets[E] = at;
  }
  __syncthreads();
}

// Stable placement of rows r0 .. r0 + n - 1 (n > 0, id_of(i) the expert of row r0 + i) from run[expert] on, by the
// first kPlaceWarps warps of a CTA, 32 rows each at a time: a row's place is its expert's running position plus
// the rows of that expert in the warps before (hist, zero on entry and exit) and in the lanes before it (a match
// over the warp).  Every thread of the CTA calls.
template <typename IdOf>
__device__ __forceinline__ void place_rows(int64_t r0, int64_t n, int* run, uint8_t (*hist)[kMaxE], const RouteBufs& b,
                                           IdOf id_of) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  for (int64_t i0 = 0; i0 < n; i0 += 32 * kPlaceWarps) {
    const int64_t i = i0 + 32 * wid + lane;
    const bool have = wid < kPlaceWarps && i < n;
    const int id = have ? id_of(i) : -1;
    const unsigned peers = __match_any_sync(kFull, id);
    const unsigned below = peers & ((1u << lane) - 1u);
    const bool first = have && below == 0u;
    if (first) hist[wid][id] = (uint8_t)__popc(peers);
    __syncthreads();
    if (have) {
      int pos = run[id] + __popc(below);
      for (int w = 0; w < wid; ++w) pos += hist[w][id];
      b.perm[pos] = (int32_t)(r0 + i);
      b.inv[r0 + i] = pos;
    }
    __syncthreads();
    if (first) {
      atomicAdd(&run[id], __popc(peers));
      hist[wid][id] = 0;
    }
    __syncthreads();
  }
}

// Up to kOneTokens tokens in one CTA: choice, counts, groups, placement.
template <int PER>
__global__ void __launch_bounds__(32 * kOneTokens) scored_one_kernel(const float* __restrict__ logits, int T, int E,
                                                                     int k, ScoreRule r, RouteBufs b) {
  __shared__ int cnt[kMaxE], tmp[kMaxE], tmp1[kMaxE], tmp2[kMaxE], warp_tmp[32];
  __shared__ int sids[32 * kOneTokens];
  __shared__ int2 won[kOneTokens][32];
  __shared__ __align__(4) uint8_t hist[kPlaceWarps][kMaxE];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int R = T * k;
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  if (R > 32)
    for (int i = threadIdx.x; i < kPlaceWarps * kMaxE / 4; i += blockDim.x) reinterpret_cast<int*>(hist)[i] = 0;
  __syncthreads();
  if (wid < T) {
    int id;
    float w;
    select_token<PER>(logits + (size_t)wid * E, r, E, k, lane, won[wid], id, w);
    if (lane < k) {
      b.ids[wid * k + lane] = id;
      b.w[wid * k + lane] = w;
      sids[wid * k + lane] = id;
      atomicAdd(&cnt[id], 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) b.counts[e] = cnt[e];
  const int none[4] = {0, 0, 0, 0};
  start_places(cnt, none, true, tmp, tmp1, tmp2, warp_tmp, E, b);
  const auto id_of = [&](int64_t i) { return sids[i]; };
  if (R > 32)
    place_rows(0, R, cnt, hist, b, id_of);
  else if (wid == 0)
    place32(0, R, lane, cnt, b, id_of);
}

// Step 1: the choice, a warp a token.  Up to 256 experts 64 registers (a few spilled), 32 warps an SM.
template <int PER>
__global__ void __launch_bounds__(32 * kChoiceWarps, PER <= 8 ? 4 : 2)
    scored_choice_kernel(const float* __restrict__ logits, int64_t T, int E, int k, ScoreRule r, RouteBufs b) {
  __shared__ int2 won[kChoiceWarps][32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + wid;
  launch_dependents();
  if (t >= T) return;
  int id;
  float w;
  select_token<PER>(logits + t * E, r, E, k, lane, won[wid], id, w);
  if (lane < k) {
    b.ids[t * k + lane] = id;
    b.w[t * k + lane] = w;
  }
}

// Step 2: a chunk's rows per expert, left in inv from the chunk's first row on.
__global__ void __launch_bounds__(32 * kPlaceWarps) scored_count_kernel(int64_t T, int E, int k, int chunk, RouteBufs b) {
  __shared__ int cnt[kMaxE];
  const int64_t t0 = (int64_t)blockIdx.x * chunk, t1 = blockIdx.x + 1 == gridDim.x ? T : t0 + chunk;
  const int64_t r0 = t0 * k, n = (t1 - t0) * k;
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  wait_dependency();
  launch_dependents();
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) atomicAdd(&cnt[b.ids[r0 + i]], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) b.inv[r0 + e] = cnt[e];
}

// Step 3: per expert the exclusive prefix over the chunks, in place, and its count.  A CTA takes 32
// experts, kScanSegs threads each a run of chunks: every load of a thread's run is under way at once.
__global__ void __launch_bounds__(32 * kScanSegs) scored_scan_kernel(int nchunks, int64_t stride, int E, RouteBufs b) {
  constexpr int kRun = kMaxChunks / kScanSegs;
  __shared__ int sums[kScanSegs][33];
  const int lane = threadIdx.x & 31, seg = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  const int per = (nchunks + kScanSegs - 1) / kScanSegs, c0 = seg * per;   // per <= kRun
  wait_dependency();
  launch_dependents();
  int v[kRun], sum = 0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    v[i] = i < per && c0 + i < nchunks && e < E ? b.inv[(c0 + i) * stride + e] : 0;
    sum += v[i];
  }
  sums[seg][lane] = sum;
  __syncthreads();
  // warp w scans expert w of the 32 over the segments
  int inc = sums[lane][seg];
  const int own = inc;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31 && blockIdx.x * 32 + seg < E) b.counts[blockIdx.x * 32 + seg] = inc;
  __syncthreads();
  sums[lane][seg] = inc - own;
  __syncthreads();
  int run = sums[seg][lane];
#pragma unroll
  for (int i = 0; i < kRun; ++i)
    if (i < per && c0 + i < nchunks && e < E) {
      b.inv[(c0 + i) * stride + e] = run;
      run += v[i];
    }
}

// Step 4: stable placement of the chunk's rows.  Every CTA scans the counts for the offsets; the last one
// writes the offsets and groups.
__global__ void __launch_bounds__(32 * kPlaceWarps) scored_place_kernel(int64_t T, int E, int k, int chunk,
                                                                        RouteBufs b) {
  __shared__ int run[kMaxE], tmp[kMaxE], tmp1[kMaxE], tmp2[kMaxE], warp_tmp[32];
  __shared__ __align__(4) uint8_t hist[kPlaceWarps][kMaxE];
  const bool last = blockIdx.x + 1 == gridDim.x;
  const int64_t t0 = (int64_t)blockIdx.x * chunk, t1 = last ? T : t0 + chunk;
  const int64_t r0 = t0 * k, n = (t1 - t0) * k;
  for (int i = threadIdx.x; i < kPlaceWarps * kMaxE / 4; i += blockDim.x) reinterpret_cast<int*>(hist)[i] = 0;
  wait_dependency();
  int pre[4];                                            // the chunk's prefixes
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * threadIdx.x + i;
    pre[i] = e < E ? b.inv[r0 + e] : 0;
  }
  for (int e = threadIdx.x; e < E; e += blockDim.x) run[e] = b.counts[e];
  __syncthreads();                                       // every count of this chunk is read
  start_places(run, pre, last, tmp, tmp1, tmp2, warp_tmp, E, b);
  place_rows(r0, n, run, hist, b, [&](int64_t i) { return b.ids[r0 + i]; });
}

// Steps 2 to 4 for few rows: every CTA counts all of the call's ids itself (those before its kFewPlace rows
// apart, which are its prefixes) and places its rows.
__global__ void __launch_bounds__(32 * kPlaceWarps) scored_count_place_kernel(int R, int E, RouteBufs b) {
  __shared__ int run[kMaxE], before[kMaxE], tmp[kMaxE], tmp1[kMaxE], tmp2[kMaxE], warp_tmp[32];
  __shared__ __align__(4) uint8_t hist[kPlaceWarps][kMaxE];
  const bool last = blockIdx.x + 1 == gridDim.x;
  const int r0 = blockIdx.x * kFewPlace, n = min(kFewPlace, R - r0);
  for (int e = threadIdx.x; e < E; e += blockDim.x) run[e] = before[e] = 0;
  for (int i = threadIdx.x; i < kPlaceWarps * kMaxE / 4; i += blockDim.x) reinterpret_cast<int*>(hist)[i] = 0;
  __syncthreads();
  wait_dependency();
  constexpr int kAhead = 8;
  for (int i0 = threadIdx.x; i0 < R; i0 += kAhead * 32 * kPlaceWarps) {
    int id[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * 32 * kPlaceWarps;
      id[j] = i < R ? b.ids[i] : -1;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (id[j] >= 0) atomicAdd(&(i0 + j * 32 * kPlaceWarps < r0 ? before : run)[id[j]], 1);
  }
  __syncthreads();
  int pre[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * threadIdx.x + i;
    pre[i] = e < E ? before[e] : 0;
    if (e < E) run[e] += pre[i];
    if (e < E && last) b.counts[e] = run[e];
  }
  __syncthreads();
  start_places(run, pre, last, tmp, tmp1, tmp2, warp_tmp, E, b);
  place_rows(r0, n, run, hist, b, [&](int64_t i) { return b.ids[r0 + i]; });
}

// A launch that may begin while the one before it ends (the kernel waits for its results itself).
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kern)(Params...), int grid, int block, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

template <int PER>
int launch_scored(const float* logits, int64_t T, int E, int k, const ScoreRule& r, const RouteBufs& b,
                  cudaStream_t s) {
  if (T <= kOneTokens) {
    scored_one_kernel<PER><<<1, 32 * kOneTokens, 0, s>>>(logits, (int)T, E, k, r, b);
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? 1 : -(int)err;
  }
  const bool few = T * k <= kFewRows;
  // A CTA's tokens: four, but eight from 513 to 1024 tokens before the counting placement.  Both sides in a graph, four /
  // eight (us), 256 experts, k = 8: 64 tokens 6.6 / 7.0, 512 8.0 / 8.5, 768 11.5 / 9.0, 1024 12.9 / 9.5, 1365 12.1 / 12.6,
  // 8192 19.8 / 20.5, 32768 47.5 / 49.0; 64 of softmax, k = 6: 768 9.6 / 8.1, 1024 10.2 / 8.3, 1365 11.3 / 11.3, 8192
  // 15.6 / 16.0; 512, k = 2: 768 9.6 / 9.9, 1024 10.7 / 10.0, 1365 12.3 / 13.9, 4096 21.1 / 23.3, 32768 77 / 82.
  const int warps = few && T > 512 && T <= 1024 ? kChoiceWarps : 4;
  scored_choice_kernel<PER><<<(unsigned)((T + warps - 1) / warps), 32 * warps, 0, s>>>(logits, T, E, k, r, b);
  if (few) {
    const int R = (int)(T * k);
    cudaError_t err =
        launch_after(scored_count_place_kernel, (R + kFewPlace - 1) / kFewPlace, 32 * kPlaceWarps, s, R, E, b);
    if (err == cudaSuccess) err = cudaGetLastError();
    return err == cudaSuccess ? 2 : -(int)err;
  }
  // A chunk's rows number at least E (its counts fit in its part of inv); the last chunk takes the
  // remainder, so none is shorter.
  const int64_t chunk = std::max<int64_t>({kChunkMin, (E + k - 1) / k, (T + kMaxChunks - 1) / kMaxChunks});
  const int nch = (int)std::max<int64_t>(1, T / chunk);
  cudaError_t err = launch_after(scored_count_kernel, nch, 32 * kPlaceWarps, s, T, E, k, (int)chunk, b);
  if (err == cudaSuccess) err = launch_after(scored_scan_kernel, (E + 31) / 32, 32 * kScanSegs, s, nch, chunk * k, E, b);
  if (err == cudaSuccess) err = launch_after(scored_place_kernel, nch, 32 * kPlaceWarps, s, T, E, k, (int)chunk, b);
  if (err == cudaSuccess) err = cudaGetLastError();
  return err == cudaSuccess ? 4 : -(int)err;
}

}  // namespace

// Experts a lane holds, 0 where the kernels do not take the shape.
int scored_per_lane(int E, int groups) {
  if (groups < 1 || groups > 32 || E % groups) return 0;
  int lpg = 32;
  while (lpg * groups > 32) lpg >>= 1;
  const int per = (E / groups + lpg - 1) / lpg;
  return per <= 64 ? per : 0;
}

int launch_route_scored(const float* logits, int64_t T, int E, int k, const ScoreRule& rule, const RouteBufs& b,
                        cudaStream_t s) {
  const int per = scored_per_lane(E, rule.groups);
  if (per == 0) return -(int)cudaErrorInvalidValue;
  ScoreRule r = rule;
  r.lpg = 32;
  while (r.lpg * r.groups > 32) r.lpg >>= 1;
  if (per <= 4) return launch_scored<4>(logits, T, E, k, r, b, s);
  if (per <= 8) return launch_scored<8>(logits, T, E, k, r, b, s);
  if (per <= 16) return launch_scored<16>(logits, T, E, k, r, b, s);
  if (per <= 32) return launch_scored<32>(logits, T, E, k, r, b, s);
  return launch_scored<64>(logits, T, E, k, r, b, s);
}

}  // namespace moe
