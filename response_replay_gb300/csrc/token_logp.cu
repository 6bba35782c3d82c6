// token_logp.cu -- log probabilities of given tokens, entropies and top alternatives of the
// vocabulary rows, and the gradient that an objective of these sends to the logits.
//
// For a row of logits z (V values), temperature tau and target y:
//   lse = log sum_v e^(z_v / tau),  logp = z_y / tau - lse,  p_v = e^(z_v / tau - lse),
//   H = -sum_v p_v log p_v = lse - sum_v p_v z_v / tau,
//   alternatives: the k largest z_v / tau - lse and their ids, equal ones by the lowest id.
// With upstream g (of logp), h (of H) and a_j (of alternative j), G = g + sum_j a_j:
//   dL/dz_v = (1 / tau) (g 1[v = y] + sum_j a_j 1[v = id_j] - p_v (G + h (log p_v + H))).
//
// Forward.  One pass over the row: every thread keeps a reference m, s = sum 2^t and
// e = sum 2^t t of t = (z - m) c (c = log2(e) / tau), so H = ln 2 (log2 s - e / s).  The
// alternatives ride along on maxima of the same registers: a row is cut into groups of 64 bytes;
// each group's maximum goes to shared memory, and a thread keeps the largest of its groups (ties
// to the lowest group, which holds the lower ids).  Behind the row the k-th largest of 32 or 64
// maxima over disjoint groups is a threshold: k logits reach it, so only groups whose maximum does
// can hold one of the k largest.  A warp reads those groups again (about 40 of 4,750 for k = 20)
// and orders the logits that pass.
// A row too long for the group maxima, or a call with few rows, is cut into parts whose results
// a second kernel merges.  Short rows go to a warp or a few each (logp_rows).
// Sums are in fp32: over 64 bytes, then over a thread's groups, then a tree; the last steps are in
// fp64.
#include <float.h>
#include <math.h>

#include "ls_chunks.h"
#include "ls_device.cuh"
#include "ls_internal.h"
#include "ls_umma.cuh"

namespace {

constexpr int kThreads = 384;  // consumers of the forward, a group of 64 bytes each a step
constexpr int kWarps = kThreads / 32;
constexpr int kGroupBytes = 64;
// Groups of a part with alternatives, whose maxima lie in shared memory: what 151,936 bf16 values take
// (4,750) and some more.  Longer rows are cut in two and merged: 4,096 rows of 200,064 take 315 us with
// 5 alternatives and 231 without, where 151,936 take 194 and 175; 7,168 groups would fit two CTAs an SM
// and have not been tried.
constexpr int kMaxGroups = 4864;
constexpr int kBwdThreads = 256, kBwdCtas = 5;  // of the backward, and blocks an SM
constexpr float kLargeSum = 2048.f;  // of 2^t t: t = 8, or many somewhat below
constexpr double kLn2d = 0.69314718055994530942;
constexpr double kLog2ed = 1.4426950408889634074;

using u64 = unsigned long long;

// An exponent of -inf is taken as one whose 2^t is 0 all the same, so that 2^t t is 0.  NaN
// stays NaN.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float floor_exp(float t) { return max_nan(t, -200.f); }

template <typename E>
struct Row;  // N: values of 16 bytes
template <>
struct Row<float> {
  static constexpr int N = 4;
  // the largest of 64 bytes (NaN only where all are)
  __device__ static float max_of(const uint4* u) {
    float m[4];
#pragma unroll
    for (int v = 0; v < 4; ++v)
      m[v] = fmaxf(fmax3(__uint_as_float(u[v].x), __uint_as_float(u[v].y), __uint_as_float(u[v].z)),
                   __uint_as_float(u[v].w));
    return fmaxf(fmax3(m[0], m[1], m[2]), m[3]);
  }
  // 16 bytes of values
  __device__ static void put(uint4* u, int i, float x) {
    reinterpret_cast<float*>(u)[i] = x;
  }
  __device__ static void unpack(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  __device__ static uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
  __device__ static float load(const float* p) { return *p; }
  __device__ static void store(float* p, float x) { *p = x; }
};
template <>
struct Row<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static float max_of(const uint4* u) {
    auto max2 = [](uint32_t x, uint32_t y) {  // of two pairs
      uint32_t r;
      asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
      return r;
    };
    uint32_t m = max2(max2(u[0].x, u[0].y), max2(u[0].z, u[0].w));
#pragma unroll
    for (int v = 1; v < 4; ++v) m = max2(m, max2(max2(u[v].x, u[v].y), max2(u[v].z, u[v].w)));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  __device__ static void put(uint4* u, int i, float x) {
    reinterpret_cast<__nv_bfloat16*>(u)[i] = __float2bfloat16_rn(x);  // of a bf16 number: exact
  }
  __device__ static void unpack(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float* x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
  }
  __device__ static float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
};

// Logits as whole numbers in their order (one zero; NaN: 0, behind all), and with their places
// as one number: larger logits first, equal ones by the lower place (the complement below).
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  if (x != x) return 0u;
  return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(u64 key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float((int32_t)o < 0 ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ u64 max64(u64 a, u64 b) { return a > b ? a : b; }

// A warp's 32 keys, largest in lane 0.
__device__ __forceinline__ u64 exchange(u64 x, int lane, int j, bool down) {
  const u64 y = __shfl_xor_sync(0xffffffffu, x, j);
  return ((lane & j) == 0) == down ? (x > y ? x : y) : (x > y ? y : x);
}
__device__ __forceinline__ u64 sort32(u64 x, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) x = exchange(x, lane, j, k == 32 || (lane & k) == 0);
  return x;
}
// The 32 largest of a sorted list and a sorted batch, sorted.
__device__ __forceinline__ u64 merge32(u64 list, u64 batch, int lane) {
  u64 x = max64(list, __shfl_sync(0xffffffffu, batch, 31 - lane));
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) x = exchange(x, lane, j, true);
  return x;
}

// A reference m (a logit, or a number between logits; none passes it by more than 2^8, or it is
// moved), s = sum 2^t, e = sum 2^t t with t = z c - r, r = m c rounded: one multiply-add an exponent.
// r is off by half a step of its size, the same in every t: where that is more than 2 (masks of
// -1e9, a temperature of 1e-6), sums would leave fp32's range, and t = (z - m) c.
struct Stat {
  float m, s, e;
};
__device__ __forceinline__ bool plain_ref(float r) { return fabsf(r) < 67108864.f; }  // 2^26
// t of one maximum under another: what moves sums from the one to the other.  Plain references
// stand for r, others for m c itself.
__device__ __forceinline__ float shift(float from, float to, float c) {
  const float a = from * c, b = to * c;
  if (plain_ref(a)) return plain_ref(b) ? a - b : -fmaf(to, c, -a);
  return plain_ref(b) ? fmaf(from, c, -b) : (from - to) * c;
}
__device__ __forceinline__ Stat move(Stat x, float m, float c) {
  if (x.m == -INFINITY || x.m == m) return x;  // no finite logit: nothing to move
  const float d = shift(x.m, m, c), f = fast_exp2(d);
  return {m, x.s * f, (x.e + x.s * floor_exp(d)) * f};
}
__device__ __forceinline__ Stat merge(Stat a, Stat b, float c) {
  const float m = fmaxf(a.m, b.m);
  a = move(a, m, c);
  b = move(b, m, c);
  return {m, a.s + b.s, a.e + b.e};
}
// Of one logit.
__device__ __forceinline__ Stat stat_of(float x, float c) {
  const float one = x == -INFINITY ? 0.f : 1.f + (x - x);  // NaN of NaN and of +inf
  const float r = x * c, t = plain_ref(r) ? fmaf(x, c, -r) : 0.f, s = one * fast_exp2(t);
  return {x != x ? -INFINITY : x, s, s * t};
}
// Over a warp's lanes, in every lane: the maximum first, so that each moves once.
__device__ __forceinline__ Stat warp_stat(Stat x, float c) {
  float m = x.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  x = move(x, m, c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x.s += __shfl_xor_sync(0xffffffffu, x.s, o);
    x.e += __shfl_xor_sync(0xffffffffu, x.e, o);
  }
  return {m, x.s, x.e};
}

// A thread's sums over its groups.
template <typename E>
struct Sums {
  static constexpr int H = Row<E>::N;
  float m, nr, c;                          // nr = -m c, or (not plain) infinity
  float2 s, e;
  __device__ __forceinline__ explicit Sums(float c_)
      : m(-INFINITY), nr(INFINITY), c(c_), s(make_float2(0.f, 0.f)), e(make_float2(0.f, 0.f)) {}

  // N vectors of 16 bytes.  The reference stays as it is as long as no logit passes it by far: of
  // 32 threads one would find a new maximum in most groups, and the warp would move its sums with
  // each.  Otherwise (the first group, sums of exponents about 8 and more, an exponent of -inf,
  // NaN, a reference that is not plain) the vectors are taken once more, carefully.  An exponent of the row's likeliest tokens
  // is off by half a step of its size, which that limit keeps to 2^-22: entropies of 1 are within
  // 2e-7 (relative, root mean square); with a limit of 2^100 they were off by 3e-6.  Rows that are
  // masked with -inf (or a bf16 row with the type's lowest value) take most vectors twice: 4,096 rows
  // of 151,936 bf16 values 175 us, with half of them masked 333, with all but 50 460; fp32 (1,531 rows
  // of 50,257) 51, 62 and 79.
  template <int N>
  __device__ __forceinline__ void add(const uint4* u) {
    // sums of these first: a short chain, then one addition
    float2 s1 = make_float2(0.f, 0.f), e1 = s1;
    const float2 b = make_float2(nr, nr), c2 = make_float2(c, c);
#pragma unroll
    for (int v = 0; v < N; ++v) {
      float x[H];
      Row<E>::unpack(u[v], x);
#pragma unroll
      for (int i = 0; i < H; i += 2) {
        const float2 t = __ffma2_rn(make_float2(x[i], x[i + 1]), c2, b);
        const float2 p = make_float2(fast_exp2(t.x), fast_exp2(t.y));
        s1 = __fadd2_rn(s1, p);
        e1 = __ffma2_rn(p, t, e1);
      }
    }
    e1 = __fadd2_rn(e, e1);
    if (e1.x + e1.y < kLargeSum) {
      s = __fadd2_rn(s, s1);
      e = e1;
    } else {
      carefully<N>(u);
    }
  }

  template <int N>
  __device__ __forceinline__ void carefully(const uint4* u) {
    float mx = -INFINITY;
#pragma unroll
    for (int v = 0; v < N; ++v) {
      float x[H];
      Row<E>::unpack(u[v], x);
#pragma unroll
      for (int i = 0; i < H; ++i) mx = fmaxf(mx, x[i]);
    }
    // many exponents below the limit that make a sum near it: the reference goes behind them
    if (e.x + e.y > kLargeSum / 2) mx = fmaxf(mx, m + log2f(s.x + s.y) / c);
    if (mx > m) {
      const Stat x = move(stat(), mx, c);
      s = make_float2(x.s, 0.f);
      e = make_float2(x.e, 0.f);
      m = mx;
      nr = plain_ref(m * c) ? -(m * c) : INFINITY;
    }
    const bool fine = plain_ref(nr);
#pragma unroll
    for (int v = 0; v < N; ++v) {
      float x[H];
      Row<E>::unpack(u[v], x);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float t = floor_exp(fine ? fmaf(x[i], c, nr) : m == -INFINITY ? x[i] : (x[i] - m) * c);
        const float p = fast_exp2(t);
        s.x += p;
        e.x = fmaf(p, t, e.x);
      }
    }
  }
  __device__ __forceinline__ Stat stat() const { return {m, s.x + s.y, e.x + e.y}; }
};

struct Out {
  float* logp;
  float* lse;
  float* entropy;
  float* top_logp;
  int32_t* top_ids;
};

struct FwdArgs {
  bool steal;       // more items than CTAs that fit: the rest of the grid is taken over
  const void* logits;
  int64_t T, ld;
  int32_t V, top, parts;
  const int32_t* targets;
  float c;          // log2(e) / tau, rounded
  double inv_tau;
  double c_off;     // by how much, relative
  Out out;
  float* part_stat;  // [T][parts][4]
  u64* part_top;     // [T][parts][32]
  uint32_t* err;
};

// The row's numbers from its statistics.  What is a difference of logits is counted from the
// reference, so that it is right whatever the logits' size: a log probability is
// (z - m) / tau - rest.  The rounding of c moves log2 of the sum by c_off times the mean exponent.
struct Norm {
  double m, rest;
  __device__ __forceinline__ float logp(float z, double inv_tau) const {
    return (float)(((double)z - m) * inv_tau - rest);
  }
};
__device__ __forceinline__ Norm finish_row(const FwdArgs& a, const Stat& x, int64_t row, bool has_y, float zy) {
  const float mean = x.e / x.s, r = x.m * a.c;
  const double log2s = (double)log2f(x.s);
  const float off = plain_ref(r) ? -fmaf(x.m, a.c, -r) : 0.f;  // r's rounding, exact
  const Norm n = {(double)x.m, kLn2d * (log2s + ((double)off - a.c_off * (double)mean))};
  const bool none = x.m == -INFINITY && x.s == 0.f;
  if (a.out.lse) a.out.lse[row] = none ? -INFINITY : (float)(n.m * a.inv_tau + n.rest);
  if (a.out.entropy) a.out.entropy[row] = (float)(kLn2d * (log2s - (double)mean));
  if (a.out.logp) a.out.logp[row] = has_y ? n.logp(zy, a.inv_tau) : NAN;
  return n;
}

// Rows whose target is -1 are padding: their outputs are zeros and ids -1.
__device__ __forceinline__ void padding_row(const FwdArgs& a, int64_t row, int lane) {
  if (lane == 0) {
    if (a.out.logp) a.out.logp[row] = 0.f;
    if (a.out.lse) a.out.lse[row] = 0.f;
    if (a.out.entropy) a.out.entropy[row] = 0.f;
  }
  if (lane < a.top) {
    a.out.top_logp[row * a.top + lane] = 0.f;
    a.out.top_ids[row * a.top + lane] = -1;
  }
}
template <typename E>
__device__ __forceinline__ bool target_logit(const FwdArgs& a, int64_t row, float* zy) {
  if (!a.targets) return false;
  const int32_t y = a.targets[row];
  if ((uint32_t)y >= (uint32_t)a.V) {
    ls_report(a.err, LS_DEVERR_CHECK);
    return false;
  }
  *zy = Row<E>::load(static_cast<const E*>(a.logits) + row * a.ld + y);
  return true;
}

// (n: lane 0's counts)
__device__ __forceinline__ void write_top(const FwdArgs& a, int64_t row, u64 key, Norm n, int lane) {
  n.m = __shfl_sync(0xffffffffu, n.m, 0);
  n.rest = __shfl_sync(0xffffffffu, n.rest, 0);
  if (lane >= a.top) return;
  a.out.top_logp[row * a.top + lane] = key ? n.logp(value_of(key), a.inv_tau) : NAN;
  a.out.top_ids[row * a.top + lane] = key ? (int32_t)~(uint32_t)key : -1;
}

// ---------------------------------------------------------------- forward
//
// A CTA an item (a part of a row), of which two fit an SM; a CTA that runs takes over others that
// have not begun (cluster launch control), so all end together whatever the SMs' shares of HBM were:
// dealt out beforehand they ended between 147 and 179 us (4,096 rows of 151,936 bf16 values; 182 us
// in all, now 175).  A producer warp streams an item's whole groups through a ring of 24 KB chunks
// by bulk copies, a group a consumer thread and chunk, and runs ahead into the next item while the
// consumers end one; a last warp takes the consumers' results and maxima, finds the candidates, reads
// those groups again and writes the row's outputs while the consumers are at the next item (with the
// consumers at the candidates 241 us for 5 alternatives and 271 for 20; now 201 and 202).  Groups that
// stick out of the row are read with plain loads.
constexpr int kChunkBytes = kThreads * kGroupBytes;
constexpr int kCtaThreads = kThreads + 64;
constexpr int kHand = kThreads + 32;  // the consumers and the last warp
template <bool kTop>
struct Cfg {
  static constexpr int kStages = kTop ? 3 : 4;
};
constexpr int kRanked = 128;  // logits that are put in order by counting
constexpr int kCand = 512;  // groups that reach the threshold, before the slow way is taken

constexpr int kFound = 32 * 16 + kRanked;

constexpr int kQueue = 4;  // items on their way from the producer to the other warps

struct FwdSmem {  // behind the ring; [2]: by parity of the item
  uint64_t full[6], empty[6], free[2], item_full[kQueue], item_empty[kQueue], taken;
  alignas(16) uint32_t taken_answer[4];
  int64_t item[kQueue];
  int32_t target[kQueue];
  int abort;
  float m[2][kWarps], s[2][kWarps], e[2][kWarps];
  uint32_t best[2][kThreads];  // the largest of a thread's groups (0: none), and which
  uint16_t bestg[2][kThreads];
  alignas(16) uint32_t tops[64];
  int topg[64];
  alignas(16) u64 found[kFound];  // logits that reach the threshold, on their way into the list
  uint16_t cand[kCand], owner[kThreads];
  alignas(16) uint16_t gmax[2][kMaxGroups];  // upper halves of the groups' maxima
};
static_assert(3 * kThreads * kGroupBytes + sizeof(FwdSmem) <= (228 * 1024 / 2 - 1024), "two CTAs an SM");

// Takes a CTA of the grid that has not begun; the answer (16 bytes) lands on `bar`.
__device__ __forceinline__ void take_cta(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   answer),
               "r"(bar)
               : "memory");
}
// Its index, or -1: none was left.
__device__ __forceinline__ int64_t taken_cta(uint32_t answer) {
  uint32_t x = 0, ok;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 r;\n ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %1, 1, 0, p;\n"
      " mov.u32 %0, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n}\n"
      : "=r"(x), "=r"(ok)
      : "r"(answer)
      : "memory");
  return ok ? (int64_t)x : -1;
}
// The consumers' results of an item.  These two have no limit of their own: a consumer warp that
// gives up hands over once more, for the item that it leaves, and the last warp looks for that
// before each take-over.  (As an mbarrier, with the limit of the other waits, 199 against 194 us for
// 4,096 rows of 151,936 bf16 values with 5 alternatives, 47 against 44 for 2,000 of 50,257.)
__device__ __forceinline__ void hand_over(int par) {
  if (par)
    asm volatile("bar.arrive 3, %0;" ::"n"(kHand) : "memory");
  else
    asm volatile("bar.arrive 2, %0;" ::"n"(kHand) : "memory");
}
__device__ __forceinline__ void take_over(int par) {
  if (par)
    asm volatile("bar.sync 3, %0;" ::"n"(kHand) : "memory");
  else
    asm volatile("bar.sync 2, %0;" ::"n"(kHand) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(mbar)
      : "memory");
}

// An item: groups [g0, g0 + ng) of a row, of which [in0, in1) lie wholly inside it.
template <typename E>
struct Item {
  static constexpr int G = kGroupBytes / sizeof(E);
  const E* zr;
  int64_t row;
  int part, lead, g0, ng, in0, in1;
  bool pad;
  static __device__ __forceinline__ int64_t row_of(const FwdArgs& a, int64_t item) {
    return a.parts == 1 ? item : item / a.parts;
  }
  // the row's target
  static __device__ __forceinline__ int32_t target(const FwdArgs& a, int64_t item) {
    return a.targets && item < a.T * a.parts ? __ldg(a.targets + row_of(a, item)) : 0;
  }
  __device__ __forceinline__ Item(const FwdArgs& a, int64_t item, int32_t y) {
    row = row_of(a, item);
    part = (int)(item - row * a.parts);
    pad = y == -1;
    zr = static_cast<const E*>(a.logits) + row * a.ld;
    lead = (int)((reinterpret_cast<uintptr_t>(zr) & (kGroupBytes - 1)) / sizeof(E));
    const int64_t all = ((int64_t)lead + a.V + G - 1) / G;
    g0 = a.parts == 1 ? 0 : (int)(all * part / a.parts);
    ng = (a.parts == 1 ? (int)all : (int)(all * (part + 1) / a.parts)) - g0;
    in0 = g0 == 0 && lead > 0 ? 1 : 0;
    in1 = ng - (part == a.parts - 1 && (lead + a.V) % G != 0 ? 1 : 0);
    if (in1 < in0) in1 = in0;  // one group that sticks out at both ends
  }
  __device__ __forceinline__ int chunks() const { return pad ? 0 : (in1 - in0 + kThreads - 1) / kThreads; }
  __device__ __forceinline__ const E* at(int g) const { return zr - lead + (int64_t)(g0 + g) * G; }
  // the place in the row of a group's first value (negative: it sticks out)
  __device__ __forceinline__ int place(int g) const { return (g0 + g) * G - lead; }
  // vectors [v0, v0 + n) of a group's 64 bytes; -inf outside the row
  template <int n>
  __device__ __forceinline__ void load(int V, int g, int v0, uint4* u) const {
    if (g >= in0 && g < in1) {
      const uint4* p = reinterpret_cast<const uint4*>(at(g)) + v0;
#pragma unroll
      for (int v = 0; v < n; ++v) u[v] = p[v];
    } else {
      const int64_t p = (int64_t)(g0 + g) * G - lead + v0 * Row<E>::N;
#pragma unroll
      for (int i = 0; i < n * Row<E>::N; ++i)
        Row<E>::put(u + i / Row<E>::N, i % Row<E>::N,
                    p + i >= 0 && p + i < V ? Row<E>::load(zr + p + i) : -INFINITY);
    }
  }
};

// Two upper halves of floats as whole numbers in their order.
__device__ __forceinline__ uint32_t order_halves(uint32_t x) {
  return x ^ (((x >> 15) & 0x00010001u) * 0xffffu | 0x80008000u);
}
// The threshold that the top-th largest of 64 maxima over disjoint groups makes, by a warp: the
// lowest maximum with fewer than top above it, and the last place among its equals.  (With 32
// maxima 32 alternatives let three times as many logits through.)
__device__ __forceinline__ void threshold(const uint32_t* tops, const int* topg, int top, int lane,
                                          uint32_t* floor_o, int* floor_g) {
  const uint32_t x = tops[lane], x2 = tops[lane + 32];
  const uint4* all = reinterpret_cast<const uint4*>(tops);
  int above = 0, above2 = 0;
#pragma unroll 4
  for (int k = 0; k < 16; ++k) {
    const uint4 y = all[k];
    above += (y.x > x) + (y.y > x) + (y.z > x) + (y.w > x);
    above2 += (y.x > x2) + (y.y > x2) + (y.z > x2) + (y.w > x2);
  }
  *floor_o = __reduce_min_sync(0xffffffffu, min(above < top ? x : 0xffffffffu, above2 < top ? x2 : 0xffffffffu));
  *floor_g = __reduce_max_sync(0xffffffffu, max(x == *floor_o ? topg[lane] : -1, x2 == *floor_o ? topg[lane + 32] : -1));
  if (*floor_o == 0) *floor_g = INT32_MAX;  // fewer groups than alternatives: all of them
}

// The 32 largest of up to 32 K keys, sorted, one a lane: each one's place is the number of larger
// ones.
template <int K>
__device__ __forceinline__ u64 rank_found(u64* buf, int found, int lane) {
  u64 mine[K];
  int rank[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    mine[i] = i * 32 + lane < found ? buf[i * 32 + lane] : 0ull;
    rank[i] = 0;
  }
  if (lane == 0) buf[found] = 0ull;
  __syncwarp();
#pragma unroll 4
  for (int j = 0; j < found; j += 2) {
    const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(buf + j);
#pragma unroll
    for (int i = 0; i < K; ++i) rank[i] += (y.x > mine[i]) + (y.y > mine[i]);
  }
  __syncwarp();
  buf[lane] = 0ull;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < K; ++i)
    if (mine[i] != 0 && rank[i] < 32) buf[rank[i]] = mine[i];
  __syncwarp();
  return buf[lane];
}
// The 32 largest of a list and `found` more, sorted, one a lane.  (The list is empty in every lane
// or in none.)
__device__ __forceinline__ u64 order_found(u64* buf, int found, u64 list, int lane) {
  if (found > kRanked || list != 0) {
    for (int i = 0; i < found; i += 32)
      list = merge32(list, sort32(i + lane < found ? buf[i + lane] : 0ull, lane), lane);
    return list;
  }
  return found <= 32 ? rank_found<1>(buf, found, lane)
       : found <= 64 ? rank_found<2>(buf, found, lane) : rank_found<kRanked / 32>(buf, found, lane);
}
__device__ __forceinline__ int prefix_sum(int x, int lane, int* total) {  // of the lanes before
  int t = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += y;
  }
  *total = __shfl_sync(0xffffffffu, t, 31);
  return t - x;
}

// The 32 largest logits of an item, sorted, one a lane, by one warp: of the groups that reach the
// threshold, or (more of them than the list holds: rows whose largest logits all lie with the
// same threads) of all groups.
template <typename E>
__device__ u64 pick(FwdSmem& sm, const Item<E>& it, const FwdArgs& a, int par, int lane) {
  constexpr int G = Item<E>::G;
  // the two largest of every lane's threads
  uint32_t o[kWarps], o1 = 0, o2 = 0;
  int i1 = -1, i2 = -1;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) o[i] = sm.best[par][lane + 32 * i];
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (o[i] > o1) {
      o2 = o1;
      i2 = i1;
      o1 = o[i];
      i1 = i;
    } else if (o[i] > o2) {
      o2 = o[i];
      i2 = i;
    }
  }
  sm.tops[2 * lane] = o1;
  sm.topg[2 * lane] = i1 < 0 ? -1 : sm.bestg[par][lane + 32 * i1];
  sm.tops[2 * lane + 1] = o2;
  sm.topg[2 * lane + 1] = i2 < 0 ? -1 : sm.bestg[par][lane + 32 * i2];
  __syncwarp();
  uint32_t floor_o;
  int floor_g;
  threshold(sm.tops, sm.topg, a.top, lane, &floor_o, &floor_g);
  // the threads that have a group that reaches it, and their groups (both zeros are one)
  int threads = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const uint32_t mask = __ballot_sync(0xffffffffu, o[i] >= floor_o);
    if (o[i] >= floor_o) sm.owner[threads + __popc(mask & ((1u << lane) - 1))] = (uint16_t)(lane + 32 * i);
    threads += __popc(mask);
  }
  __syncwarp();
  const uint32_t floor16 = (floor_o >> 16) == 0x8000u ? 0x7fffu : floor_o >> 16;
  auto reaches = [&](int g) { return (order_halves(sm.gmax[par][g]) & 0xffffu) >= floor16; };
  constexpr int kSteps = (kMaxGroups + kThreads - 1) / kThreads;
  static_assert(kSteps <= 30, "a bit a group");
  int cands = 0;
  for (int t0 = 0; t0 < threads; t0 += 32) {
    const bool has = t0 + lane < threads;
    const int first = it.in0 + (has ? sm.owner[t0 + lane] : 0);
    uint32_t mask = 0;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
      if (has && first + k * kThreads < it.in1 && reaches(first + k * kThreads)) mask |= 1u << k;
    // the groups that stick out of the row
    if (t0 == 0 && lane == 0 && it.in0 > 0 && reaches(0)) mask |= 1u << 30;
    if (t0 == 0 && lane == 0 && it.in1 < it.ng && reaches(it.ng - 1)) mask |= 1u << 31;
    int total, at = cands + prefix_sum(__popc(mask), lane, &total);
    for (; mask; mask &= mask - 1, ++at) {
      const int k = __ffs(mask) - 1;
      if (at < kCand) sm.cand[at] = (uint16_t)(k == 30 ? 0 : k == 31 ? it.ng - 1 : first + k * kThreads);
    }
    cands += total;
  }
  __syncwarp();
  if (cands <= kCand) {
    const float floor = floor_o ? value_of((u64)floor_o << 32) : -INFINITY;
    int found = 0;
    for (int j0 = 0; j0 < cands && found <= kRanked; j0 += 32) {  // a group a lane
      const int g = j0 + lane < cands ? sm.cand[j0 + lane] : -1;
      uint32_t mask = 0;
      uint4 u[4];
      int place = 0;
      if (g >= 0) {
        place = it.place(g);
        it.template load<4>(a.V, g, 0, u);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float x[Row<E>::N];
          Row<E>::unpack(u[v], x);
#pragma unroll
          for (int i = 0; i < Row<E>::N; ++i)
            if (x[i] > floor || (x[i] == floor && g <= floor_g)) mask |= 1u << (v * Row<E>::N + i);
        }
        // what lies in the row
        if (place < 0) mask &= ~0u << -place;
        if (a.V - place < G) mask &= (1u << (a.V - place)) - 1;
      }
      int total, at = found + prefix_sum(__popc(mask), lane, &total);
      if (found + total <= kRanked) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float x[Row<E>::N];
          Row<E>::unpack(u[v], x);
#pragma unroll
          for (int i = 0; i < Row<E>::N; ++i) {
            const int b = v * Row<E>::N + i;
            if (mask & (1u << b)) sm.found[at++] = (u64)order_of(x[i]) << 32 | (uint32_t)~(uint32_t)(place + b);
          }
        }
      }
      found += total;
    }
    __syncwarp();
    if (found <= kRanked) {
      const u64 list = order_found(sm.found, found, 0, lane);
      __syncwarp();
      return list;
    }
  }
  // ---- more groups or logits than that: a value a lane and round, the list kept in order
  constexpr int kHalf = G / 2;
  const bool all = cands > kCand;
  const int n = all ? it.ng : cands;
  u64 kth = 0, list = 0;
  int found = 0;
  for (int j0 = 0; j0 < n; j0 += 16) {  // half a group a lane
    const int j = j0 + (lane >> 1), g = all ? j : j < n ? sm.cand[j] : 0;
    float x[kHalf];
    const int place = it.place(g) + (lane & 1) * kHalf;
    if (j < n) {
      uint4 u[2];
      it.template load<2>(a.V, g, 2 * (lane & 1), u);
      Row<E>::unpack(u[0], x);
      Row<E>::unpack(u[1], x + kHalf / 2);
    } else {
#pragma unroll
      for (int i = 0; i < kHalf; ++i) x[i] = NAN;
    }
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      const uint32_t ox = order_of(x[i]);
      bool in = ox > floor_o || (ox == floor_o && ox != 0 && g <= floor_g);
      const u64 key = (u64)ox << 32 | (uint32_t)~(uint32_t)(place + i);
      in = in && key > kth && place + i >= 0 && place + i < a.V;
      const uint32_t mask = __ballot_sync(0xffffffffu, in);
      if (mask == 0) continue;
      if (in) sm.found[found + __popc(mask & ((1u << lane) - 1))] = key;
      found += __popc(mask);
    }
    __syncwarp();
    if (found > kRanked) {  // more than are put in order by counting
      while (found >= 32) {
        found -= 32;
        list = merge32(list, sort32(sm.found[found + lane], lane), lane);
      }
      kth = __shfl_sync(0xffffffffu, list, a.top - 1);
      __syncwarp();
    }
  }
  list = order_found(sm.found, found, list, lane);
  __syncwarp();
  return list;
}

template <typename E, bool kTop>
__global__ void __launch_bounds__(kCtaThreads, 2) logp_fwd(const FwdArgs a) {
  using R = Row<E>;
  constexpr int kStages = Cfg<kTop>::kStages;
  extern __shared__ __align__(1024) uint8_t ring[];
  FwdSmem& sm = *reinterpret_cast<FwdSmem*>(ring + kStages * kChunkBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t full0 = smem_u32(sm.full), empty0 = smem_u32(sm.empty), ring0 = smem_u32(ring);
  const uint32_t free0 = smem_u32(sm.free), item_full0 = smem_u32(sm.item_full);
  const uint32_t item_empty0 = smem_u32(sm.item_empty);
  volatile int* abort = &sm.abort;
  // a wait that gives up records the error and stops every later wait of the CTA
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (umma::mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (umma::mbar_wait(bar, parity)) return true;
    ls_report(a.err, LS_DEVERR_TIMEOUT);
    *abort = 1;
    return false;
  };
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      umma::mbar_init(full0 + 8 * s, 1);
      umma::mbar_init(empty0 + 8 * s, kWarps);
    }
    umma::mbar_init(free0, 1);
    umma::mbar_init(free0 + 8, 1);
    for (int s = 0; s < kQueue; ++s) {
      umma::mbar_init(item_full0 + 8 * s, 1);
      umma::mbar_init(item_empty0 + 8 * s, kWarps + 1);
    }
    umma::mbar_init(smem_u32(&sm.taken), 1);
    sm.abort = 0;
    umma::fence_barrier_init();
  }
  __syncthreads();
  // the merge may be launched: its blocks wait for this grid before they read from it
  if (a.parts > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  umma::RingPos<kStages> rp;
  if (warp == kWarps) {
    // ---- producer
    if (lane == 0) {
      int issued = 0;
      umma::RingPos<kQueue> qp;
      auto push = [&](int64_t item, int32_t y) {
        if (!wait(item_empty0 + 8 * qp.stage, qp.phase ^ 1u)) return;
        sm.item[qp.stage] = item;
        sm.target[qp.stage] = y;
        umma::mbar_arrive(item_full0 + 8 * qp.stage);
        qp.advance();
      };
      const uint32_t answer = smem_u32(sm.taken_answer), taken = smem_u32(&sm.taken);
      uint32_t answers = 0;
      bool asked = false;
      for (int64_t item = blockIdx.x; item >= 0 && !*abort;) {
        if (a.steal) {  // the next item, while this one is streamed
          umma::mbar_expect_tx(taken, 16);
          take_cta(answer, taken);
          asked = true;
        }
        const int32_t y = Item<E>::target(a, item);
        push(item, y);
        const Item<E> it(a, item, y);
        const int n = it.chunks();
        const uint8_t* src = reinterpret_cast<const uint8_t*>(it.at(it.in0));
        for (int k = 0; k < n; ++k) {
          const uint32_t bytes = ls_chunk_bytes<kGroupBytes, kThreads>(it.in1 - it.in0, k);
          if (!wait(empty0 + 8 * rp.stage, rp.phase ^ 1u)) break;
          umma::mbar_expect_tx(full0 + 8 * rp.stage, bytes);
          bulk_load(ring0 + rp.stage * kChunkBytes, src + (int64_t)k * kChunkBytes, bytes,
                    full0 + 8 * rp.stage);
          ++issued;
          rp.advance();
        }
        item = -1;
        if (asked && wait(taken, answers & 1)) {
          ++answers;
          asked = false;
          item = taken_cta(answer);
          umma::fence_proxy_async_smem();  // read before the next answer is written
        }
      }
      push(-1, 0);
      if (asked) umma::mbar_wait(taken, answers & 1);
      // no copy may still be landing when the CTA exits
      for (int s = 0; s < kStages && s < issued; ++s) {
        rp.stage = rp.stage == 0 ? kStages - 1 : rp.stage - 1;
        if (rp.stage == kStages - 1) rp.phase ^= 1u;
        umma::mbar_wait(full0 + 8 * rp.stage, rp.phase);
      }
    }
    return;
  }

  int q = 0;
  umma::RingPos<kQueue> qp;
  int64_t item = 0;
  int32_t y = 0;
  auto next = [&]() {  // the CTA's next item, by a warp, whose lanes give up together
    if (!__all_sync(0xffffffffu, wait(item_full0 + 8 * qp.stage, qp.phase))) return false;
    item = sm.item[qp.stage];
    y = sm.target[qp.stage];
    __syncwarp();
    if (lane == 0) umma::mbar_arrive(item_empty0 + 8 * qp.stage);
    qp.advance();
    return item >= 0;
  };
  if (warp == kWarps + 1) {
    // ---- outputs
    while (next()) {
      const Item<E> it(a, item, y);
      if (it.pad) {
        if (it.part == 0) padding_row(a, it.row, lane);
        continue;
      }
      float zy = 0.f;
      bool has_y = false;
      if (lane == 0 && a.parts == 1) has_y = target_logit<E>(a, it.row, &zy);
      const int par = q & 1;
      ++q;
      if (__any_sync(0xffffffffu, *abort)) break;
      take_over(par);
      Stat st = {-INFINITY, 0.f, 0.f};
      if (lane < kWarps) st = Stat{sm.m[par][lane], sm.s[par][lane], sm.e[par][lane]};
      st = warp_stat(st, a.c);
      u64 list = 0;
      if (kTop) {
        list = pick<E>(sm, it, a, par, lane);
      }
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(free0 + 8 * par);
      if (a.parts > 1) {
        const int64_t at = it.row * a.parts + it.part;
        if (lane == 0) *reinterpret_cast<float4*>(a.part_stat + 4 * at) = make_float4(st.m, st.s, st.e, 0.f);
        if (kTop) a.part_top[at * 32 + lane] = list;
      } else {
        Norm norm{};
        if (lane == 0) norm = finish_row(a, st, it.row, has_y, zy);
        if (kTop) write_top(a, it.row, list, norm, lane);
      }
    }
    return;
  }

  // ---- consumers
  const float c = a.c;
  const int mine = tid * kGroupBytes + ((tid >> 1) & 3) * 16;  // of a chunk
  while (next()) {
    const Item<E> it(a, item, y);
    if (it.pad) continue;
    Sums<E> sums(c);
    // buffers that the last warp is done with
    const int par = q & 1;
    if (q >= 2) wait(free0 + 8 * par, ((q >> 1) - 1) & 1);
    ++q;
    float bestv = NAN;  // the largest of this thread's groups (the first of its equals), which
    int bestg = -1;
    uint16_t* gmax = sm.gmax[par];
    auto best = [&](int g, float mx) {
      gmax[g] = (uint16_t)(__float_as_uint(mx) >> 16);
      if (!(mx <= bestv)) {
        bestv = mx;
        bestg = g;
      }
    };
    // a group that sticks out of the row: the first and the last warp take theirs, a value a lane
    const bool sticks = (warp == 0 && it.in0 > 0) || (warp == kWarps - 1 && it.in1 < it.ng);
    const int edge_g = warp == 0 ? 0 : it.ng - 1, edge_at = it.place(edge_g) + lane;
    const bool has_edge = sticks && lane < Item<E>::G && edge_at >= 0 && edge_at < a.V;
    float edge = NAN;
    if (has_edge) edge = R::load(it.zr + edge_at);
    // a thread's 64 bytes of every chunk, in an order that keeps eight threads' loads apart; the
    // chunk is released as soon as they are in registers
    const int n = it.chunks();
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      uint4 u[4];
      const int g = it.in0 + k * kThreads + tid;
      const bool has = wait(full0 + 8 * rp.stage, rp.phase) && g < it.in1;
      const uint8_t* chunk = ring + rp.stage * kChunkBytes;
#pragma unroll
      for (int v = 0; v < 4; ++v) u[v] = *reinterpret_cast<const uint4*>(chunk + (mine ^ (16 * v)));
      __syncwarp();
      if (lane == 0) umma::mbar_arrive(empty0 + 8 * rp.stage);
      rp.advance();
      if (has) {  // (the maximum first: behind the sums it costs registers, 227 against 201 us)
        if (kTop) best(g, R::max_of(u));
        sums.template add<4>(u);
      }
    }
    // ---- the item's results
    Stat st = sums.stat();
    if (sticks) {
      if (has_edge) st = merge(st, stat_of(edge, c), c);
      if (kTop) {
        const uint32_t o = __reduce_max_sync(0xffffffffu, has_edge ? order_of(edge) : 0u);
        const float mx = o ? value_of((u64)o << 32) : NAN;
        if (lane == 0 && mx == bestv && edge_g < bestg) bestg = edge_g;
        if (lane == 0) best(edge_g, mx);
      }
    }
    st = warp_stat(st, c);
    if (lane == 0) {
      sm.m[par][warp] = st.m;
      sm.s[par][warp] = st.s;
      sm.e[par][warp] = st.e;
    }
    if (kTop) {
      sm.best[par][tid] = bestg < 0 ? 0u : order_of(bestv);
      sm.bestg[par][tid] = (uint16_t)bestg;
    }
    hand_over(par);
  }
  if (__any_sync(0xffffffffu, *abort)) hand_over(q & 1);
}

// ---------------------------------------------------------------- forward, many rows
//
// With many rows a streaming CTA a row would spend its time between rows: its results, threshold
// and candidates take as long as 100 KB of logits.  Here W warps take a row, 8 / W rows a CTA, and
// the other rows on the SM cover that time.  A group is a vector of 16 bytes (the values in front of
// the row's first whole vector are group 0, those behind its last one the last group); the two
// largest of every lane's groups (of every lane's, where several warps share a row) make the
// threshold, and the groups that reach it are read again.
constexpr int kRowsThreads = 256;
constexpr int kRowsWarps = kRowsThreads / 32;
constexpr int kRowsCand = 256;                  // groups that reach the threshold
constexpr int kRowsFound = 32 * 8 + kRanked;    // values that are found before they are ordered

struct RowSmem {
  Stat red[kRowsWarps];
  int cands;
  alignas(16) uint32_t tops[64];
  int topg[64];
  alignas(16) u64 found[kRowsFound];
  uint16_t cand[kRowsCand];
};

template <int W>
__device__ __forceinline__ void row_sync(int group) {
  if (W == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * W) : "memory");
}

// A row as vectors of 16 bytes.
template <typename E>
struct Vecs {
  static constexpr int N = Row<E>::N;
  const E* zr;
  int V, head, nvec, tail;  // values in front, whole vectors, values behind
  __device__ __forceinline__ Vecs(const E* z, int V_) : zr(z), V(V_) {
    const int in = (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(E));
    head = min(in ? N - in : 0, V);
    nvec = (V - head) / N;
    tail = V - head - nvec * N;
  }
  __device__ __forceinline__ const uint4* vec(int i) const { return reinterpret_cast<const uint4*>(zr + head) + i; }
  __device__ __forceinline__ int groups() const { return nvec + 2; }
  // values of group g and the place of the first; what is not in the row is NaN
  __device__ __forceinline__ int values(int g, float* x) const {
    if (g > 0 && g <= nvec) {
      Row<E>::unpack(*vec(g - 1), x);
      return head + (g - 1) * N;
    }
    const int at = g == 0 ? 0 : head + nvec * N, n = g == 0 ? head : tail;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < n ? Row<E>::load(zr + at + i) : NAN;
    return at;
  }
};

template <typename E>
__device__ __forceinline__ float vec_max(const uint4& u);
template <>
__device__ __forceinline__ float vec_max<float>(const uint4& u) {
  return fmaxf(fmax3(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z)), __uint_as_float(u.w));
}
template <>
__device__ __forceinline__ float vec_max<__nv_bfloat16>(const uint4& u) {
  auto max2 = [](uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
  };
  const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

template <typename E, bool kTop, int W>
__global__ void __launch_bounds__(kRowsThreads, 4) logp_rows(const FwdArgs a, int cap) {
  using R = Row<E>;
  extern __shared__ __align__(16) uint8_t rows_smem[];
  const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) / W, wl = (threadIdx.x >> 5) % W;
  const int l = wl * 32 + lane;
  constexpr int L = 32 * W;
  RowSmem& sm = reinterpret_cast<RowSmem*>(rows_smem)[group];
  // the upper halves of the groups' maxima
  uint16_t* gmax = reinterpret_cast<uint16_t*>(rows_smem + (kRowsWarps / W) * sizeof(RowSmem)) + group * cap;
  const int64_t row = (int64_t)blockIdx.x * (kRowsWarps / W) + group;
  if (row >= a.T) return;  // (a row's warps leave together)
  if (a.targets && __ldg(a.targets + row) == -1) {
    if (wl == 0) padding_row(a, row, lane);
    return;
  }
  const Vecs<E> v(static_cast<const E*>(a.logits) + row * a.ld, a.V);
  float zy = 0.f;
  bool has_y = false;
  if (l == 0) has_y = target_logit<E>(a, row, &zy);
  if (kTop && l == 0) sm.cands = 0;

  Sums<E> sums(a.c);
  float bestv = NAN, secondv = NAN;  // the largest of this lane's groups, the next
  int bestg = -1, secondg = -1;
  auto largest = [&](int g, float mx) {
    if (!(mx <= bestv)) {
      if (W == 1) {
        secondv = bestv;
        secondg = bestg;
      }
      bestv = mx;
      bestg = g;
    } else if (W == 1 && !(mx <= secondv)) {
      secondv = mx;
      secondg = g;
    }
  };
  auto take = [&](int g, float mx) {
    gmax[g] = (uint16_t)(__float_as_uint(mx) >> 16);
    largest(g, mx);
  };
  // one value outside the vectors a lane: the head's, then the tail's
  float edge = NAN;
  const bool in_head = l < v.head, has_edge = l < v.head + v.tail;
  if (has_edge) edge = R::load(v.zr + (in_head ? l : v.nvec * Vecs<E>::N + l));
  if (kTop) {  // (their maxima: the first lanes are one warp's)
    if (wl == 0) {
      const uint32_t o = has_edge ? order_of(edge) : 0u;
      const uint32_t oh = __reduce_max_sync(0xffffffffu, in_head ? o : 0u);
      const uint32_t ot = __reduce_max_sync(0xffffffffu, in_head ? 0u : o);
      if (lane == 0) {  // (a negative NaN where there are none: below every threshold)
        gmax[0] = oh ? (uint16_t)(__float_as_uint(value_of((u64)oh << 32)) >> 16) : 0xffffu;
        gmax[v.nvec + 1] = ot ? (uint16_t)(__float_as_uint(value_of((u64)ot << 32)) >> 16) : 0xffffu;
      }
      if (in_head && o) largest(0, edge);
    }
  }
  int i = l;
#pragma unroll 1
  for (; i + 3 * L < v.nvec; i += 4 * L) {
    uint4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = __ldg(v.vec(i + k * L));
    if (kTop) {  // (before the sums, as above)
#pragma unroll
      for (int k = 0; k < 4; ++k) take(i + k * L + 1, vec_max<E>(u[k]));
    }
    sums.template add<4>(u);
  }
#pragma unroll 1
  for (; i < v.nvec; i += L) {
    const uint4 u = __ldg(v.vec(i));
    if (kTop) take(i + 1, vec_max<E>(u));
    sums.template add<1>(&u);
  }
  if (kTop && has_edge && !in_head && edge == edge) largest(v.nvec + 1, edge);
  const uint32_t best = bestg < 0 ? 0u : order_of(bestv), second = secondg < 0 ? 0u : order_of(secondv);
  Stat st = sums.stat();
  if (has_edge) st = merge(st, stat_of(edge, a.c), a.c);
  st = warp_stat(st, a.c);
  if (W > 1 && lane == 0) sm.red[wl] = st;

  uint32_t floor_o = 0;
  int floor_g = INT32_MAX;
  if (kTop) {
    if (W <= 2) {
      const int at = W == 1 ? 2 * lane : l;
      sm.tops[at] = best;
      sm.topg[at] = bestg;
      if (W == 1) {
        sm.tops[at + 1] = second;
        sm.topg[at + 1] = secondg;
      }
    } else {  // the largest 64 / W of every warp's lanes
      uint32_t o = best;
      for (int k = wl; k < 64; k += W) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, o);
        const uint32_t at = __reduce_min_sync(0xffffffffu, o == top ? (uint32_t)bestg : 0xffffffffu);
        if (lane == 0) {
          sm.tops[k] = top;
          sm.topg[k] = top ? (int)at : -1;
        }
        if (o == top && (uint32_t)bestg == at) o = 0u;
      }
    }
    row_sync<W>(group);
    threshold(sm.tops, sm.topg, a.top, lane, &floor_o, &floor_g);
    const uint32_t floor16 = (floor_o >> 16) == 0x8000u ? 0x7fffu : floor_o >> 16;  // (both zeros are one)
    const int n = v.groups();
    for (int g0 = l * 8; g0 < n; g0 += L * 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(gmax + g0);
      const uint32_t ws[4] = {order_halves(w.x), order_halves(w.y), order_halves(w.z), order_halves(w.w)};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t o = k & 1 ? ws[k >> 1] >> 16 : ws[k >> 1] & 0xffffu;
        if (o >= floor16 && g0 + k < n) {
          const int at = atomicAdd(&sm.cands, 1);
          if (at < kRowsCand) sm.cand[at] = (uint16_t)(g0 + k);
        }
      }
    }
  }
  if (W > 1 || kTop) row_sync<W>(group);
  if (wl != 0) return;
  if (W > 1) st = warp_stat(lane < W ? sm.red[lane] : Stat{-INFINITY, 0.f, 0.f}, a.c);
  Norm norm{};
  if (lane == 0) norm = finish_row(a, st, row, has_y, zy);
  if (!kTop) return;

  // ---- the candidates' values, or (more of them than the list holds) all values
  const bool every = sm.cands > kRowsCand;
  const int n = every ? v.groups() : sm.cands;
  u64 kth = 0, list = 0;
  int found = 0;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    float x[Vecs<E>::N];
    int place = 0;
    const int g = j < n ? (every ? j : sm.cand[j]) : -1;
    if (g >= 0) {
      place = v.values(g, x);
    } else {
#pragma unroll
      for (int k = 0; k < Vecs<E>::N; ++k) x[k] = NAN;
    }
#pragma unroll
    for (int k = 0; k < Vecs<E>::N; ++k) {
      const uint32_t o = order_of(x[k]);
      const u64 key = (u64)o << 32 | (uint32_t)~(uint32_t)(place + k);
      const bool in = o != 0 && (o > floor_o || (o == floor_o && g <= floor_g)) && key > kth;
      const uint32_t mask = __ballot_sync(0xffffffffu, in);
      if (mask == 0) continue;
      if (in) sm.found[found + __popc(mask & ((1u << lane) - 1))] = key;
      found += __popc(mask);
    }
    __syncwarp();
    if (found >= kRanked) {  // as many as are put in order by counting
      while (found >= 32) {
        found -= 32;
        list = merge32(list, sort32(sm.found[found + lane], lane), lane);
      }
      kth = __shfl_sync(0xffffffffu, list, a.top - 1);
      __syncwarp();
    }
  }
  write_top(a, row, order_found(sm.found, found, list, lane), norm, lane);
}

// Rows that were cut into parts: a block a row, its warps take the parts by turns and their
// results meet in pairs.
constexpr int kMergeWarps = 8;
template <typename E, bool kTop>
__global__ void __launch_bounds__(kMergeWarps * 32) logp_merge(const FwdArgs a) {
  __shared__ Stat red[kMergeWarps];
  __shared__ u64 lists[kMergeWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  float zy = 0.f;
  bool has_y = false;
  if (threadIdx.x == 0 && !(a.targets && a.targets[row] == -1)) has_y = target_logit<E>(a, row, &zy);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.targets && a.targets[row] == -1) return;  // written by the row's first part
  Stat st = {-INFINITY, 0.f, 0.f};
  u64 list = 0;
  for (int p0 = warp; p0 < a.parts; p0 += 32 * kMergeWarps) {  // a lane a part
    const int p = p0 + lane * kMergeWarps;
    Stat x = {-INFINITY, 0.f, 0.f};
    if (p < a.parts) {
      const float4 f = __ldcg(reinterpret_cast<const float4*>(a.part_stat + 4 * (row * a.parts + p)));
      x = Stat{f.x, f.y, f.z};
    }
    st = merge(st, warp_stat(x, a.c), a.c);
  }
  if (kTop) {
    constexpr int kBatch = 4;  // lists that are loaded together
    for (int p0 = warp; p0 < a.parts; p0 += kBatch * kMergeWarps) {
      u64 x[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int p = p0 + b * kMergeWarps;
        x[b] = p < a.parts ? __ldcg(a.part_top + (row * a.parts + p) * 32 + lane) : 0ull;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (p0 + b * kMergeWarps < a.parts) list = merge32(list, x[b], lane);
    }
  }
  if (lane == 0) red[warp] = st;
#pragma unroll
  for (int half = kMergeWarps / 2; half > 0; half >>= 1) {
    if (kTop) lists[warp][lane] = list;
    __syncthreads();
    if (kTop && warp < half) list = merge32(list, lists[warp + half][lane], lane);
    __syncthreads();
  }
  if (warp != 0) return;
  st = warp_stat(lane < kMergeWarps ? red[lane] : Stat{-INFINITY, 0.f, 0.f}, a.c);
  Norm norm{};
  if (lane == 0) norm = finish_row(a, st, row, has_y, zy);
  if (kTop) write_top(a, row, list, norm, lane);
}

// ---------------------------------------------------------------- backward
struct BwdArgs {
  const void* logits;
  void* dlogits;
  int64_t T, ld, dld;
  int32_t V, top, parts;
  const int32_t* targets;
  const int32_t* top_ids;
  const float* lse;
  const float* entropy;
  const float* d_logp;
  const float* d_entropy;
  const float* d_top;
  float inv_hi, inv_lo;  // 1 / tau = inv_hi + inv_lo
  uint32_t* err;
};

// The row's gradient at one logit: p (a + b u) / tau of u = log p, a and b with their signs.
template <typename E>
struct RowGrad {
  float lse, a, b, hi, lo;
  __device__ __forceinline__ float2 at(float2 z) const {
    // u = z / tau - lse, rounded once.  The rounding of 1 / tau shows in fp32 gradients only
    // (20 half steps of it at a logit of 20), which take its rest; with it an infinite logit
    // has to be a finite one (the lowest: lse may be as low).
    if (sizeof(E) == 4) {
      z.x = max_nan(z.x, -FLT_MAX);
      z.y = max_nan(z.y, -FLT_MAX);
    }
    float2 u = __ffma2_rn(z, make_float2(hi, hi), make_float2(-lse, -lse));
    if (sizeof(E) == 4) u = __ffma2_rn(z, make_float2(lo, lo), u);
    u.x = floor_exp(u.x);
    u.y = floor_exp(u.y);
    const float k = 1.4426950408889634f;
    const float2 p = make_float2(fast_exp2(u.x * k), fast_exp2(u.y * k));
    return __fmul2_rn(p, __ffma2_rn(u, make_float2(b, b), make_float2(a, a)));
  }
  __device__ __forceinline__ float one(float z) const { return at(make_float2(z, z)).x; }
};

// A block takes a part of a row; its first loads go out before the row's scalars are there.
// Bound by HBM: 4,096 rows of 151,936 bf16 values 368 us, all of the copy's rate.  (Five blocks
// of 256 threads an SM and parts of 128 KB; with six and 64 KB 378 us, three of 512 422, two of
// 512, whose scalars nothing hides, 448.)  Where z and dz lie at other parts of 16 bytes (a padded
// odd vocabulary's rows and a dense gradient) dz is stored a value at a time: 2,000 bf16 rows of
// 50,257 values 261 us, 69 where they agree.
constexpr int kBwdVecs = 8192;
template <typename E>
__global__ void __launch_bounds__(kBwdThreads, kBwdCtas) logp_bwd(const BwdArgs a) {
  using R = Row<E>;
  constexpr int N = R::N;
  constexpr int kUnroll = 4;
  __shared__ float s_total;
  __shared__ int32_t special[33];  // the target and the alternatives
  __shared__ float special_z[33], special_g[33];
  const int tid = threadIdx.x;
  const int64_t row = a.parts == 1 ? blockIdx.x : blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - row * a.parts);
  const E* zr = static_cast<const E*>(a.logits) + row * a.ld;
  E* gr = static_cast<E*>(a.dlogits) + row * a.dld;
  const int lead = (int)((reinterpret_cast<uintptr_t>(zr) & 15) / sizeof(E));
  const int all = (int)(((int64_t)lead + a.V + N - 1) / N);
  const int v0 = (int)((int64_t)all * part / a.parts), v1 = (int)((int64_t)all * (part + 1) / a.parts);
  // vectors that lie wholly in the row
  const int in0 = lead > 0 ? 1 : 0, in1 = (lead + a.V) / N;
  const uint4* zv = reinterpret_cast<const uint4*>(zr - lead);
  uint4 u[kUnroll];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = i0 + k * kBwdThreads;
      if (i < v1 && i >= in0 && i < in1) u[k] = __ldcs(zv + i);
    }
  };
  load(v0 + tid);
  const int32_t y = a.targets ? __ldg(a.targets + row) : 0;
  const bool pad = a.targets && y == -1;
  const float h = a.d_entropy && !pad ? __ldg(a.d_entropy + row) : 0.f;
  const float lse = pad ? 0.f : __ldg(a.lse + row);
  const float he = h != 0.f ? h * __ldg(a.entropy + row) : 0.f;
  // ---- the row's upstream: g at the target, a_j at the alternatives, their sum
  if (tid < 32) {
    const bool has = tid < a.top && !pad;
    int32_t id = has ? a.top_ids[row * a.top + tid] : -1;
    float g = has ? a.d_top[row * a.top + tid] : 0.f;
    if (has && (uint32_t)id >= (uint32_t)a.V) {
      if (part == 0) ls_report(a.err, LS_DEVERR_CHECK);
      id = -1;
      g = NAN;
    }
    float sum = g;
    if (a.top > 0) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    special[1 + tid] = id;
    special_g[1 + tid] = g;
    if (id >= 0) special_z[1 + tid] = R::load(zr + id);
    if (tid == 0) {
      float gy = 0.f;
      special[0] = -1;
      if (a.targets && !pad) {
        gy = a.d_logp ? a.d_logp[row] : 0.f;
        if ((uint32_t)y < (uint32_t)a.V) {
          special[0] = y;
          special_z[0] = R::load(zr + y);
        } else {
          if (part == 0) ls_report(a.err, LS_DEVERR_CHECK);
          gy = NAN;
        }
      }
      special_g[0] = gy;
      s_total = sum + gy;
    }
  }
  __syncthreads();
  RowGrad<E> rg;
  rg.lse = lse;
  rg.hi = a.inv_hi;
  rg.lo = a.inv_lo;
  rg.a = -(s_total + he) * a.inv_hi;
  rg.b = -h * a.inv_hi;
  const bool same = ((reinterpret_cast<uintptr_t>(gr) - reinterpret_cast<uintptr_t>(zr)) & 15) == 0;
  for (int i0 = v0 + tid; i0 < v1; i0 += kUnroll * kBwdThreads) {
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = i0 + k * kBwdThreads;
      if (i >= v1) continue;
      float x[N];
      const bool whole = i >= in0 && i < in1;
      const int64_t at = (int64_t)i * N - lead;
      if (whole) {
        R::unpack(u[k], x);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = at + e >= 0 && at + e < a.V ? R::load(zr + at + e) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float2 g = pad ? make_float2(0.f, 0.f) : rg.at(make_float2(x[e], x[e + 1]));
        x[e] = g.x;
        x[e + 1] = g.y;
      }
      if (whole && same) {
        __stcs(reinterpret_cast<uint4*>(gr + at), R::pack(x));
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (at + e >= 0 && at + e < a.V) R::store(gr + at + e, x[e]);
      }
    }
    load(i0 + kUnroll * kBwdThreads);
  }
  // ---- the target and the alternatives, over what the pass wrote there
  __syncthreads();
  if (!pad && tid < 33 && special[tid] >= 0) {
    const int32_t v = special[tid];
    const int i = (v + lead) / N;
    bool first = i >= v0 && i < v1;
    float g = 0.f;
    for (int j = 0; j < 33; ++j)
      if (special[j] == v) {
        if (j < tid) first = false;
        g += special_g[j];
      }
    if (first) R::store(gr + v, fmaf(g, a.inv_hi, rg.one(special_z[tid])));
  }
}

}  // namespace

namespace {
int groups_of(bool is_bf16, int V) {  // of a row that begins inside a group
  const int G = is_bf16 ? 32 : 16;
  return (int)(((int64_t)V + G - 1 + G - 1) / G);
}
}  // namespace

namespace {
size_t rows_smem_bytes(int cap, bool top, int W) {
  const size_t rows = kRowsWarps / W;
  if (!top) return W > 1 ? rows * sizeof(RowSmem) : 0;
  return rows * (sizeof(RowSmem) + cap * sizeof(uint16_t));
}
int rows_cap(bool is_bf16, int V) { return (V / (is_bf16 ? 8 : 4) + 2 + 7) & ~7; }


// Warps that take a row, 0: rows are streamed (logp_fwd).  Rows go to warps where what follows a row
// costs more than its logits: up to 80 KB a row (4,096 bf16 rows of 32,003 values: 48 us against 66
// streamed, 2,000 of 50,257: 51 against 44), with alternatives up to 160 KB of bf16 or 96 KB of fp32
// (with 20 of them 4,096 bf16 rows of 1,000 values: 14 against 196 us, of 32,003: 73 against 182; of
// 151,936: 272 against 200; 4,096 fp32 rows of 16,000: 60 against 110, 2,000 of 50,257: 97 against 70),
// but few long rows, which are cut into parts over all SMs.  More warps a row until four CTAs fit an
// SM and 12 warps an SM have a row, two vectors a lane at least, and a lane adds at most 512 pairs
// (1,000 rows of 8,000 values with 20 alternatives: 17, 14, 16, 20 us with 1, 2, 4, 8 warps; 4,096 of
// 32,003: 102, 83, 89, 106; all of these before the maxima went in front of the sums).
int rows_warps(bool is_bf16, int64_t T, int V, int top, int sms) {
  const int64_t bytes = (int64_t)V * (is_bf16 ? 2 : 4);
  if (bytes > (top == 0 ? 80 : is_bf16 ? 160 : 96) * 1024 || (bytes > 64 * 1024 && T < sms)) return 0;
  const int cap = rows_cap(is_bf16, V);
  int W = 1;
  while (W < kRowsWarps && (rows_smem_bytes(cap, top > 0, W) > 56 * 1024 ||
                            (T * W < 12 * sms && bytes > 16 * 64 * W) || V > 32768 * W))
    W *= 2;
  return W;
}
}  // namespace

// Parts of a row: as many as its group maxima take blocks of shared memory, and with few rows
// as many as make an item for every SM, of a chunk at least.
int ls_token_logp_parts(bool is_bf16, int64_t T, int V, int top, int sms) {
  if (rows_warps(is_bf16, T, V, top, sms) > 0) return 1;
  const int64_t groups = groups_of(is_bf16, V), room = kMaxGroups;
  int64_t parts = top > 0 ? (groups + room - 1) / room : 1;
  if (T > 0 && T * parts < sms) {
    int64_t more = sms / T;
    const int64_t most = (groups + kThreads - 1) / kThreads;
    if (more > most) more = most;
    if (more > parts) parts = more;
  }
  return (int)parts;
}
size_t ls_token_logp_ws_bytes(int64_t T, int parts) {
  return parts > 1 ? (size_t)T * parts * (16 + 32 * 8) : 0;
}

namespace {
template <typename E, bool kTop, int W>
cudaError_t launch_rows(const FwdArgs& a, cudaStream_t st) {
  const int cap = rows_cap(sizeof(E) == 2, a.V);
  const size_t smem = rows_smem_bytes(cap, kTop, W);
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(logp_rows<E, kTop, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int64_t rows = kRowsWarps / W;
  logp_rows<E, kTop, W><<<(unsigned)((a.T + rows - 1) / rows), kRowsThreads, smem, st>>>(a, cap);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}
template <typename E, bool kTop>
cudaError_t launch_rows(const FwdArgs& a, int W, cudaStream_t st) {
  return W == 1 ? launch_rows<E, kTop, 1>(a, st) : W == 2 ? launch_rows<E, kTop, 2>(a, st)
       : W == 4 ? launch_rows<E, kTop, 4>(a, st) : launch_rows<E, kTop, 8>(a, st);
}

template <typename E, bool kTop>
cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t st) {
  // without alternatives nothing behind `red` is used
  const size_t smem = Cfg<kTop>::kStages * kChunkBytes + (kTop ? sizeof(FwdSmem) : offsetof(FwdSmem, best));
  cudaError_t e =
      cudaFuncSetAttribute(logp_fwd<E, kTop>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  logp_fwd<E, kTop><<<(unsigned)(a.T * a.parts), kCtaThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ls_note_launch();
  if (a.parts == 1) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.T);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, logp_merge<E, kTop>, a);
  if (e == cudaSuccess) ls_note_launch();
  return e;
}
}  // namespace

cudaError_t ls_launch_token_logp_fwd(const LsTokenLogpArgs& b, int parts, int sms, cudaStream_t st) {
  FwdArgs a{};
  a.logits = b.logits;
  a.T = b.T;
  a.ld = b.ld;
  a.V = b.V;
  a.top = b.top;
  a.parts = parts;
  a.steal = b.T * parts > 2 * sms;
  a.targets = b.targets;
  a.inv_tau = 1.0 / (double)b.temperature;
  a.c = (float)(kLog2ed * a.inv_tau);
  a.c_off = ((double)a.c - kLog2ed * a.inv_tau) / (double)a.c;
  a.out = {b.logp, b.lse, b.entropy, b.top_logp, b.top_ids};
  a.part_top = static_cast<u64*>(b.workspace);
  a.part_stat = reinterpret_cast<float*>(a.part_top + (size_t)b.T * parts * 32);
  a.err = b.err;
  const int W = rows_warps(b.is_bf16, b.T, b.V, b.top, sms);
  if (W > 0) {
    if (b.is_bf16)
      return b.top > 0 ? launch_rows<__nv_bfloat16, true>(a, W, st) : launch_rows<__nv_bfloat16, false>(a, W, st);
    return b.top > 0 ? launch_rows<float, true>(a, W, st) : launch_rows<float, false>(a, W, st);
  }
  if (b.is_bf16)
    return b.top > 0 ? launch_fwd<__nv_bfloat16, true>(a, st) : launch_fwd<__nv_bfloat16, false>(a, st);
  return b.top > 0 ? launch_fwd<float, true>(a, st) : launch_fwd<float, false>(a, st);
}

// Parts of up to 128 KB, smaller ones when there are few rows.
int64_t ls_token_logp_bwd_parts(const LsTokenLogpBwdArgs& b, int sms) {
  const int N = b.is_bf16 ? 8 : 4;
  const int64_t vecs = ((int64_t)b.V + N - 1) / N + 1;
  int64_t parts = (vecs + kBwdVecs - 1) / kBwdVecs;
  if (b.T * parts < 2 * sms) {
    parts = (2 * sms + b.T - 1) / b.T;
    const int64_t most = (vecs + kBwdThreads - 1) / kBwdThreads;
    if (parts > most) parts = most;
  }
  return parts;
}

cudaError_t ls_launch_token_logp_bwd(const LsTokenLogpBwdArgs& b, int sms, cudaStream_t st) {
  BwdArgs a{};
  a.logits = b.logits;
  a.dlogits = b.dlogits;
  a.T = b.T;
  a.ld = b.ld;
  a.dld = b.dld;
  a.V = b.V;
  a.top = b.top;
  a.targets = b.targets;
  a.top_ids = b.top_ids;
  a.lse = b.lse;
  a.entropy = b.entropy;
  a.d_logp = b.d_logp;
  a.d_entropy = b.d_entropy;
  a.d_top = b.d_top;
  const double inv = 1.0 / (double)b.temperature;
  a.inv_hi = (float)inv;
  a.inv_lo = (float)(inv - (double)a.inv_hi);
  a.err = b.err;
  const int64_t parts = ls_token_logp_bwd_parts(b, sms);
  a.parts = (int)parts;
  if (b.is_bf16)
    logp_bwd<__nv_bfloat16><<<(unsigned)(a.T * parts), kBwdThreads, 0, st>>>(a);
  else
    logp_bwd<float><<<(unsigned)(a.T * parts), kBwdThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}
