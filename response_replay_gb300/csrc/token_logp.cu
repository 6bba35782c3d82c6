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
// Forward.  One pass over the row: every thread keeps a running maximum m, s = sum 2^t and
// e = sum 2^t t of t = (z - m) c (c = log2(e) / tau), so H = ln 2 (log2 s - e / s).  The
// alternatives ride along on the maxima that the pass takes anyway: a row is cut into groups
// of 32 bytes; each group's maximum goes to shared memory, and a thread keeps the largest of
// its groups (ties to the lowest group, which holds the lower ids).  Behind the row a warp
// takes the k-th largest of 32 maxima over disjoint groups, tau: k distinct logits reach it, so
// only groups whose maximum does can hold one of the k largest.  It reads those groups again
// (about 40 of 9,500 for k = 20) and sorts the logits that pass.
// A row too long for the group maxima, or a call with few rows, is cut into parts whose results
// a second kernel merges.
// Sums are in fp32 (a thread adds V / 512 terms, then a tree), the last steps in fp64.
#include <math.h>

#include "ls_device.cuh"
#include "ls_internal.h"

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxGroups = 12288;  // group maxima of a part: 48 KB
constexpr int kCand = 256;         // groups collected before they are read again
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
struct Row;  // 32-byte groups of a row
template <>
struct Row<float> {
  static constexpr int G = 8;
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
  static constexpr int G = 16;
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

// Logits and places as one number that orders them: larger logits first, equal ones (one
// zero) by the lower place.  NaN: 0, behind all.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  if (x != x) return 0u;
  return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ u64 key_of(float x, uint32_t place) {
  const uint32_t o = order_of(x);
  return o ? (u64)o << 32 | (uint32_t)~place : 0ull;
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

// Running maximum m of the logits, s = sum 2^t, e = sum 2^t t with t = (z - m) c.
struct Stat {
  float m, s, e;
};
__device__ __forceinline__ Stat merge(Stat a, Stat b, float c) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, a.s + b.s, a.e + b.e};  // no finite logit (or NaN sums)
  auto move = [&](Stat x) {
    if (x.m == -INFINITY) return x;
    const float d = (x.m - m) * c, f = fast_exp2(d);
    return Stat{m, x.s * f, (x.e + x.s * floor_exp(d)) * f};
  };
  a = move(a);
  b = move(b);
  return {m, a.s + b.s, a.e + b.e};
}

struct Out {
  float* logp;
  float* lse;
  float* entropy;
  float* top_logp;
  int32_t* top_ids;
};

// The row's numbers from its statistics; returns lse.
__device__ __forceinline__ double finish_row(const Stat& a, double inv_tau, const Out& out,
                                             int64_t row, bool has_y, float zy) {
  const double log2s = (double)log2f(a.s);
  const double lse = a.m == -INFINITY && a.s == 0.f ? -INFINITY
                                                    : (double)a.m * inv_tau + kLn2d * log2s;
  if (out.lse) out.lse[row] = (float)lse;
  if (out.entropy) out.entropy[row] = (float)(kLn2d * (log2s - (double)a.e / (double)a.s));
  if (out.logp) out.logp[row] = has_y ? (float)((double)zy * inv_tau - lse) : NAN;
  return lse;
}

struct FwdArgs {
  const void* logits;
  int64_t T, ld;
  int32_t V, top, parts;
  const int32_t* targets;
  float c;          // log2(e) / tau
  double inv_tau;
  Out out;
  float* part_stat;  // [T][parts][4]
  u64* part_top;     // [T][parts][32]
  uint32_t* err;
};

// Rows whose target is -1 are padding: their outputs are zeros and ids -1.
__device__ __forceinline__ bool padding_row(const FwdArgs& a, int64_t row, bool first, int lane) {
  if (!a.targets || a.targets[row] != -1) return false;
  if (first) {
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
  return true;
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

// What warp 0 needs besides to pick a part's largest logits.
struct TopSmem {
  u64 best[kThreads];  // each thread's largest group
  u64 found[64];       // logits that passed, on their way into the sorted list
  int32_t cand[kCand];
  float gmax[kMaxGroups];
};

// The 32 largest logits of groups [g0, g0 + ng), sorted, one a lane of the calling warp.
template <typename E>
__device__ u64 pick(TopSmem& sm, const E* zr, int V, int lead, int g0, int ng, int k, int lane) {
  constexpr int G = Row<E>::G;
  u64 mine = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) mine = max64(mine, sm.best[lane + 32 * i]);
  const u64 floor = __shfl_sync(0xffffffffu, sort32(mine, lane), k - 1);
  u64 list = 0;
  int found = 0, cands = 0;
  auto flush = [&] {
    __syncwarp();
    constexpr int kPer = 32 / G, kBatch = 8;  // groups a step; steps whose loads go together
    for (int j0 = 0; j0 < cands; j0 += kPer * kBatch) {
      u64 key[kBatch];
      bool pass[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int j = j0 + b * kPer + lane / G;
        key[b] = 0;
        pass[b] = false;
        if (j < cands) {
          const int g = sm.cand[j], at = (g0 + g) * G + lane % G - lead;
          if (at >= 0 && at < V) {
            const float x = Row<E>::load(zr + at);
            key[b] = key_of(x, at);
            pass[b] = key_of(x, g) >= floor;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const u64 kth = __shfl_sync(0xffffffffu, list, k - 1);  // by all lanes
        const bool in = pass[b] && key[b] > kth;
        const uint32_t mask = __ballot_sync(0xffffffffu, in);
        if (mask == 0) continue;
        if (in) sm.found[found + __popc(mask & ((1u << lane) - 1))] = key[b];
        found += __popc(mask);
        __syncwarp();
        if (found >= 32) {
          list = merge32(list, sort32(sm.found[found - 32 + lane], lane), lane);
          found -= 32;
          __syncwarp();
        }
      }
    }
    cands = 0;
  };
  for (int i = 0; i < kWarps; ++i) {
    const u64 b = sm.best[lane + 32 * i];
    uint32_t threads = __ballot_sync(0xffffffffu, b != 0 && b >= floor);
    while (threads) {
      const int t = 32 * i + __ffs(threads) - 1;
      threads &= threads - 1;
      for (int c0 = 0; t + c0 * kThreads < ng; c0 += 32) {
        const int g = t + (c0 + lane) * kThreads;
        const bool in = g < ng && key_of(sm.gmax[g], g) >= floor;
        const uint32_t mask = __ballot_sync(0xffffffffu, in);
        if (in) sm.cand[cands + __popc(mask & ((1u << lane) - 1))] = g;
        cands += __popc(mask);
        if (cands > kCand - 32) flush();
      }
    }
  }
  flush();
  if (found) list = merge32(list, sort32(lane < found ? sm.found[lane] : 0ull, lane), lane);
  return list;
}

__device__ __forceinline__ void write_top(const Out& out, int64_t row, int top, u64 key, double lse,
                                          double inv_tau, int lane) {
  if (lane >= top) return;
  out.top_logp[row * top + lane] = key ? (float)((double)value_of(key) * inv_tau - lse) : NAN;
  out.top_ids[row * top + lane] = key ? (int32_t)~(uint32_t)key : -1;
}

template <typename E, bool kTop>
__global__ void __launch_bounds__(kThreads, 3) logp_fwd(const FwdArgs a) {
  using R = Row<E>;
  constexpr int G = R::G, H = G / 2;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Stat red[kWarps];
  TopSmem& sm = *reinterpret_cast<TopSmem*>(dyn);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - row * a.parts);
  // the merge may be launched: its blocks wait for this grid before they read from it
  if (a.parts > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (padding_row(a, row, part == 0 && warp == 0, lane)) return;
  const E* zr = static_cast<const E*>(a.logits) + row * a.ld;
  // groups of 32 bytes by address; the first and the last one may stick out of the row
  const int lead = (int)((reinterpret_cast<uintptr_t>(zr) & 31) / sizeof(E));
  const int64_t all = ((int64_t)lead + a.V + G - 1) / G;
  const int g0 = (int)(all * part / a.parts), ng = (int)(all * (part + 1) / a.parts) - g0;
  const E* base = zr - lead + (int64_t)g0 * G;  // of the part's first group
  const float c = a.c;
  float m = -INFINITY, bestv = -INFINITY;
  int bestg = -1;
  float2 s = {0.f, 0.f}, e = {0.f, 0.f};
  auto add = [&](const float* x, int g) {
    float mx = fmax3(x[0], x[1], x[2]);
#pragma unroll
    for (int i = 3; i + 1 < G; i += 2) mx = fmax3(mx, x[i], x[i + 1]);
    mx = fmaxf(mx, x[G - 1]);
    if (kTop) {
      sm.gmax[g] = mx;
      if (mx > bestv || bestg < 0) {
        bestv = mx;
        bestg = g;
      }
    }
    if (mx > m) {
      if (m != -INFINITY) {
        const float d = (m - mx) * c, f = fast_exp2(d), dd = floor_exp(d);
        e.x = (e.x + s.x * dd) * f;
        e.y = (e.y + s.y * dd) * f;
        s.x *= f;
        s.y *= f;
      }
      m = mx;
    }
    const float nm = m == -INFINITY ? 0.f : -m;
    const float2 c2 = make_float2(c, c), b = make_float2(nm, nm);
#pragma unroll
    for (int i = 0; i < G; i += 2) {
      float2 t = __fmul2_rn(__fadd2_rn(make_float2(x[i], x[i + 1]), b), c2);
      t.x = floor_exp(t.x);
      t.y = floor_exp(t.y);
      const float2 p = make_float2(fast_exp2(t.x), fast_exp2(t.y));
      s = __fadd2_rn(s, p);
      e = __ffma2_rn(p, t, e);
    }
  };
  auto edge = [&](int g) {  // a group that sticks out of the row
    float x[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int64_t at = (int64_t)(g0 + g) * G + i - lead;
      x[i] = at >= 0 && at < a.V ? R::load(zr + at) : -INFINITY;
    }
    add(x, g);
  };
  const bool cut0 = g0 == 0 && lead > 0, cut1 = part == a.parts - 1 && (lead + (int64_t)a.V) % G != 0;
  const int in0 = cut0 ? 1 : 0, in1 = ng - (cut1 ? 1 : 0);
  constexpr int kUnroll = 2;
  for (int gg = tid; gg < ng; gg += kUnroll * kThreads) {
    uint4 u[kUnroll][2];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int g = gg + k * kThreads;
      if (g >= in0 && g < in1) {
        const uint4* p = reinterpret_cast<const uint4*>(base + (int64_t)g * G);
        u[k][0] = __ldcs(p);
        u[k][1] = __ldcs(p + 1);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int g = gg + k * kThreads;
      if (g >= in0 && g < in1) {
        float x[G];
        R::unpack(u[k][0], x);
        R::unpack(u[k][1], x + H);
        add(x, g);
      } else if (g < ng) {
        edge(g);
      }
    }
  }
  Stat st = {m, s.x + s.y, e.x + e.y};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    st = merge(st, Stat{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                        __shfl_xor_sync(0xffffffffu, st.e, o)}, c);
  if (lane == 0) red[warp] = st;
  if (kTop) sm.best[tid] = bestg < 0 ? 0ull : key_of(bestv, bestg);
  __syncthreads();
  if (warp != 0) return;
  st = lane < kWarps ? red[lane] : Stat{-INFINITY, 0.f, 0.f};
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1)
    st = merge(st, Stat{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                        __shfl_xor_sync(0xffffffffu, st.e, o)}, c);
  st = Stat{__shfl_sync(0xffffffffu, st.m, 0), __shfl_sync(0xffffffffu, st.s, 0),
            __shfl_sync(0xffffffffu, st.e, 0)};
  u64 list = 0;
  if (kTop) list = pick<E>(sm, zr, a.V, lead, g0, ng, a.top, lane);
  if (a.parts > 1) {
    const int64_t at = row * a.parts + part;
    if (lane == 0) *reinterpret_cast<float4*>(a.part_stat + 4 * at) = make_float4(st.m, st.s, st.e, 0.f);
    if (kTop) a.part_top[at * 32 + lane] = list;
    return;
  }
  double lse = 0.0;
  if (lane == 0) {
    float zy = 0.f;
    const bool has = target_logit<E>(a, row, &zy);
    lse = finish_row(st, a.inv_tau, a.out, row, has, zy);
  }
  if (kTop) write_top(a.out, row, a.top, list, __shfl_sync(0xffffffffu, lse, 0), a.inv_tau, lane);
}

// Rows that were cut into parts: a block a row, its warps take the parts by turns.
constexpr int kMergeWarps = 8;
template <typename E, bool kTop>
__global__ void __launch_bounds__(kMergeWarps * 32) logp_merge(const FwdArgs a) {
  __shared__ Stat red[kMergeWarps];
  __shared__ u64 lists[kMergeWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (padding_row(a, row, false, lane)) return;
  Stat st = {-INFINITY, 0.f, 0.f};
  u64 list = 0;
  for (int p = warp; p < a.parts; p += kMergeWarps) {
    const int64_t at = row * a.parts + p;
    const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part_stat + 4 * at));
    st = merge(st, Stat{x.x, x.y, x.z}, a.c);
    if (kTop) list = merge32(list, __ldcg(a.part_top + at * 32 + lane), lane);
  }
  if (lane == 0) red[warp] = st;
  if (kTop) lists[warp][lane] = list;
  __syncthreads();
  if (warp != 0) return;
  for (int w = 1; w < kMergeWarps; ++w) {
    st = merge(st, red[w], a.c);
    if (kTop) list = merge32(list, lists[w][lane], lane);
  }
  double lse = 0.0;
  if (lane == 0) {
    float zy = 0.f;
    const bool has = target_logit<E>(a, row, &zy);
    lse = finish_row(st, a.inv_tau, a.out, row, has, zy);
  }
  if (kTop) write_top(a.out, row, a.top, list, __shfl_sync(0xffffffffu, lse, 0), a.inv_tau, lane);
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
    // has to be a finite one.
    if (sizeof(E) == 4) {
      z.x = max_nan(z.x, -1e30f);
      z.y = max_nan(z.y, -1e30f);
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

template <typename E>
__global__ void __launch_bounds__(kThreads) logp_bwd(const BwdArgs a) {
  using R = Row<E>;
  constexpr int N = R::G / 2;  // values of 16 bytes
  __shared__ float s_total;
  __shared__ int32_t special[33];  // the target and the alternatives
  __shared__ float special_z[33], special_g[33];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - row * a.parts);
  const E* zr = static_cast<const E*>(a.logits) + row * a.ld;
  E* gr = static_cast<E*>(a.dlogits) + row * a.dld;
  const int lead = (int)((reinterpret_cast<uintptr_t>(zr) & 15) / sizeof(E));
  const int64_t all = ((int64_t)lead + a.V + N - 1) / N;
  const int64_t v0 = all * part / a.parts, v1 = all * (part + 1) / a.parts;
  const int32_t y = a.targets ? a.targets[row] : 0;
  const bool pad = a.targets && y == -1;
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
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    special[1 + tid] = id;
    special_g[1 + tid] = g;
    if (id >= 0) special_z[1 + tid] = R::load(zr + id);
    if (tid == 0) {
      float gy = 0.f;
      special[0] = -1;
      if (a.targets && !pad) {
        gy = a.d_logp[row];
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
  const float h = a.d_entropy && !pad ? a.d_entropy[row] : 0.f;
  rg.lse = pad ? 0.f : a.lse[row];
  rg.hi = a.inv_hi;
  rg.lo = a.inv_lo;
  rg.a = -(s_total + (h != 0.f ? h * a.entropy[row] : 0.f)) * a.inv_hi;
  rg.b = -h * a.inv_hi;
  const bool zero = pad;
  const bool same = ((reinterpret_cast<uintptr_t>(gr) - reinterpret_cast<uintptr_t>(zr)) & 15) == 0;
  constexpr int kUnroll = 4;
  for (int64_t i0 = v0 + tid; i0 < v1; i0 += kUnroll * kThreads) {
    uint4 u[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int64_t i = i0 + k * kThreads, at = i * N - lead;
      if (i < v1 && at >= 0 && at + N <= a.V && !zero) u[k] = __ldcs(reinterpret_cast<const uint4*>(zr + at));
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int64_t i = i0 + k * kThreads, at = i * N - lead;
      if (i >= v1) continue;
      float x[N];
      const bool whole = at >= 0 && at + N <= a.V;
      if (zero) {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = 0.f;
      } else {
        if (whole) {
          R::unpack(u[k], x);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) x[e] = at + e >= 0 && at + e < a.V ? R::load(zr + at + e) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float2 g = rg.at(make_float2(x[e], x[e + 1]));
          x[e] = g.x;
          x[e + 1] = g.y;
        }
      }
      if (whole && same) {
        __stcs(reinterpret_cast<uint4*>(gr + at), R::pack(x));
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (at + e >= 0 && at + e < a.V) R::store(gr + at + e, x[e]);
      }
    }
  }
  // ---- the target and the alternatives, over what the pass wrote there
  __syncthreads();
  if (!zero && tid < 33 && special[tid] >= 0) {
    const int32_t v = special[tid];
    const int64_t i = ((int64_t)v + lead) / N;
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
  const int G = is_bf16 ? 16 : 8;
  return (int)(((int64_t)V + G - 1 + G - 1) / G);
}
}  // namespace

// Parts of a row: as many as its group maxima take blocks of shared memory, and with few rows
// as many as make a block for every SM, of a group a thread at least.
int ls_token_logp_parts(bool is_bf16, int64_t T, int V, int top, int sms) {
  const int64_t groups = groups_of(is_bf16, V);
  int64_t parts = top > 0 ? (groups + kMaxGroups - 1) / kMaxGroups : 1;
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
template <typename E, bool kTop>
cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t st) {
  const size_t smem = kTop ? sizeof(TopSmem) : 0;
  if (kTop) {
    const cudaError_t e =
        cudaFuncSetAttribute(logp_fwd<E, kTop>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  logp_fwd<E, kTop><<<(unsigned)(a.T * a.parts), kThreads, smem, st>>>(a);
  cudaError_t e = cudaGetLastError();
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

cudaError_t ls_launch_token_logp_fwd(const LsTokenLogpArgs& b, int parts, cudaStream_t st) {
  FwdArgs a{};
  a.logits = b.logits;
  a.T = b.T;
  a.ld = b.ld;
  a.V = b.V;
  a.top = b.top;
  a.parts = parts;
  a.targets = b.targets;
  a.c = (float)(kLog2ed / (double)b.temperature);
  a.inv_tau = 1.0 / (double)b.temperature;
  a.out = {b.logp, b.lse, b.entropy, b.top_logp, b.top_ids};
  a.part_top = static_cast<u64*>(b.workspace);
  a.part_stat = reinterpret_cast<float*>(a.part_top + (size_t)b.T * parts * 32);
  a.err = b.err;
  if (b.is_bf16)
    return b.top > 0 ? launch_fwd<__nv_bfloat16, true>(a, st) : launch_fwd<__nv_bfloat16, false>(a, st);
  return b.top > 0 ? launch_fwd<float, true>(a, st) : launch_fwd<float, false>(a, st);
}

// Parts of about 64 KB, smaller ones when there are few rows.
int64_t ls_token_logp_bwd_parts(const LsTokenLogpBwdArgs& b, int sms) {
  const int N = b.is_bf16 ? 8 : 4;
  const int64_t vecs = ((int64_t)b.V + N - 1) / N + 1;
  int64_t parts = (vecs + 4095) / 4096;
  if (b.T * parts < 2 * sms) {
    parts = (2 * sms + b.T - 1) / b.T;
    const int64_t most = (vecs + kThreads - 1) / kThreads;
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
    logp_bwd<__nv_bfloat16><<<(unsigned)(a.T * parts), kThreads, 0, st>>>(a);
  else
    logp_bwd<float><<<(unsigned)(a.T * parts), kThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}
