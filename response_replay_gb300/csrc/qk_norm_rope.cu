// qk_norm_rope.cu -- the stage between a layer's projections and its attention: the
// per-head RMS norm of queries and keys with the rotary positions in the same pass,
// its backward, and the forward with keys and values written to pages by slot.
//
// A row is one head of one token, x of 128 values:
//   r = 1 / sqrt(mean x^2 + eps),  u_i = x_i r (w_offset + w_i),
//   y = u with each of its first `rot_dim` values' pairs (a, b) turned by the token's
//   angle of that pair: (a cos - b sin, b cos + a sin); pairs are (i, i + rot_dim / 2)
//   or, interleaved, (2 i, 2 i + 1).
// Backward, with g the pairs of dy turned back, xh = x r, h = g (w_offset + w):
//   dx = r (h - xh mean(h xh)),  dw_i = sum over rows g_i xh_i.
//
// Angles.  angle = position x inv_freq, with positions up to 2^31: the product in 32
// bits would lose the angle (at position 4,194,304 one fp32 step is 0.25 rad for the
// fastest pair).  A pair's turns per position (inv_freq / 2 pi, its fractional part) are
// taken as a 64-bit fixed-point fraction, so that position x fraction modulo 2^64 is the
// angle's fraction of a turn exactly.  The error until there is that of the fraction (2^-54
// of a turn per position for frequencies up to 2 pi: 2^-32 at 4,194,304).  Its top 32 bits,
// as an fp32 number of half turns in [-1, 1) (a rounding of up to 2^-26 of a turn, which is
// what the angle is off by), go through sincospif.
#include "ls_device.cuh"
#include "ls_internal.h"

namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = kThreads / 16;  // half-warps
constexpr float kOverflow = 3.0e38f;

// How the rows are spread.  A warp works on two neighbouring tokens at once, one a
// half-warp (16 lanes of 8 values), head by head; a token's rows are its query heads, its
// key heads and, where they are asked for, its value heads.  All rows of all pairs of
// tokens form one sequence that is cut evenly over the warps of the grid: a warp's part
// may begin and end inside a pair, so every warp has the same work whatever T and the
// head counts are (dealing out whole tokens left SMs idle for 16% of the time at 4,096).
struct Spread {
  int64_t total;   // ceil(T / 2) x rows
  int32_t rows;    // rows of a token
  int32_t warps;   // warps that have a part
};

// A warp's rows as batches of up to kMax rows of one kind (0 query, 1 key, 2 value) of one
// pair.  Within a run of one kind a step is an addition and a comparison.
template <int kMax>
struct Walk {
  int64_t pair;
  int32_t left;          // the warp's rows from this batch on
  int32_t r, n, end;     // first row of the token, rows, end of the run
  int32_t kind;
  bool first;            // first batch of its run

  __device__ __forceinline__ void begin(const LsNormRopeArgs& a, const Spread& s, int32_t warp) {
    const int64_t i0 = s.total * warp / s.warps;
    left = warp < s.warps ? (int32_t)(s.total * (warp + 1) / s.warps - i0) : 0;
    pair = i0 / s.rows;
    r = (int32_t)(i0 - pair * s.rows);
    run(a);
  }
  __device__ __forceinline__ void next(const LsNormRopeArgs& a, const Spread& s) {
    r += n;
    left -= n;
    first = false;
    n = min(kMax, end - r);
    if (n > 0) return;
    if (r == s.rows) {
      r = 0;
      ++pair;
    }
    run(a);
  }
  // first head of the batch
  __device__ __forceinline__ int32_t head(const LsNormRopeArgs& a) const {
    return r - (kind > 0 ? a.hq : 0) - (kind > 1 ? a.hkv : 0);
  }

 private:
  __device__ __forceinline__ void run(const LsNormRopeArgs& a) {
    kind = r < a.hq ? 0 : (r < a.hq + a.hkv ? 1 : 2);
    end = min(kind == 0 ? a.hq : a.hq + kind * a.hkv, r + left);
    n = min(kMax, end - r);
    first = true;
  }
};

// The block's constants in shared memory.
struct Const {
  unsigned long long f[kD / 2];     // turns per position of each pair, as a fraction of 2^64
  int32_t axis[kD / 2];
  __align__(16) float w[2][kD];     // w_offset + w of queries and keys
  __align__(16) float2 tab[kGroups][kD / 2];  // (cos, sin) of a half-warp's token
};

__device__ __forceinline__ void load_const(const LsNormRopeArgs& a, Const& c) {
  const int i = threadIdx.x;
  {
    const void* p = a.w[i / kD];
    float v = 1.f;
    if (a.norm && p)
      v = a.w_offset + (a.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i % kD])
                                 : static_cast<const float*>(p)[i % kD]);
    c.w[i / kD][i % kD] = v;
  }
  if (i < kD / 2) {
    int ax = 0;
    unsigned long long f = 0;
    if (i < a.half) {
      ax = a.pair_axis ? __ldg(a.pair_axis + i) : 0;
      if ((uint32_t)ax >= (uint32_t)a.axes) {
        ls_report(a.err, LS_DEVERR_CHECK);
        ax = 0;
      }
      const double turns = __ldg(a.inv_freq + i) * 0.15915494309189533577;  // 1 / (2 pi)
      f = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
    }
    c.f[i] = f;
    c.axis[i] = ax;
  }
}
static_assert(kThreads == 2 * kD, "a thread per weight");

// A half-warp's angles: lane l has pairs l, l + 16, l + 32, l + 48.  The next token's
// positions are loaded while the current one's rows go by.
struct Positions {
  int32_t p[4];
  __device__ __forceinline__ void fetch(const LsNormRopeArgs& a, const Const& c, int64_t t, int l) {
    if (t >= a.T) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = l + 16 * i;
      p[i] = j < a.half ? __ldg(a.pos + c.axis[j] * a.T + t) : 0;
    }
  }
  // position x turns per position, modulo a turn, exactly; its top 32 bits to (cos, sin)
  __device__ __forceinline__ void angles(const LsNormRopeArgs& a, const Const& c, int l,
                                         float2* tab) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = l + 16 * i;
      if (j >= a.half) break;
      const unsigned long long ph = (unsigned long long)(long long)p[i] * c.f[j];
      float2 cs;
      sincospif((float)(int32_t)(ph >> 32) * 4.656612873077392578125e-10f, &cs.y, &cs.x);
      tab[j] = cs;
    }
  }
};

// What a lane needs of the rotation of its values 8 l .. 8 l + 7, as pairs of values:
// y = u cos + (other half of the pair) sin, sin negated for the first of a pair.
template <bool kInter>
struct Turn {
  float2 c[4], s[4];

  __device__ __forceinline__ void load(const LsNormRopeArgs& a, const float2* tab, int l, int partner,
                                       bool back) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = make_float2(1.f, 1.f);
      s[i] = make_float2(0.f, 0.f);
    }
    if (l >= a.half / 4) return;
    if (kInter) {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float4 v = *reinterpret_cast<const float4*>(tab + 4 * l + i);
        c[i] = make_float2(v.x, v.x);
        c[i + 1] = make_float2(v.z, v.z);
        s[i] = back ? make_float2(v.y, -v.y) : make_float2(-v.y, v.y);
        s[i + 1] = back ? make_float2(v.w, -v.w) : make_float2(-v.w, v.w);
      }
    } else {
      const bool first = l < partner;
      const float sg = first != back ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(tab + 8 * (first ? l : partner) + 2 * i);
        c[i] = make_float2(v.x, v.z);
        s[i] = make_float2(sg * v.y, sg * v.w);
      }
    }
  }
};

// Split halves: lane of the half-warp with the other halves of lane l's pairs.
__device__ __forceinline__ int partner_of(const LsNormRopeArgs& a, int l) {
  if (a.interleaved || l >= a.half / 4) return l;
  return l < a.half / 8 ? l + a.half / 8 : l - a.half / 8;
}

__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float2 swap2(float2 v) { return make_float2(v.y, v.x); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ void unpack8(const uint4& w, float2* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const float2* x) {
  return make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y), pack_bf16(x[2].x, x[2].y),
                    pack_bf16(x[3].x, x[3].y));
}
__device__ __forceinline__ float dot8(const float2* x, const float2* y) {
  float2 s = __fmul2_rn(x[0], y[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = __ffma2_rn(x[i], y[i], s);
  return s.x + s.y;
}

// bf16 values reach 3e38, whose squares do not fit fp32: the values of such a row are
// scaled by 2^-80 and summed again, and eps with their squares.
constexpr float kDown = 8.271806125530277e-25f;
__device__ __forceinline__ float rsqrt_ftz(float x) {  // x is a normal number here
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_down(float ss, float eps) {
  return rsqrt_ftz(fmaf(ss, 1.f / kD, eps * kDown * kDown));
}
__device__ __forceinline__ void scale8(float2* x, float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __fmul2_rn(x[i], both(f));
}

__device__ __forceinline__ void weights8(const float* w, int l, float2* x) {
  const float4 p = *reinterpret_cast<const float4*>(w + 8 * l);
  const float4 q = *reinterpret_cast<const float4*>(w + 8 * l + 4);
  x[0] = make_float2(p.x, p.y);
  x[1] = make_float2(p.z, p.w);
  x[2] = make_float2(q.x, q.y);
  x[3] = make_float2(q.z, q.w);
}

// Rows come through a ring in shared memory (cp.async): a warp works on one batch while the
// next one is on its way, across heads, kinds and tokens.  The ring is a warp's own, so it
// needs no barrier of the block, costs no registers (held in registers the rows took 32 to
// 48, and the kernels spilled), and gives a lane the other halves of its pairs with one or
// two 16-byte reads instead of four or eight shuffles.
__device__ __forceinline__ void cp_async16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Forward.  It reads and writes every row once and is bound by that: 32,768 tokens of 24
// query, 4 key and 4 value heads 87 us, 6.2 TB/s, 91% of what a plain copy reaches; 8,191
// tokens of 32 heads with three axes 26 us, 77%, where the launch and the first and last rows
// count; 256 tokens 4.8 us, a launch.  Two blocks an SM and four rows a batch: with two rows
// a batch the 32,768 tokens take 101 us, with six 95; three blocks, whose registers spill,
// 102 us with four rows and 89 with three.
constexpr int kFwdRows = 4, kFwdCtas = 2;

template <bool kAppend, bool kInter>
__global__ void __launch_bounds__(kThreads, kFwdCtas)
norm_rope_fwd_kernel(const __grid_constant__ LsNormRopeArgs a, const __grid_constant__ LsRows x,
                     const __grid_constant__ LsRows y, const __grid_constant__ LsPoolDst dst,
                     const __grid_constant__ Spread sp) {
  __shared__ Const cst;
  __shared__ uint4 ring[2][kFwdRows][kThreads];
  const int l = threadIdx.x & 15, grp = threadIdx.x >> 4, half = grp & 1;
  float2* tab = cst.tab[grp];
  const int partner = partner_of(a, l);
  const bool active = l < a.half / 4;  // the lane's values are rotated

  Walk<kFwdRows> w;  // one batch ahead
  w.begin(a, sp, blockIdx.x * kWarps + (threadIdx.x >> 5));
  const uint4* src = nullptr;
  int64_t shs = 0;
  auto load = [&](int to) {
    if (w.n > 0 && 2 * w.pair + half < a.T) {
      if (w.first) {
        shs = x.hs[w.kind] >> 3;
        src = static_cast<const uint4*>(x.p[w.kind]) +
              (((2 * w.pair + half) * x.ts[w.kind] + w.head(a) * x.hs[w.kind]) >> 3) + l;
      }
#pragma unroll
      for (int i = 0; i < kFwdRows; ++i) {
        if (i < w.n) cp_async16(&ring[to][i][threadIdx.x], src);
        src += shs;
      }
    }
    cp_async_commit();
  };

  load(0);
  load_const(a, cst);
  Positions pos;
  int32_t next_slot = -1;
  int64_t t = 2 * w.pair + half;
  if (kAppend && t < a.T) next_slot = __ldg(dst.slots + t);
  __syncthreads();
  pos.fetch(a, cst, t, l);
  float2 cw[4], sw[4];  // cos and sin with the scale of the value they meet
  bool live = false, paged = false;
  int64_t pair = -1, page_row = 0;  // page_row: row of the token's slot in a pool, head 0
  uint4* out = nullptr;
  int64_t ohs = 0;
  int slot = 0;
  bool write = false;

  while (w.n > 0) {
    const int n = w.n, kind = w.kind, head = w.head(a);
    const int64_t p = w.pair;
    const bool first = w.first;
    w.next(a, sp);
    __syncwarp();  // the other slot has been read by all
    load(slot ^ 1);
    if (p != pair) {  // another pair of tokens
      pair = p;
      t = 2 * pair + half;
      live = t < a.T;
      __syncwarp();  // the last pair's angles have been read
      pos.angles(a, cst, l, tab);
      if (kAppend) {
        const int32_t s = next_slot;
        live = live && s >= 0;  // a padding token: nothing of it is written
        paged = live && (s >> dst.ps_log2) < dst.num_pages;
        if (live && !paged && l == 0) ls_report(a.err, LS_DEVERR_CHECK);
        page_row = ((int64_t)(s >> dst.ps_log2) * a.hkv << dst.ps_log2) + (s & ((1 << dst.ps_log2) - 1));
        next_slot = t + 2 < a.T ? __ldg(dst.slots + t + 2) : -1;
      }
      pos.fetch(a, cst, t + 2, l);
      __syncwarp();
    }
    if (first) {  // another kind of head, or another pair
      Turn<kInter> turn;
      turn.load(a, tab, l, partner, false);
      float2 wt[4];
      weights8(cst.w[kind & 1], l, wt);
#pragma unroll
      for (int i = 0; i < 4; ++i) cw[i] = __fmul2_rn(turn.c[i], wt[i]);
      if (kInter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sw[i] = __fmul2_rn(turn.s[i], swap2(wt[i]));
      } else {
        weights8(cst.w[kind & 1], partner, wt);
#pragma unroll
        for (int i = 0; i < 4; ++i) sw[i] = __fmul2_rn(turn.s[i], wt[i]);
      }
      write = live;
      if (kAppend && kind > 0) {
        out = static_cast<uint4*>(kind == 1 ? dst.k_pool : dst.v_pool) +
              (page_row + ((int64_t)head << dst.ps_log2)) * 16 + l;
        ohs = 16ll << dst.ps_log2;
        write = paged;
      } else {
        out = static_cast<uint4*>(const_cast<void*>(y.p[kind])) +
              ((t * y.ts[kind] + head * y.hs[kind]) >> 3) + l;
        ohs = y.hs[kind] >> 3;
      }
    }
    cp_async_wait<1>();
    __syncwarp();  // the batch is there for all
#pragma unroll
    for (int i = 0; i < kFwdRows; ++i) {
      if (i >= n) break;
      uint4 v = ring[slot][i][threadIdx.x];
      if (kind < 2) {
        float2 u[4], o[4];
        unpack8(v, u);
        if (!kInter) unpack8(ring[slot][i][(threadIdx.x & ~15) | partner], o);
        float r = 1.f;
        if (a.norm) {
          float ss = sum16(dot8(u, u));
          r = rsqrt_ftz(fmaf(ss, 1.f / kD, a.eps));
          if (__any_sync(0xffffffffu, ss > kOverflow)) {
            const bool big = ss > kOverflow;
            scale8(u, big ? kDown : 1.f);
            if (!kInter) scale8(o, big ? kDown : 1.f);
            ss = sum16(dot8(u, u));
            if (big) r = rsqrt_down(ss, a.eps);
          }
        }
        if (kInter) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = swap2(u[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = __fmul2_rn(u[e], cw[e]);
        if (active) {  // values behind the rotated ones have no pair
#pragma unroll
          for (int e = 0; e < 4; ++e) u[e] = __ffma2_rn(o[e], sw[e], u[e]);
        }
        if (a.norm) scale8(u, r);
        v = pack8(u);
      }
      if (write) *out = v;
      out += ohs;
    }
    slot ^= 1;
  }
}

// Backward: the same walk, with the gradient rows behind the inputs' in the ring.  fp32
// gradients are copied as whole 256-byte runs (lane l takes 16-byte units l and l + 16) and
// put down so that the two units a lane reads, 2 l and 2 l + 1, lie 16 lanes' units apart.
// A lane sums the weight gradients of its eight values over the rows of one kind of a
// token, then into its half-warp's place in shared memory; a block leaves one partial per
// weight, which norm_rope_dw sums in block order.
// 4,096 tokens of 24 / 4 / 4 heads with fp32 gradients take 36 us with the sum (54% of the
// copy's rate), 20,011 tokens of 12 / 2 / 2 with bf16 48 us (73%): a row takes about 210
// instructions a warp and two reductions over 16 lanes, a vote between them and the next row,
// so a warp has one row's chain under way, which 16 warps an SM do not hide (63% of the
// issue slots).  Two rows a batch: 36 and 48 us where three took 35 and 47, four 39 and 47;
// three blocks an SM spill registers (81 and 76 us).
constexpr int kBwdRows = 3, kBwdCtas = 2;
template <bool kBf16> constexpr int bwd_units() { return kBf16 ? 2 : 3; }  // 16 bytes each

// A lane's eight gradients at `in`.
template <bool kBf16>
__device__ __forceinline__ void unpack_grad(const uint4* in, float2* g) {
  const uint4 p = in[kThreads];
  if (kBf16) {
    unpack8(p, g);
  } else {
    const uint4 q = in[2 * kThreads];
    g[0] = make_float2(__uint_as_float(p.x), __uint_as_float(p.y));
    g[1] = make_float2(__uint_as_float(p.z), __uint_as_float(p.w));
    g[2] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
    g[3] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
  }
}

template <bool kBf16, bool kInter>
__global__ void __launch_bounds__(kThreads, kBwdCtas)
norm_rope_bwd_kernel(const __grid_constant__ LsNormRopeArgs a, const __grid_constant__ LsRows x,
                     const __grid_constant__ LsRows dy, const __grid_constant__ LsRows dx,
                     float* part, const __grid_constant__ Spread sp) {
  constexpr int kU = bwd_units<kBf16>(), kSh = kBf16 ? 3 : 2;
  __shared__ Const cst;
  extern __shared__ __align__(16) uint4 smem[];
  uint4* ring = smem;                                                              // [2][kBwdRows][kU][kThreads]
  float* red = reinterpret_cast<float*>(smem + 2 * kBwdRows * kU * kThreads);      // [2][kGroups][128]
  const int l = threadIdx.x & 15, grp = threadIdx.x >> 4, half = grp & 1;
  float2* tab = cst.tab[grp];
  const int partner = partner_of(a, l);
  const bool active = l < a.half / 4;
  // the sum of the partials may be launched: its blocks wait for this grid
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Walk<kBwdRows> w;  // one batch ahead
  w.begin(a, sp, blockIdx.x * kWarps + (threadIdx.x >> 5));
  const uint4 *xs = nullptr, *gs = nullptr;
  int64_t xhs = 0, ghs = 0;
  auto load = [&](int to) {
    if (w.n > 0 && 2 * w.pair + half < a.T) {
      if (w.first) {
        const int64_t t = 2 * w.pair + half;
        const int32_t h = w.head(a);
        xhs = x.hs[w.kind] >> 3;
        ghs = dy.hs[w.kind] >> kSh;
        xs = static_cast<const uint4*>(x.p[w.kind]) + ((t * x.ts[w.kind] + h * x.hs[w.kind]) >> 3) + l;
        gs = static_cast<const uint4*>(dy.p[w.kind]) + ((t * dy.ts[w.kind] + h * dy.hs[w.kind]) >> kSh) + l;
      }
      uint4* d = ring + to * (kBwdRows * kU * kThreads) + threadIdx.x;
      uint4* dg = kBf16 ? d + kThreads : d - l + (l >> 1) + (1 + (l & 1)) * kThreads;
      const bool with_x = w.kind < 2 && a.norm;
#pragma unroll
      for (int i = 0; i < kBwdRows; ++i) {
        if (i < w.n) {
          if (with_x) cp_async16(d + i * (kU * kThreads), xs);
          cp_async16(dg + i * (kU * kThreads), gs);
          if (!kBf16) cp_async16(dg + i * (kU * kThreads) + 8, gs + 16);
        }
        xs += xhs;
        gs += ghs;
      }
    }
    cp_async_commit();
  };

  load(0);
  load_const(a, cst);
  for (int i = threadIdx.x; i < 2 * kGroups * kD; i += kThreads) red[i] = 0.f;
  Positions pos;
  int64_t t = 2 * w.pair + half;
  __syncthreads();
  pos.fetch(a, cst, t, l);
  Turn<kInter> turn;
  float2 wt[4], dw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[i] = make_float2(0.f, 0.f);
  bool live = false;
  int64_t pair = -1, ohs = 0;
  uint4* out = nullptr;
  int sums = -1, slot = 0;  // sums: the kind that dw belongs to
  auto flush = [&]() {
    if (sums < 0 || sums > 1) return;
    float2* p = reinterpret_cast<float2*>(red + (sums * kGroups + grp) * kD + 8 * l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = __fadd2_rn(p[i], dw[i]);
      dw[i] = make_float2(0.f, 0.f);
    }
  };

  while (w.n > 0) {
    const int n = w.n, kind = w.kind, head = w.head(a);
    const int64_t p = w.pair;
    const bool first = w.first;
    w.next(a, sp);
    __syncwarp();  // the other slot has been read by all
    load(slot ^ 1);
    if (p != pair) {
      pair = p;
      t = 2 * pair + half;
      live = t < a.T;
      pos.angles(a, cst, l, tab);
      pos.fetch(a, cst, t + 2, l);
      __syncwarp();
      turn.load(a, tab, l, partner, true);
      __syncwarp();
    }
    if (first) {
      flush();
      sums = kind;
      weights8(cst.w[kind & 1], l, wt);
      out = static_cast<uint4*>(const_cast<void*>(dx.p[kind])) +
            ((t * dx.ts[kind] + head * dx.hs[kind]) >> 3) + l;
      ohs = dx.hs[kind] >> 3;
    }
    cp_async_wait<1>();
    __syncwarp();  // the batch is there for all
#pragma unroll
    for (int i = 0; i < kBwdRows; ++i) {
      if (i >= n) break;
      const uint4* in = ring + (slot * kBwdRows + i) * (kU * kThreads) + threadIdx.x;
      float2 g[4];
      unpack_grad<kBf16>(in, g);
      if (kind < 2) {
        float2 o[4];
        if (kInter) {
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = swap2(g[e]);
        } else {
          unpack_grad<kBf16>(in - l + partner, o);
        }
        if (active) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            g[e] = __ffma2_rn(o[e], turn.s[e], __fmul2_rn(g[e], turn.c[e]));
        }
        if (a.norm) {
          float2 u[4], h[4];
          unpack8(in[0], u);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = __fmul2_rn(g[e], wt[e]);
          float ss = sum16(dot8(u, u)), hx = sum16(dot8(h, u));
          float r = rsqrt_ftz(fmaf(ss, 1.f / kD, a.eps)), r_dx = r;
          // a sum has passed fp32 (that of h and u, too, where neither's squares do)
          const bool over = !(ss + fabsf(hx) <= kOverflow);
          hx *= r;  // from here on the sum of h xh
          if (__any_sync(0xffffffffu, over)) {
            const bool big = ss > kOverflow;
            scale8(u, big ? kDown : 1.f);
            ss = sum16(dot8(u, u));
            if (big) {
              r = rsqrt_down(ss, a.eps);
              r_dx = r * kDown;
            }
            scale8(u, r);
            const float sum = sum16(dot8(h, u));
            if (over) hx = sum;  // the warp's other row keeps its bits
            r = 1.f;
          }
          scale8(u, r);
          if (live) {  // else the ring holds something older
#pragma unroll
            for (int e = 0; e < 4; ++e) dw[e] = __ffma2_rn(g[e], u[e], dw[e]);
          }
          const float2 nm = both(-hx * (1.f / kD));  // the mean of h xh
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = __fmul2_rn(__ffma2_rn(nm, u[e], h[e]), both(r_dx));
        }
      }
      if (live) *out = pack8(g);
      out += ohs;
    }
    slot ^= 1;
  }
  if (!part) return;
  flush();
  __syncthreads();
  float s = 0.f;  // 256 threads: a weight each, its 16 half-warps in order
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
    s += red[((threadIdx.x >> 7) * kGroups + i) * kD + (threadIdx.x & (kD - 1))];
  part[(int64_t)blockIdx.x * 2 * kD + threadIdx.x] = s;
}

__device__ __forceinline__ float sum32(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// dw[c] (+)= sum over blocks of part[block][c], in a fixed order: 128 chains of blocks,
// then the chains.  256 columns (queries, keys), 32 a block, 4 a thread.  3 us of latency for
// 304 partials, most of it overlapped with the end of the kernel above; in 64-bit
// sums, one thread a column, it took 14 us.
constexpr int kDwCols = 32, kDwChains = 128;
__global__ void __launch_bounds__(1024) norm_rope_dw(const float* part, int blocks,
                                                     float* dwq, float* dwk, int accumulate) {
  __shared__ float red[kDwChains][kDwCols + 1];
  const int c = threadIdx.x & 7, chain = threadIdx.x >> 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials are written
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int b = chain; b < blocks; b += kDwChains) {
    const float4 v = *(reinterpret_cast<const float4*>(part + (int64_t)b * 2 * kD + blockIdx.x * kDwCols) + c);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  red[chain][4 * c] = s.x;
  red[chain][4 * c + 1] = s.y;
  red[chain][4 * c + 2] = s.z;
  red[chain][4 * c + 3] = s.w;
  __syncthreads();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;  // a warp per column
  float sum = (red[lane][w] + red[lane + 32][w]) + (red[lane + 64][w] + red[lane + 96][w]);
  sum = sum32(sum);
  const int col = blockIdx.x * kDwCols + w;
  float* dw = col < kD ? dwq : dwk;
  if (lane || !dw) return;
  float* p = dw + (col & (kD - 1));
  *p = accumulate ? *p + sum : sum;
}

Spread spread(const LsNormRopeArgs& a, bool with_v, int max_ctas, int* ctas) {
  Spread s;
  s.rows = a.hq + (with_v ? 2 : 1) * a.hkv;
  s.total = (a.T + 1) / 2 * s.rows;
  const int64_t need = (s.total + kWarps - 1) / kWarps;
  *ctas = (int)(need < max_ctas ? need : max_ctas);
  const int64_t warps = (int64_t)*ctas * kWarps;
  s.warps = (int32_t)(s.total < warps ? s.total : warps);
  return s;
}

}  // namespace

cudaError_t ls_launch_norm_rope_fwd(const LsNormRopeArgs& a, const LsRows& x, const LsRows& y,
                                    const LsPoolDst* dst, int sms, cudaStream_t st) {
  int ctas;
  const Spread sp = spread(a, x.p[2] != nullptr, sms * kFwdCtas, &ctas);
  const LsPoolDst d = dst ? *dst : LsPoolDst{};
  if (dst && a.interleaved)
    norm_rope_fwd_kernel<true, true><<<ctas, kThreads, 0, st>>>(a, x, y, d, sp);
  else if (dst)
    norm_rope_fwd_kernel<true, false><<<ctas, kThreads, 0, st>>>(a, x, y, d, sp);
  else if (a.interleaved)
    norm_rope_fwd_kernel<false, true><<<ctas, kThreads, 0, st>>>(a, x, y, d, sp);
  else
    norm_rope_fwd_kernel<false, false><<<ctas, kThreads, 0, st>>>(a, x, y, d, sp);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}

int ls_norm_rope_bwd_ctas(int64_t T, int sms) {
  return T > 0 ? sms * kBwdCtas : 0;  // most partials a call leaves
}

cudaError_t ls_launch_norm_rope_bwd(const LsNormRopeArgs& a, const LsRows& x, const LsRows& dy,
                                    int dy_bf16, const LsRows& dx, float* dwq, float* dwk,
                                    int accumulate, float* part, int sms, cudaStream_t st) {
  const bool dw = dwq || dwk;
  int ctas = 0;
  cudaError_t e = cudaSuccess;
  if (a.T > 0) {  // no tokens: zero weight gradients only
    Spread sp = spread(a, dy.p[2] != nullptr, sms * kBwdCtas, &ctas);
    float* pt = dw ? part : nullptr;
    const int smem = 2 * kBwdRows * (dy_bf16 ? bwd_units<true>() : bwd_units<false>()) * kThreads * 16 +
                     2 * kGroups * kD * 4;
    const void* fn = dy_bf16 ? (a.interleaved ? (const void*)norm_rope_bwd_kernel<true, true>
                                              : (const void*)norm_rope_bwd_kernel<true, false>)
                             : (a.interleaved ? (const void*)norm_rope_bwd_kernel<false, true>
                                              : (const void*)norm_rope_bwd_kernel<false, false>);
    if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
      return e;
    void* args[] = {(void*)&a, (void*)&x, (void*)&dy, (void*)&dx, (void*)&pt, (void*)&sp};
    if ((e = cudaLaunchKernel(fn, dim3(ctas), dim3(kThreads), args, smem, st)) != cudaSuccess) return e;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ls_note_launch();
  }
  if (dw) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * kD / kDwCols);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = ctas > 0 ? 1 : 0;  // only behind the kernel above, which lets it start early
    e = cudaLaunchKernelEx(&cfg, norm_rope_dw, (const float*)part, ctas, dwq, dwk, accumulate);
    if (e == cudaSuccess) ls_note_launch();
  }
  return e;
}
